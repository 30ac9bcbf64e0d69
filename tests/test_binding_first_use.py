"""The binding's first calls: several threads at once."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

THREADS = """
import importlib, threading, time, traceback
import torch, tensor_sharded_linear_gqa_gb300 as tp
slow, load = threading.Event(), importlib.import_module
def late(name, package=None):
    if name == "._describe":
        slow.set()
        time.sleep(0.3)
    return load(name, package)
importlib.import_module = late
empty, one = torch.empty(0, dtype=torch.float32), tp.TpTensor(16, tp.TP_F32, 0, 2, 8, 8)
calls = [lambda: tp._dev_ptr(empty, "torch.float32"), lambda: tp._args(2).one(one), lambda: tp._args(2).many([one, one], 2),
         lambda: tp._args(2).row(one), lambda: tp._workspace(empty), lambda: tp._describe, lambda: tp.tensor(torch.empty(0, 4)),
         lambda: tp._entry("rotary")]
wrong = []
def use(call):
    try:
        call()
    except BaseException:
        wrong.append(traceback.format_exc()[-400:])
first = threading.Thread(target=use, args=(calls[FIRST],))
first.start()
assert slow.wait(60)
rest = [threading.Thread(target=use, args=(c,)) for c in calls]
for t in rest: t.start()
for t in [first] + rest: t.join(60)
assert not wrong, wrong
assert tp._entry("rotary") is tp._entry("rotary")
"""


@pytest.mark.parametrize("first", [0, 1, 2, 5, 6])
def test_threads_that_call_while_the_module_is_loaded(first):
    r = subprocess.run([sys.executable, "-c", THREADS.replace("FIRST", str(first))], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
