"""What the package loads and when: nothing of its own is mapped until a call needs it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def mapped(code):
    """Objects of the repository that a fresh interpreter has mapped after `code`."""
    if not os.path.exists("/proc/self/maps"):
        pytest.skip("no /proc/self/maps")
    code += "\nprint(*[l.split()[-1] for l in open('/proc/self/maps') if '.so' in l])"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, check=True)
    return {os.path.basename(p) for p in r.stdout.split() if os.path.realpath(p).startswith(os.path.realpath(ROOT) + os.sep)}


def test_import_maps_nothing():
    assert mapped("from tensor_sharded_linear_gqa_gb300 import inputs") == set()
    assert mapped("import tensor_sharded_linear_gqa_gb300 as tp\ntp.TpTensor()") == set()


def test_the_first_described_tensor_loads_the_extension_module():
    torch = pytest.importorskip("torch")  # noqa: F841
    import tensor_sharded_linear_gqa_gb300 as tp
    if tp._describe is None:
        pytest.skip("the extension module is not built")
    code = "import torch, tensor_sharded_linear_gqa_gb300 as tp\ns = tp._Scratch(4)\ntp._args(4).one(torch.empty(0, 4))"
    assert mapped(code) == {"_describe.so"}


def test_without_the_extension_module_interpreted_code_describes():
    pytest.importorskip("torch")
    code = ("import sys, torch\nsys.modules['tensor_sharded_linear_gqa_gb300._describe'] = None\n"
            "import tensor_sharded_linear_gqa_gb300 as tp\n"
            "s = tp._args(8)\nd = tp.TpTensor(16, tp.TP_F32, 0, 2, 8, 8)\n"
            "first = s.many([torch.empty(0, 4), d], 2)\ns.row(d)\n"
            "assert tp._describe is None and s.used == 3 * tp._DESC_SIZE\n"
            "assert bytes(s.buf[tp._DESC_SIZE:2 * tp._DESC_SIZE]) == bytes(d)")
    assert mapped(code) == set()
