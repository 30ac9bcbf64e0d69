"""The extension module reads tensors through the layout of the torch that it was built with, and of no other; callers
who pass descriptors and addresses need no torch at all."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import tensor_sharded_linear_gqa_gb300 as tp
from tensor_sharded_linear_gqa_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = f"{torch.version.__version__} {torch.version.git_version}"


def run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120, env=dict(os.environ, **env))
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_build_knows_the_installed_torch():
    assert build._torch() == (HERE, os.path.dirname(torch.__file__))


@pytest.mark.skipif(tp._describe is None, reason="the extension module is not built")
def test_another_torch_than_the_one_of_the_build():
    other = ("import torch\ntorch.version.git_version = '0' * 40\nimport tensor_sharded_linear_gqa_gb300 as tp\n"
             "d = tp._load_describe()\nseen = []\n")
    # asked with the version at hand on the first use, and from then on without torch's layout
    run(other + f"assert d.reads_torch({HERE!r}) in (False, True) and not d.reads_torch({HERE!r} + 'a')\n"
        "for v in ('', '2', '2.0.0 0'): assert not d.reads_torch(v)\n")
    run(other + "import types\nasked = []\n"
        "tp._loaded, fake = False, types.SimpleNamespace(**{n: getattr(d, n) for n in dir(d) if n[0] != '_'})\n"
        "fake.reads_torch = asked.append\n"
        "tp.importlib = types.SimpleNamespace(import_module=lambda *a: fake)\n"
        "tp._load_describe()\nassert asked == [torch.version.__version__ + ' ' + '0' * 40], asked\n")
    for bad in ((), (1,), (HERE, HERE)):
        with pytest.raises(TypeError):
            tp._describe.reads_torch(*bad)


@pytest.mark.parametrize("error", ["OSError('libc10.so')", "ImportError('x')", "RuntimeError('x')"])
def test_descriptors_without_a_torch_that_loads(tmp_path, error):
    os.makedirs(tmp_path / "torch")
    (tmp_path / "torch" / "__init__.py").write_text(f"raise {error}\n")
    run("import tensor_sharded_linear_gqa_gb300 as tp\n"
        "plan = tp.tp_plan_create(1, 512, 4, 2, 128, 64)\n"
        "t = lambda rows, cols, p: tp.TpTensor(p << 40, tp.TP_BF16, 0, rows, cols, cols)\n"
        "q, k = t(4, 512, 1), t(9, 256, 2)\n"
        "s = tp._args(4)\ns.one(q)\ns.many([q, k], 2)\ns.row(t(1, 8, 1))\nassert s.used == 4 * tp._DESC_SIZE\n"
        "for call in (lambda: tp.tp_window_attn(plan, [q], [k], [k], 0, 0, [q], stream=1),\n"
        "             lambda: tp.tp_add_rmsnorm(q, None, t(1, 512, 1), 1e-5, None, k, stream=1)):\n"
        "    try:\n        call()\n        raise SystemExit('not refused')\n    except tp.TPError:\n        pass\n",
        PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))


def test_a_torch_that_comes_after_the_first_use(tmp_path):
    os.makedirs(tmp_path / "torch")
    (tmp_path / "torch" / "__init__.py").write_text("raise ImportError('not yet')\n")
    run("import sys, tensor_sharded_linear_gqa_gb300 as tp\n"
        "tp._args(2).one(tp.TpTensor(16, tp.TP_F32, 0, 2, 8, 8))\n"
        "for _ in range(2):\n"
        "    try:\n        tp._dtypes()\n        raise SystemExit('no torch, and no error')\n    except ImportError as e:\n        assert 'not yet' in str(e)\n"
        f"sys.path.remove({str(tmp_path)!r})\n"
        "import torch\n"
        "assert tp.tensor(torch.empty(0, 4)).dtype == tp.TP_F32 and tp._args(1).one(torch.empty(0, 4))\n",
        PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))


@pytest.mark.gpu
def test_cuda_tensors_by_their_attributes():
    from gpu_util import need_gpu
    need_gpu()
    import ctypes
    d, out = tp._load_describe(), tp.TpTensor()
    t, n = torch.zeros(6, 64, device="cuda")[:, 8:40], torch.zeros(5, device="cuda", dtype=torch.int32)
    direct = d.reads_torch(HERE)
    try:
        assert d.vector(n, 4, 5) == (n.data_ptr() if direct else None)
        assert not d.reads_torch("another")
        assert d.matrix(t, ctypes.addressof(out))
        assert (out.ptr, out.dtype, out.rows, out.cols, out.ld) == (t.data_ptr(), tp.TP_F32, 6, 32, 64)
        assert d.vector(n, 4, 5) is None and d.bytes(n) is None
        assert tp._dev_ptr(n, "torch.int32", 5) == n.data_ptr() and tp._workspace(n) == (n.data_ptr(), 20)
    finally:
        d.reads_torch(HERE)
