"""What the norm and optimiser calls do with their tensors on the host: no GPU is needed."""
import gc
import subprocess
import sys
import weakref

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import linear_cross_entropy_03_gb300 as flce
from linear_cross_entropy_03_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return flce.lib()


def test_a_failing_call_lets_go_of_its_gradients():
    """A tensor without memory makes torch throw inside the extension: what an iterator yielded goes all the same."""
    with FakeTensorMode():
        held = [torch.empty(4, device="cuda")]
    seen = weakref.ref(held[0])

    def yields():
        yield held.pop()

    with pytest.raises(RuntimeError):
        flce.grad_norm(yields())
    gc.collect()
    assert seen() is None


# ------------------------------------------------------------ the largest tensors

FAKE, FAR = 0x10000, 1 << 40   # never dereferenced by a refused call
INVALID = 1


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [(1 << 41) + 1, 1 << 42, 1 << 62])
def test_a_tensor_too_long_for_a_launch_is_refused(n, bits):
    """A step over such a tensor of 8-bit moments did nothing, to it and to those after it, and returned no error."""
    scales = dict(exp_avg_scale=FAKE, exp_avg_sq_scale=FAKE) if bits == 8 else {}
    table = (flce.AdamWEntry * 1)(flce.AdamWEntry(
        param=FAKE, grad=FAR, exp_avg=2 * FAR, exp_avg_sq=3 * FAR, n=n, lr_scale=1.0, weight_decay=0.1, param_dtype=1,
        grad_dtype=1, moment_bits=bits, **scales))
    numbers = flce.AdamWNumbers(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=1.0)
    assert flce.adamw_step(table, 1, numbers, 0) == INVALID


@pytest.mark.parametrize("dtype,n,count", [(1, 1 << 41, 9), (1, 1 << 40, 17), (0, 1 << 41, 17), (1, 1 << 41, 4000)])
def test_gradients_that_make_more_launches_than_the_workspace_is_for_are_refused(dtype, n, count):
    """Launches that ended early, at 2^31 chunks, had their partial sums written past the stated size."""
    table = (flce.TensorEntry * count)(*[flce.TensorEntry(FAKE, n, dtype, 0)] * count)
    size = flce.grad_norm_workspace_size(count)
    assert flce.grad_norm_raw(table, count, 1.0, 1.0, 1e-6, FAKE, FAKE, size, 0) == INVALID


# ------------------------------------------------------------ a build without the extension

@pytest.mark.parametrize("without", ["torch", "Python.h"])
def test_the_library_is_built_where_the_extension_cannot_be(without, monkeypatch, tmp_path):
    """C callers need neither torch nor Python's headers."""
    ran = []

    def run(what, cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libflce03.so"))
    if without == "torch":
        monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
        monkeypatch.setitem(sys.modules, "torch", None)      # `import torch` raises
    else:
        monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert not _build.up_to_date()
    with pytest.warns(UserWarning, match="only the library"):
        assert _build.build() == _build.LIB
    assert (tmp_path / "libflce03.so").exists() and not any("binding" in part for cmd in ran for part in cmd)
    assert _build.up_to_date()
    del ran[:]
    assert _build.build() == _build.LIB and ran == []        # and not again


def test_a_build_that_fails_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libflce03.so"))
    monkeypatch.setattr(_build, "_nvcc", lambda: sys.executable)
    monkeypatch.setenv("CXX", sys.executable)
    with pytest.raises(RuntimeError, match="failed"):
        _build.build()


def test_the_build_runs_as_a_program():
    """As the README has it, without a warning."""
    r = subprocess.run([sys.executable, "-W", "error::RuntimeWarning", "-m", _build.__name__], capture_output=True,
                       text=True, cwd=_build.ROOT)
    assert r.returncode == 0 and r.stdout.strip() == _build.LIB, r.stderr
