"""Every entry point of the binding makes its tensors' GPU the current one for
the call (the library plans for and launches on the current device), and
leaves the caller's as it was.  On the host: stand-ins for tensors of a second
GPU, and for what would run on it."""
import contextlib
import os
import shutil
import subprocess
import sys

import pytest
import torch

import int4_weight_mixed_gb300 as w4


class Tensor:
    """What the binding reads of a tensor on GPU 1."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float16, index=1):
        self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", index)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


@pytest.fixture
def gpu(monkeypatch):
    """The current device as the binding sees it, and the devices that were
    current when something reached the library or an allocation."""
    state = {"current": 0, "seen": [], "switched": 0}

    @contextlib.contextmanager
    def device(dev):
        before, state["current"] = state["current"], torch.device(dev).index
        state["switched"] += 1
        try:
            yield
        finally:
            state["current"] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                state["seen"].append((name, state["current"]))
                return 0
            return call

    class Host(Library):  # what it does with tensors of another device is tested below
        def __getattr__(self, name):
            call = super().__getattr__(name)
            return lambda t, *args: (call(t, *args) if t.device.index == state["current"]
                                     else NotImplemented)

    def made(*args, **kw):
        state["seen"].append(("torch.empty", state["current"]))
        return Tensor(4, 128)

    def capturing():
        state["seen"].append(("capturing", state["current"]))
        return False

    monkeypatch.setattr(w4, "_current_index", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", capturing)
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: made())
    monkeypatch.setattr(w4, "load", lambda: Library())
    monkeypatch.setattr(w4, "_lib", Library())
    monkeypatch.setattr(w4, "_host", Host())
    monkeypatch.setattr(w4, "_ws_cache", {})
    monkeypatch.setattr(w4, "_stream", lambda dev: 0)
    return state


def _calls(i):
    a = lambda: Tensor(4, 128, index=i)
    b = lambda: Tensor(8192, dtype=torch.uint8, index=i)
    s = lambda: Tensor(1, 128, index=i)
    q = lambda: Tensor(4, 128, dtype=torch.int8, index=i)
    return {
        "prepack_B": lambda: w4.prepack_B(Tensor(16, 128, dtype=torch.int32, index=i), 0, 0, 128, 128),
        "unprepack_B": lambda: w4.unprepack_B(b(), 0, 0, 128, 128),
        "workspace": lambda: w4.workspace(torch.device("cuda", i), 1024),
        "gemm": lambda: w4.gemm(a(), b(), 0, 128, scales=s()),
        "gemm, bias": lambda: w4.gemm(a(), b(), 0, 128, scales=s(), bias=Tensor(128, index=i)),
        "gemm, epilogue": lambda: w4.gemm(a(), b(), 0, 128, scales=s(), act=w4.ACT_SILU),
        "gemm, by keywords": lambda: w4.gemm(a=a(), b_packed=b(), wtype=0, N=128, scales=s(),
                                             residual=a()),
        "gemm_dynamic": lambda: w4.gemm_dynamic(a(), b(), 2, 128),
        "gemm_dynamic, epilogue": lambda: w4.gemm_dynamic(a(), b(), 2, 128, gated=True),
        "quantize_per_token": lambda: w4.quantize_per_token(
            a(), q(), Tensor(4, dtype=torch.float32, index=i)),
        "quantize_per_token_fp8": lambda: w4.quantize_per_token_fp8(
            a(), Tensor(4, 128, dtype=torch.float8_e4m3fn, index=i),
            Tensor(4, dtype=torch.float32, index=i)),
        "rmsnorm": lambda: w4.rmsnorm(a()),
        "rmsnorm_quant": lambda: w4.rmsnorm_quant(a(), residual=a()),
        "check_status": lambda: w4.check_status(Tensor(1024, dtype=torch.uint8, index=i)),
    }


@pytest.mark.parametrize("name", list(_calls(1)))
def test_the_tensors_gpu_is_current_during_a_call(gpu, name):
    _calls(1)[name]()
    seen = [c for c in gpu["seen"] if c[0] not in ("w4_prepacked_size",)]
    assert seen and all(dev == 1 for _, dev in seen), seen
    assert gpu["current"] == 0
    # nothing is switched for tensors of the current GPU
    gpu["switched"] = 0
    _calls(0)[name]()
    assert gpu["switched"] == 0 and gpu["seen"][-1][1] == 0


def test_an_error_leaves_the_callers_gpu(gpu, monkeypatch):
    class Refuses:
        def norm(self, x, *args):
            if x.device.index != gpu["current"]:
                return NotImplemented
            raise ValueError("refused")

    monkeypatch.setattr(w4, "_host", Refuses())
    with pytest.raises(ValueError, match="refused"):
        w4.rmsnorm(Tensor(4, 128))
    assert gpu["current"] == 0


# Tensors of a GPU that is not there, through DLPack: nothing reads their
# memory, and with GPU 0 current the extension module must not go on to a
# stream, an allocation or the library.
ANOTHER_GPU = """
import ctypes
import torch
import int4_weight_mixed_gb300 as w4

torch.cuda._initialized = True  # (a machine without a GPU)
i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class Tensor(ctypes.Structure):
    _fields_ = [("data", p), ("device_type", i32), ("device_id", i32), ("ndim", i32),
                ("code", ctypes.c_uint8), ("bits", ctypes.c_uint8), ("lanes", ctypes.c_uint16),
                ("shape", ctypes.POINTER(i64)), ("strides", ctypes.POINTER(i64)),
                ("byte_offset", ctypes.c_uint64), ("manager", p), ("deleter", p)]


capsule = ctypes.pythonapi.PyCapsule_New
capsule.restype, capsule.argtypes = ctypes.py_object, [p, ctypes.c_char_p, p]
keep = []


def tensor(*shape, code=2, bits=16):
    dims = (i64 * len(shape))(*shape)
    t = Tensor(data=0x10000, device_type=2, device_id=1, ndim=len(shape), code=code, bits=bits,
               lanes=1, shape=dims)
    keep.append((t, dims))
    return torch._C._from_dlpack(capsule(ctypes.addressof(t), b"dltensor", None))


w4._load_host()
x, b, s = tensor(4, 128), tensor(8192, code=1, bits=8), tensor(1, 128)
assert x.device == torch.device("cuda", 1) and x.dtype == torch.float16
for done in (w4._host.norm(x, None, 1e-6, x, None, None, None, -1),
             w4._host.norm(x, None, 1e-6, None, None, None, None, w4.S8),
             w4._host.gemm(x, b, 0, 128, s, None, -1, None, None, -1, None, None, -1, None, 2, False,
                           None),
             w4._host.gemm_dynamic(x, b, 2, 128, w4.S8, None, -1, None, None, None, None, None, 2,
                                   False, None)):
    assert done is NotImplemented, done
print("another GPU: ok")
"""


def test_the_extension_module_hands_back_another_gpus_tensors(tmp_path):
    if torch.cuda.is_available():
        pytest.skip("on the host: needs no GPU in the machine")
    w4.build()
    src, so = tmp_path / "current.c", tmp_path / "current.so"
    src.write_text("int cudaGetDevice(int* d) { *d = 0; return 0; }\n")
    subprocess.check_call([shutil.which("gcc") or "gcc", "-shared", "-fPIC", str(src), "-o", str(so)])
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", ANOTHER_GPU], cwd=root, capture_output=True,
                          text=True, env=dict(os.environ, LD_PRELOAD=str(so)))
    assert "another GPU: ok" in done.stdout, done.stderr[-2000:]
