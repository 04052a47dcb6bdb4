"""libw4 over the recording CUDA runtime of fake_cuda.cpp: what a call
enqueues, without a GPU."""
import ctypes
import glob
import os
import shutil
import subprocess

import int4_weight_mixed_gb300 as w4

HERE = os.path.dirname(os.path.abspath(__file__))


class Recorder:
    def __init__(self, path):
        self.lib = ctypes.CDLL(path)
        real = w4.load()
        for name in dir(real):
            if name.startswith("w4_") and getattr(real, name).argtypes is not None:
                fn = getattr(self.lib, name)
                fn.argtypes, fn.restype = getattr(real, name).argtypes, getattr(real, name).restype
        self.lib.w4_schedule_name.restype = ctypes.c_char_p
        self.lib.w4_last_error.restype = ctypes.c_char_p
        self.lib.fake_thread.restype = ctypes.c_uint64
        self.lib.fake_kernel.restype = ctypes.c_char_p

    def reset(self, pause_us=0):
        """Forgets the launches; each of the next ones takes pause_us more."""
        self.lib.fake_reset(pause_us)

    def launches(self):
        """(thread, mangled kernel name) in the order they were enqueued."""
        return [(self.lib.fake_thread(i), self.lib.fake_kernel(i).decode())
                for i in range(self.lib.fake_count())]


def build(folder):
    """libw4's objects and the recording runtime as one library in `folder`."""
    w4.build()
    w4.load()
    objs = [os.path.join(w4._build_lib.BUILD, s.replace(".cu", ".o"))
            for s in w4._build_lib.SOURCES]
    nvcc = os.path.realpath(w4._build_lib._nvcc())
    inc = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    out = os.path.join(str(folder), "libw4_recorded.so")
    subprocess.check_call([shutil.which("g++") or "g++", "-O1", "-std=c++17", "-shared", "-fPIC",
                           "-I", inc, os.path.join(HERE, "fake_cuda.cpp"), *objs,
                           "-Wl,-Bsymbolic", "-Wl,--no-undefined", "-lpthread", "-o", out])
    return Recorder(out)
