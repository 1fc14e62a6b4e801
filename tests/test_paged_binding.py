"""The extension module of the paged cache's calls, with the library's entry points replaced by functions that look at
the interpreter: no GPU is needed, and nothing launches."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = """
extern "C" int PyGILState_Check(void);
static int calls;
extern "C" { int stub_fails = 0; }
static int look() { ++calls; return PyGILState_Check() || stub_fails; }   // status 1: an error
extern "C" int mla_append_paged(...) { return look(); }
extern "C" int mla_tree_plan(...) { return look(); }
extern "C" int mla_decode_attend_paged(...) { return look(); }
extern "C" int mla_commit_paged(...) { return look(); }
extern "C" int stub_calls() { return calls; }
"""

SCRIPT = """
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)   # ahead of the library, whose symbols the module finds after it
import torch
from mla_latent_kv_12_gb300 import mla
from tests import test_paged_host as T
mla._native.setup(mla.MLAError, lambda: -1, lambda device: 0)   # CPU tensors are on device -1
for n, (name, (call, _)) in enumerate(T.CALLS.items()):
    try:
        call(mla, T.tensors())
    except mla.MLAError:
        sys.exit(f"{name}: the interpreter's lock is held during the call")
    assert stub.stub_calls() == n + 1, name
ctypes.c_int.in_dll(stub, "stub_fails").value = 1   # an error status still becomes an exception
for call, _ in T.CALLS.values():
    try:
        call(mla, T.tensors())
        sys.exit("no exception")
    except mla.MLAError:
        pass
print("ok")
"""


def test_other_threads_run_during_a_call(tmp_path):
    """A launch waits while its stream's queue is full; what empties the queue may need another Python thread."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, lib = tmp_path / "stub.cpp", tmp_path / "libstub.so"
    src.write_text(STUB)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", str(src), "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(SCRIPT), str(lib)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_an_array_listed_twice_is_refused():
    """Its rows would be moved by two workers at once.  (The pointers are no device memory: nothing may launch.)"""
    from mla_latent_kv_12_gb300 import mla
    mb = 1 << 20
    for order in ([0, 1, 2, 1], [3, 2, 1, 3], [5, 5], list(range(250)) + [17]):
        states = (mla.StateArray * len(order))()
        for s, k in zip(states, order):
            s.data, s.token_stride_bytes, s.batch_stride_bytes, s.row_bytes = mb * (k + 1), 1024, 16384, 1024
        assert mla.lib.mla_commit_paged(states, len(order), mb, 8, 8, 16, 100, mb, mb, 16, 16, mb, None, 4, None, None) == 1
        assert "twice" in mla.lib.mla_last_error_detail().decode()
