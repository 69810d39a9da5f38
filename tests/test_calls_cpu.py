"""The two ways the binding calls the serving entry points, without a GPU: the CPython module and plain ctypes."""
import ctypes
import importlib.util
import subprocess
import sys
import sysconfig
from pathlib import Path

import numpy as np
import pytest

import decode_attention_host_b200 as dkv

ROOT = Path(__file__).resolve().parent.parent
PKG = ROOT / "decode_attention_host_b200"
CALLS = {"extend_tables": 14, "store_kv": 13, "attn_chunk": 22, "attn_decode_window": 17}


def test_the_package_imports_and_calls_without_the_cpython_module():
    """As on a machine without Python's headers, or in a tree that was built with another Python."""
    code = """
import sys
sys.modules["decode_attention_host_b200._dkv_call"] = None      # an import of it fails
import decode_attention_host_b200 as dkv
assert type(dkv._dkv_call).__name__ == "_CtypesCalls"
try:
    dkv.dkv_attn_decode_window(None, 1, 0, 0, *[None] * 7, 0, None, None, 1, 1, 0)
except dkv.DkvError as e:
    assert e.code == dkv.DKV_ERR_INVALID_ARG and "null handle" in str(e)
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr


def test_the_cpython_module_is_named_for_one_python():
    spec = importlib.util.spec_from_file_location("dkv_build", PKG / "build.py")
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    assert build.CALL_LIB.name == "_dkv_call" + sysconfig.get_config_var("EXT_SUFFIX") != "_dkv_call.so"
    assert not (PKG / "_dkv_call.so").exists()


def ways():
    both = [dkv._CtypesCalls()]
    if not isinstance(dkv._dkv_call, dkv._CtypesCalls):
        both.append(dkv._dkv_call)
    return both


@pytest.mark.parametrize("name,n", CALLS.items())
def test_both_ways_refuse_alike(name, n):
    sig = getattr(dkv.lib, "dkv_" + name).argtypes
    assert len(sig) == n
    args = [None if t is ctypes.c_void_p else 0 for t in sig]
    number = next(i for i, t in enumerate(sig) if t is ctypes.c_int)
    for way in ways():
        f = getattr(way, name)
        assert f(*args) == dkv.DKV_ERR_INVALID_ARG      # a null handle
        with pytest.raises(TypeError):
            f(*args[1:])
        for bad, error in ((1 << 31, OverflowError), (-(1 << 31) - 1, OverflowError), (1.0, TypeError),
                           (None, TypeError)):
            with pytest.raises(error):
                f(*args[:number], bad, *args[number + 1:])


def test_both_ways_take_no_host_array_for_an_address():
    """A numpy array lies in host memory: the kernels would read its address."""
    args = [None if t is ctypes.c_void_p else 0 for t in dkv.lib.dkv_store_kv.argtypes]
    for way in ways():
        with pytest.raises(AttributeError):
            way.store_kv(args[0], np.zeros(4), *args[2:])
