"""The attention's choice of its two forms (host code of csrc/kv_paged.cuh)."""
import ctypes
import functools
import os
import subprocess
import tempfile

from nvfp4_w4a4_quantized_04_b200 import build as nvbuild

SOURCE = r"""
#include "kv_paged.cuh"
extern "C" int forms(long long batch, long long tokens, long long max_query, int group, int heads_kv, long long keys,
                     int offsets, int sms) {
  const nvfp4::kv::Forms f = nvfp4::kv::choose_forms(batch, tokens, max_query, group, heads_kv, keys, offsets != 0, sms);
  return f.row_cap * 2 + f.prefill;
}
"""


@functools.lru_cache(maxsize=None)
def _lib():
    d = tempfile.mkdtemp(prefix="forms")
    src, so = os.path.join(d, "f.cpp"), os.path.join(d, "f.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + nvbuild.CSRC, src, "-o", so])
    lib = ctypes.CDLL(so)
    i64 = ctypes.c_longlong
    lib.forms.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, i64, ctypes.c_int, ctypes.c_int]
    return lib


def choose_forms(batch, tokens, max_query, group, heads_kv, keys, offsets=True, sms=148):
    """(most rows of a sequence that the decode form takes, 0 = none; whether the prefill form runs)"""
    f = _lib().forms(batch, tokens, max_query, group, heads_kv, keys, int(offsets), sms)
    return f >> 1, bool(f & 1)
