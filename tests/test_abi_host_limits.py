"""Row strides whose products with the row count pass 64 bits: refused, in a child process, since
a wrapped product may also end the process."""
import os
import subprocess
import sys

import pytest

cbq = pytest.importorskip("codebook_bit_quantized_amd")

STRIDES = [1 << 28, 1 << 30, 1 << 59, 1 << 60, 1 << 61, 1 << 62, (1 << 62) + (1 << 61), (1 << 63) - 4]

CHILD = """
import ctypes, sys
import codebook_bit_quantized_amd as cbq
lib = cbq.load_library()
P = ctypes.c_void_p(0x1000)
W = ctypes.byref(cbq.cbq_weights(0x1000, 0x1000, 1, 96, 128, 4, 0))
G = (cbq.cbq_weights * 2)(*[cbq.cbq_weights(0x1000, 0x1000, 1, 96, 128, 4, 0)] * 2)
for ldo in %s:
    for T in (1, 2, 3, 4, 8, 33, 1 << 20, (1 << 31) - 1):
        %s
        assert rc == cbq.CBQ_EUNSUPPORTED and lib.cbq_last_error(), (ldo, T, rc)
print("refused")
"""

ADAPTER = """rc = lib.cbq_codebook_adapter_gemm(P, P, 4, T, W, P, 128, P, P, None, 3, 16, P, P, ldo, P, 1 << 50, None)"""


def _child(call):
    if not os.path.exists(cbq.LIB_PATH):
        pytest.skip("libcbq.so not built")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD % (STRIDES, call)], capture_output=True, text=True, cwd=root, timeout=120)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_codebook_adapter_gemm_strides():
    _child(ADAPTER)


def test_codebook_lut_gemm_strides():
    _child("rc = lib.cbq_codebook_lut_gemm(P, P, 4, T, None, None, W, 1, 0, 0, P, ldo, None, 0, None)")
    # bf16 rows: one of 2^28 elements is half a GiB, and not to be refused
    _child("if T * ldo < 1 << 29: continue\n"
           "        rc = lib.cbq_codebook_lut_gemm(P, P, 4, T, None, None, G, 2, 1, 2, P, ldo, None, 0, None)")
