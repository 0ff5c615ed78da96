"""The paged calls in a CUDA context that was destroyed and made again: what a call remembers from
one step to the next must not outlive its context. In a process of its own, through the driver
API, since resetting a device ends what else its process has there."""

from __future__ import annotations

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

CHILD = """
import ctypes as C
import struct
import mass_adaptive_causal_b200 as mala

cu, L = C.CDLL("libcuda.so.1"), mala.lib()


def ok(code):
    assert code == 0, code


def alloc(data):
    p = C.c_uint64()
    ok(cu.cuMemAlloc_v2(C.byref(p), C.c_size_t(max(256, len(data)))))
    ok(cu.cuMemcpyHtoD_v2(p, data, C.c_size_t(len(data))))
    return p.value


def steps(dev):
    ctx = C.c_void_p()
    ok(cu.cuDevicePrimaryCtxRetain(C.byref(ctx), dev))
    ok(cu.cuCtxSetCurrent(ctx))
    # one page of sixteen tokens, values 1, in a table of sixteen entries
    k, v = alloc(bytes(16 * 128)), alloc(b"\\x38" * (16 * 128))
    scale, table, lens = alloc(struct.pack("f", 1.0)), alloc(bytes(64)), alloc(struct.pack("i", 5))
    cache = mala._CacheStruct(k, v, scale, scale, table, 2048, 2048, 128, 2048, 2048, 128, 16, 1, 16,
                              16, 1, 128)
    for heads, tau, bound in ((1, 0.0, 16), (1, 1.0, 256), (8, 0.0, 16), (8, 1.0, 256)):
        q, o = alloc(bytes(256 * heads)), alloc(b"\\xff" * 256 * heads)
        ok(L.mala_decode_paged(C.addressof(cache), q, o, lens, 1, heads, bound, tau, 0.0, 0, None, None,
                               None))
        ok(L.mala_check(None))
        out = C.create_string_buffer(256 * heads)
        ok(cu.cuMemcpyDtoH_v2(out, C.c_uint64(o), C.c_size_t(256 * heads)))
        assert out.raw == b"\\x80\\x3f" * 128 * heads


ok(cu.cuInit(0))
dev = C.c_int()
ok(cu.cuDeviceGet(C.byref(dev), 0))
steps(dev)
ok(cu.cuDevicePrimaryCtxReset_v2(dev))
steps(dev)
"""


def test_decode_after_its_context_was_reset():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
