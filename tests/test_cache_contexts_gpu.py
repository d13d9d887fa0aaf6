"""The 8-bit cache's calls in contexts of the caller's own (driver API), made, destroyed and made again, the way a plugin hosted by
another runtime uses the C library: what a kernel needs set in a context has to be set in each.  PyTorch's CUDA state is never
touched in the child."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_CHILD = r'''
import ctypes, sys
import numpy as np
sys.path.insert(0, sys.argv[1])
from attention_flash_attn_gb300 import _capi

cu = ctypes.CDLL("libcuda.so.1")
def ck(r, what):
    if r != 0:
        raise SystemExit(f"{what}: CUresult {r}")
ck(cu.cuInit(0), "cuInit")
dev = ctypes.c_int()
ck(cu.cuDeviceGet(ctypes.byref(dev), 0), "cuDeviceGet")
L = _capi.lib()
r = ctypes.byref
H, page, pages, n = 2, 64, 300, 300 * 64 - 5       # an eviction that selects with more than 48 KB
rng = np.random.default_rng(3)
table = rng.permutation(pages).astype(np.int32)
scales = np.full((pages + 2, H), 2.0 ** -6, np.float32)
weights = rng.random((H, pages * page), np.float32)

def case(D, Hq, Sq, dtype, primary=False):
    """One sequence: attention (scores and weights too), then an eviction to 100 tokens; in a new context, ended behind it."""
    ctx = ctypes.c_void_p()
    if primary:
        ck(cu.cuDevicePrimaryCtxRetain(r(ctx), dev), "cuDevicePrimaryCtxRetain")
        ck(cu.cuCtxSetCurrent(ctx), "cuCtxSetCurrent")
    else:
        ck(cu.cuCtxCreate_v2(r(ctx), 0, dev), "cuCtxCreate")
    bufs = []
    def up(a):
        p = ctypes.c_uint64()
        ck(cu.cuMemAlloc_v2(r(p), ctypes.c_size_t(max(256, a.nbytes))), "cuMemAlloc")
        ck(cu.cuMemcpyHtoD_v2(p, a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes)), "HtoD")
        bufs.append(p)
        return p.value
    def down(p, a):
        ck(cu.cuMemcpyDtoH_v2(a.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(p), ctypes.c_size_t(a.nbytes)), "DtoH")
        return a
    g = np.random.default_rng(D + Sq)
    codes = [g.integers(-127, 128, (pages + 2, H, page, D), np.int8) for _ in range(2)]
    q = g.normal(0, 1, (Sq, Hq, D)).astype(np.float32)
    if dtype == 1:
        q = (q.view(np.uint32) >> 16).astype(np.uint16)   # bf16 by truncation
    c = _capi.AttnCacheArgs(_capi.ATTN_CACHE_INT8, pages + 2, page, H, D, up(codes[0]), up(codes[1]), up(scales), up(scales),
                            up(np.zeros(256, np.uint8)))
    s = _capi.AttnCacheSeqs(1, pages, up(table), pages, up(np.array([n], np.int32)))
    w = up(weights)
    a = _capi.AttnCacheFwdArgs(dtype, Sq, Hq, up(q), Sq * Hq * D, Hq * D, D, 1, 0, 0.0, 0.1, None, 0, w, w, H * pages * page, pages * page)
    path = L.attn_cache_path_name(r(c), r(s), r(a)).decode()
    need = L.attn_cache_fwd_workspace_size(r(c), r(s), r(a))
    O, LSE = np.zeros_like(q), np.zeros((Hq, Sq), np.float32)
    dO, dL, ws = up(O), up(LSE), up(np.zeros(need, np.uint8))
    st = L.attn_cache_fwd(r(c), r(s), r(a), dO, dL, ws, need, None)
    if st != 0:
        raise SystemExit(f"attn_cache_fwd ({path}, D = {D}): {st}")
    kept, left = np.zeros((H, 100), np.int32), np.zeros((H, 100), np.float32)
    dk, dl = up(kept), up(left)
    e = _capi.AttnCacheEvictArgs(100, 4, 10, w, H * pages * page, pages * page, up(np.array([pages, pages + 1], np.int32)), 2, dk,
                                 up(np.zeros(1, np.int32)), dl)
    st = L.attn_cache_evict(r(c), r(s), r(e), None)
    if st != 0:
        raise SystemExit(f"attn_cache_evict: {st}")
    ck(cu.cuCtxSynchronize(), "sync")
    st = L.attn_check_device_status(c.status, None)
    if st != 0:
        raise SystemExit(f"status: {st}")
    out = [down(dO, O), down(dL, LSE), down(dk, kept), down(dl, left)]
    for p in bufs:
        ck(cu.cuMemFree_v2(p), "cuMemFree")
    if primary:
        ck(cu.cuCtxSetCurrent(None), "cuCtxSetCurrent")
        ck(cu.cuDevicePrimaryCtxRelease_v2(dev), "cuDevicePrimaryCtxRelease")
        ck(cu.cuDevicePrimaryCtxReset_v2(dev), "cuDevicePrimaryCtxReset")
    else:
        ck(cu.cuCtxDestroy_v2(ctx), "cuCtxDestroy")
    return path, codes, out

paths = set()
for D, Hq, Sq, dtype in ((64, 8, 1, 1), (128, 8, 1, 1), (128, 40, 1, 1), (256, 8, 1, 1), (128, 8, 1, 2), (128, 64, 4, 1), (64, 256, 4, 1),
                         (320, 2, 1, 2)):
    path, codes, one = case(D, Hq, Sq, dtype)
    paths.add(path)
    for primary in (False, True, True):
        _, _, two = case(D, Hq, Sq, dtype, primary)
        assert all(np.array_equal(x, y) for x, y in zip(one, two)), (path, D, primary)
    # The last query's LSE of the first head against float64, and the eviction's order.
    q = np.random.default_rng(D + Sq)
    for _ in range(2):
        q.integers(-127, 128, (pages + 2, H, page, D), np.int8)
    q = q.normal(0, 1, (Sq, Hq, D)).astype(np.float32)
    if dtype == 1:
        q = ((q.view(np.uint32) >> 16) << 16).view(np.float32)
    k = codes[0][table, 0].reshape(-1, D)[:n].astype(np.float64) * 2.0 ** -6
    t = 0.1 * (k @ q[-1, 0].astype(np.float64))
    want = t.max() + np.log(np.exp(t - t.max()).sum())
    assert abs(one[1][0, -1] - want) < 1e-3 * abs(want), (path, D, one[1][0, -1], want)
    assert (np.diff(one[2], axis=1) > 0).all() and (one[2][:, :4] == np.arange(4)).all()
assert paths == {"tc", "mma", "simt"}, paths
print("ok")
'''


def test_calls_in_contexts_made_one_after_another():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHILD, root], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.stdout[-2000:], r.stderr[-4000:])
