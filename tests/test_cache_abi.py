"""Refusals of ssa_rope_axes and of the 8-bit cache's calls: every call here fails
validation on the host, before any CUDA call.  Also pins of the plain forms that
the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from block_top_sparse_b200 import _lib as L
from block_top_sparse_b200 import build as B

from . import cache_ref as R

P = ctypes.c_void_p(256)  # never read: validation fails first
ODD = ctypes.c_void_p(264)
INV, UNS, WS = L.SSA_ERR_INVALID_ARG, L.SSA_ERR_UNSUPPORTED, L.SSA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return L.load()


def dims(**over):
    base = dict(B=2, H=8, T=1024, d=128, s=64, k=0, dtype=0, scale=0.088, Hkv=2)
    base.update(over)
    return L.Dims(base["B"], base["H"], base["T"], base["d"], base["s"], base["k"], base["dtype"], base["scale"],
                  base["Hkv"])


def ref(d):
    return None if d is None else ctypes.byref(d)


def append(d, n=4, cache_len=P, n_new=None, K=P, ks=None, V=P, vs=None, K8=P, Ks=P, V8=P, Vs=P, Kbar=P):
    return L.load().ssa_cache_append(ref(d), n, cache_len, n_new, K, ks, V, vs, K8, Ks, V8, Vs, Kbar, None)


def decode(d, cache_len=P, q=P, K8=P, Ks=P, V8=P, Vs=P, Kbar=P, idx=P, o=P, lse=P, win=None, wout=None, ws=P,
           ws_bytes=1 << 40):
    return L.load().ssa_cache_decode(ref(d), cache_len, q, K8, Ks, V8, Vs, Kbar, idx, o, lse, win, wout, ws, ws_bytes,
                                     None)


def evict(d, keep=4, sink=0, recent=0, cache_len=P, new_len=P, win=P, wout=P, K8=P, Ks=P, V8=P, Vs=P, Kbar=P, kept=P,
          ws=P, ws_bytes=1 << 40):
    return L.load().ssa_cache_evict(ref(d), keep, sink, recent, cache_len, new_len, win, wout, K8, Ks, V8, Vs, Kbar, kept,
                                    ws, ws_bytes, None)


BAD = [(dict(B=0), INV), (dict(T=-64), INV), (dict(T=1000), UNS), (dict(d=64), UNS), (dict(s=32), UNS),
       (dict(dtype=1), UNS), (dict(dtype=7), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
       (dict(H=7), INV), (dict(Hkv=-1), INV), (dict(k=-1), INV), (dict(k=17), INV),
       (dict(T=64 * 8193), UNS),                       # blocks beyond the selection's shared memory
       (dict(B=4096, T=64 * 8192), UNS)]               # cache rows beyond int32


@pytest.mark.parametrize("over,code", BAD)
def test_shapes(over, code):
    d = dims(**over)
    assert append(d) == code
    assert decode(d) == code
    assert evict(d) == code
    assert L.ssa_workspace_size(d, L.SSA_OP_CACHE_DECODE) == 0
    assert L.ssa_workspace_size(d, L.SSA_OP_CACHE_EVICT) == 0


def test_append_refusals():
    d = dims()
    assert append(None) == INV
    for name in ("cache_len", "K", "V", "K8", "Ks", "V8", "Vs"):
        assert append(d, **{name: None}) == INV, name
    for name in ("K", "V", "K8", "V8"):
        assert append(d, **{name: ODD}) == INV, name
    assert append(d, n=0) == INV
    assert append(d, n=1025) == INV
    st = lambda *v: (ctypes.c_int64 * 3)(*v)  # noqa: E731
    assert append(d, ks=st(4096, 2048, 132)) == INV   # rows off a 16-byte boundary
    assert append(d, vs=st(4096, -2048, 128)) == INV


def test_decode_refusals():
    d = dims()
    assert decode(None) == INV
    for name in ("cache_len", "q", "K8", "Ks", "V8", "Vs", "o", "lse"):
        assert decode(d, **{name: None}) == INV, name
    for name in ("q", "K8", "V8", "o", "Kbar"):
        assert decode(d, **{name: ODD}) == INV, name
    assert decode(dims(k=3), idx=None) == INV
    assert decode(dims(k=3), Kbar=None) == INV
    assert decode(d, win=P, wout=None) == INV
    assert decode(dims(H=66, Hkv=2)) == UNS            # 33 query heads per key/value head
    need = L.ssa_workspace_size(d, L.SSA_OP_CACHE_DECODE)
    assert need > 0
    assert decode(d, ws_bytes=need - 1) == WS
    assert decode(d, ws=None) == WS
    assert decode(d, ws=ODD, ws_bytes=need) == WS
    # workspace: the blocks' maxima and sums per query head and attended block
    assert L.ssa_workspace_size(dims(T=65536), L.SSA_OP_CACHE_DECODE) - need >= 2 * 8 * (1024 - 16) * 8
    assert L.ssa_workspace_size(dims(T=65536, k=4), L.SSA_OP_CACHE_DECODE) < need


def test_evict_refusals():
    d = dims()
    assert evict(None) == INV
    for name in ("cache_len", "win", "K8", "Ks", "V8", "Vs", "kept"):
        assert evict(d, **{name: None}) == INV, name
    for name in ("K8", "V8", "Kbar"):
        assert evict(d, **{name: ODD}) == INV, name
    for bad in (dict(keep=0), dict(keep=17), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=2), dict(sink=5),
                dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert evict(d, **bad) == INV, bad
    need = L.ssa_workspace_size(d, L.SSA_OP_CACHE_EVICT)
    assert need >= 2 * 2 * 16 * 4
    assert evict(d, ws_bytes=need - 1) == WS
    assert evict(d, ws=None) == WS


def test_rope_axes_refusals():
    def call(d, pos=P, sections=(16, 24, 24), flags=0, base=1e4, factor=1.0, Q=P, qs=None, Qr=P, qrs=None, K=P, ks=None,
             Kr=P, krs=None, axes=None):
        n = len(sections)
        return L.load().ssa_rope_axes(ref(d), pos, n if axes is None else axes, (ctypes.c_int32 * max(n, 1))(*sections),
                                      flags, base, factor, Q, qs, Qr, qrs, K, ks, Kr, krs, None)

    st = lambda *v: (ctypes.c_int64 * 3)(*v)  # noqa: E731
    d = dims(T=5)  # any length
    assert call(None) == INV
    for over in (dict(B=0), dict(T=0), dict(H=0), dict(Hkv=-2), dict(dtype=3)):
        assert call(dims(**over)) == INV, over
    assert call(dims(d=96), sections=(16, 16, 16)) == UNS
    for bad in (dict(pos=None), dict(Q=None), dict(Qr=None), dict(Kr=None), dict(Q=None, Qr=None, K=None, Kr=None),
                dict(sections=(16, 24, 23)), dict(sections=(64, 0)), dict(sections=(65, -1)), dict(axes=0),
                dict(sections=(12, 13, 13, 13, 13)), dict(flags=8), dict(base=1.0), dict(base=float("inf")),
                dict(factor=0.0), dict(factor=float("nan")), dict(Q=ODD), dict(Kr=ODD)):
        assert call(d, **bad) == INV, bad
    assert call(d, qs=st(5120, 640, 132)) == INV       # rows off a 16-byte boundary
    assert call(d, qs=st(5120, 640, -128)) == INV
    assert call(d, qrs=st(5120, 640, 0)) == INV        # output rows on top of one another
    assert call(d, qs=st(5120, 128, 1024)) == INV      # in place with other strides
    far = ctypes.c_void_p(1 << 20)
    assert call(d, Qr=far, qrs=st(5120, 128, 128)) == INV       # rows of two heads on top of each other
    assert call(d, Qr=far, qrs=st(5120 - 128, 640, 128)) == INV  # the last row of a sequence and the next one's first
    assert call(d, Qr=far, qrs=st(640, 128, 1024)) == INV


def test_plain_forms():
    # every code is its own nearest value, halfway points go to the even code
    finite = [c for c in range(256) if c & 0x7F != 0x7F]
    assert np.array_equal(R.encode(R.CODES[finite]), np.array(finite, dtype=np.uint8))
    mid = (R._FINITE[:-1] + R._FINITE[1:]) / 2
    assert np.all(R.encode(mid) % 2 == 0)
    assert R.encode(np.nan) == 0x7F
    for a in (448.0, 448.0 * 2.0 ** 20, 1e-30):
        s = R.smallest_scale(a)
        assert a / s <= 448.0 and (a / (s / 2) > 448.0)
    assert R.smallest_scale(0.0) == R.MIN_SCALE
    # one axis: the single-axis rotation of the definition; the transpose undoes it
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((1, 2, 3, 64)), np.array([[[0, 7, 100000]]])
    y = R.rope_axes(x, pos, [32], 1e4, 2.0)
    a = 7 * 1e4 ** (-2.0 * 5 / 64) / 2.0
    assert y[0, 1, 1, 5] == pytest.approx(x[0, 1, 1, 5] * np.cos(a) - x[0, 1, 1, 37] * np.sin(a), abs=1e-12)
    np.testing.assert_allclose(R.rope_axes(y, pos, [32], 1e4, 2.0, transpose=True), x, atol=1e-10)
