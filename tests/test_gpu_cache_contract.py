"""The 8-bit cache's calls where their contract is narrowest, against the 64-bit
definitions (cache_ref.py); the ordinary shapes are in test_gpu_cache.py, whose
bounds hold here too unless a tighter one is derived at the test."""
import numpy as np
import pytest

from block_top_sparse_b200 import _lib as L
from block_top_sparse_b200 import ops

from . import cache_ref as R
from .test_gpu_cache import D, check_append, check_decode, check_evict, filled, gen, i32, query, snapshot, unchanged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from block_top_sparse_b200 import build
    build.build()


@pytest.mark.parametrize("G", [1, 4, 8, 13, 32])
@pytest.mark.parametrize("s", [64, 128])
@pytest.mark.parametrize("place", ["one block", "next block", "next block, larger values"])
def test_decode_weights_hold_16_bits(s, G, place):
    """Two values that cancel but for 2^-10 of their weights: what is left shows the weights' rounding, which the
    output's own rounding hides elsewhere.

    Bound of the weights: four terms of 4 significant bits, each at most 2^-4 off what the ones before it left, so
    (2^-4)^4 = 2^-16 of the weight; below the last term's normal range half its step of 2^-9,
    2^-10 / (256 * 16^3) = 2^-30 of the unit that stands for 256 (at most the tile's largest weight times its largest
    value scale, 1 here, for each of the two keys).  Logits and exponentials in fp32 as in test_gpu_cache.py; the
    output is rounded to bf16 (2^-8).  With three terms (2^-12) one in 25 of these heads is out of bounds."""
    B, Hkv = 16, 4
    dims = L.make_dims(B, G * Hkv, 2 * s, D, s, 0, Hkv=Hkv)
    c = filled(dims, [2 * s - 1] * B, garbage=False)
    for t in (c.K8.view(torch.uint8), c.V8.view(torch.uint8)):
        t.zero_()
    for t in (c.Kscale, c.Vscale):
        t.fill_(1.0)
    at = 1 if place == "one block" else s
    if place == "next block, larger values":
        c.Vscale[:, :, 0] = 2.0 ** -8
    L_new = at + 1
    K, V = torch.zeros(B, Hkv, 2, D, device="cuda"), torch.zeros(B, Hkv, 2, D, device="cuda")
    K[..., 0], K[..., 1, 1] = -1.0, -2.0 ** -6
    V[..., 0, :], V[..., 1, :] = 1.0, -1.0
    c.K8[:, :, at:at + 2].copy_(K.to(torch.float8_e4m3fn))
    c.V8[:, :, at:at + 2].copy_(V.to(torch.float8_e4m3fn))
    q = torch.zeros(B, G * Hkv, D, device="cuda")
    q[..., 0] = (0.05 + 3.0 * torch.rand(B, G * Hkv, device="cuda", generator=gen(G))) / dims.scale
    q[..., 1] = 2.0 ** -4 / dims.scale                       # the second key's logit is 2^-10 lower
    q = q.bfloat16()
    o, _, _ = ops.cache_decode(dims, c, i32(*[L_new] * B), q)
    assert L.ssa_get_device_error() == L.SSA_OK
    tokens = np.arange(L_new + 1)
    K8, V8 = c.K8.view(torch.uint8).cpu().numpy(), c.V8.view(torch.uint8).cpu().numpy()
    Ks, Vs = c.Kscale.cpu().numpy(), c.Vscale.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            Kd, Vd = R.dequantise(K8[b, h], Ks[b, h], s), R.dequantise(V8[b, h], Vs[b, h], s)
            ro, _, p, size = R.attend(q[b, heads].double().cpu().numpy(), Kd, Vd, tokens, dims.scale)
            e = 2.0 ** -20 * (size + 1.0)[:, None]
            spread = p @ np.abs(Vd[tokens])
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -16 + 2 * e) * spread + 2 * 2.0 ** -30 * p.max(1, keepdims=True)
            off = np.abs(o[b, heads].double().cpu().numpy() - ro) / tol
            assert np.all(off <= 1.0), (b, h, np.max(off))


@pytest.mark.parametrize("n,news", [(1, None), (1, [1, 1, 0, 1]), (100, None), (100, [100, 100, 0, 37])])
@pytest.mark.parametrize("s", [64, 128])
def test_idle_rows_are_idle_in_every_call(s, n, news):
    """cache_len = -1 in a batch whose other rows work: one tensor of lengths serves append, decode and eviction; the
    idle row keeps its cache, weights and length, whatever n_new says of it, and is no error."""
    B, Hkv, T = 4, 2, 8 * s
    dims = L.make_dims(B, 4, T, D, s, 0, Hkv=Hkv)
    lens = [5 * s + 3, -1, -1, 4 * s - 1]
    c = filled(dims, [T - 1] * B, seed=n)
    cache_len = i32(*lens)
    K, V = (torch.randn(B, Hkv, n, D, device="cuda", generator=gen(n + i)).bfloat16() for i in range(2))
    n_new = None if news is None else i32(*news)
    added = [0 if x < 0 else n if news is None else m for x, m in zip(lens, news or [n] * B)]
    before = snapshot(c)
    ops.cache_append(dims, c, cache_len, K, V, n_new)
    assert L.ssa_get_device_error() == L.SSA_OK
    assert unchanged(c, before, slice(1, 3))
    check_append(dims, c, before, lens, added, K, V)

    q, w = query(B, 4), torch.rand(B, Hkv, 8, device="cuda", generator=gen(3))
    was = w.clone()
    out = ops.cache_decode(dims, c, cache_len, q, weight_in=w, weight_out=w)
    assert L.ssa_get_device_error() == L.SSA_OK
    check_decode(dims, c, lens, q, out, was, w)

    held = [x + m for x, m in zip(lens, added)]
    before, was = snapshot(c), w.clone()
    kept, new_len = ops.cache_evict(dims, c, i32(*held), 2, w, 1, 1, weight_out=w)
    assert L.ssa_get_device_error() == L.SSA_OK
    assert unchanged(c, before, slice(1, 3)) and torch.equal(w[1:3], was[1:3])
    assert new_len.tolist() == [2 * s + held[0] % s, -1, -1, 2 * s + held[3] % s]
    assert bool((kept[1:3] == -1).all()) and bool((kept[[0, 3]] >= 0).all())


def test_lengths_below_idle_are_errors():
    dims = L.make_dims(2, 2, 256, D, 64, 0)
    c = filled(dims, [255] * 2)
    before = snapshot(c)
    for n in (1, 5):
        K = torch.randn(2, 2, n, D, device="cuda", generator=gen(n)).bfloat16()
        for lens in ([-2, -1], [-1, -2 ** 31]):
            ops.cache_append(dims, c, i32(*lens), K, K)
            assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
        ops.cache_append(dims, c, i32(-1, -1), K, K, i32(0, n + 1))  # a count out of range stays one
        assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
    w = torch.rand(2, 2, 4, device="cuda", generator=gen(1))
    _, new_len = ops.cache_evict(dims, c, i32(-2, -1), 1, w)
    assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
    assert new_len.tolist() == [-2, -1] and unchanged(c, before)


def test_the_documented_loop_with_several_layers():
    """Three layers of a model share one tensor of lengths over a prompt, pieces, single tokens and idle rows, by the
    loop of Cache8's documentation as it is written; every call against the definitions."""
    from .test_cache_loop import documented_loop
    B, H, Hkv, s, T, keep, layers = 4, 4, 2, 64, 512, 3, 3
    dims = L.make_dims(B, H, T, D, s, 2, Hkv=Hkv)
    caches = [filled(dims, [-1] * B, seed=i) for i in range(layers)]   # nothing held: all garbage
    weights = [torch.zeros(B, Hkv, T // s, device="cuda") for _ in range(layers)]
    g, cache_len = gen(5), i32(0, 0, -1, 0)
    calls = []

    class Checked:
        rope_axes = staticmethod(ops.rope_axes)

        @staticmethod
        def cache_append(dims, c, cache_len, K, V, n_new):
            before = snapshot(c)
            ops.cache_append(dims, c, cache_len, K, V, n_new)
            check_append(dims, c, before, cache_len.tolist(), n_new.tolist(), K, V)

        @staticmethod
        def cache_decode(dims, c, last, q, weight_in, weight_out):
            was = weight_in.clone()
            out = ops.cache_decode(dims, c, last, q, weight_in, weight_out)
            check_decode(dims, c, last.tolist(), q, out, was, weight_out)
            return out

        @staticmethod
        def cache_evict(dims, c, cache_len, keep, weight, sink, recent, weight_out):
            before, was, lens = snapshot(c), weight.clone(), cache_len.tolist()
            kept, new_len = ops.cache_evict(dims, c, cache_len, keep, weight, sink, recent, weight_out)
            for b, n in enumerate(lens):
                if n < 0:
                    assert unchanged(c, before, slice(b, b + 1)) and int(new_len[b]) == -1
            live = [b for b, n in enumerate(lens) if n >= 0]
            if len(live) == len(lens):
                check_evict(dims, c, before, lens, keep, sink, recent, was, kept, new_len, weight_out)
            else:
                sub = lambda t: t[live].contiguous()  # noqa: E731
                check_evict(L.make_dims(len(live), H, T, D, s, 0, Hkv=Hkv),
                            ops.Cache8(*(sub(t.view(torch.uint8)).view(t.dtype) for t in c)), [sub(t) for t in before],
                            [lens[b] for b in live], keep, sink, recent, sub(was), kept[live], new_len[live], sub(weight_out))
            calls.append(lens)
            return kept, new_len

    loop = documented_loop()
    for step, news in enumerate([[300, 1, 0, 64], [40, 0, 0, 100], [1, 1, 0, 1], [7, 0, 0, 90], [1, 1, 0, 1], [1, 200, 1, 1]]):
        if step == 5:
            cache_len[2] = 0  # a sequence takes the idle row
        n = max(news)
        qkv = [torch.randn(B, n, H + 2 * Hkv, D, device="cuda", generator=g).bfloat16() for _ in range(layers)]
        project = lambda x, i: tuple(t.transpose(1, 2) for t in qkv[i].split([H, Hkv, Hkv], 2))  # noqa: E731
        env = dict(ops=Checked, torch=torch, dims=dims, dims_n=L.make_dims(B, H, n, D, s, 0, Hkv=Hkv), caches=caches,
                   pos=torch.randint(0, 5000, (3, B, n), device="cuda", dtype=torch.int32, generator=g),
                   sections=[16, 24, 24], layers=[lambda x, i=i: project(x, i) for i in range(layers)], x=None,
                   weights=weights, cache_len=cache_len, n_new=i32(*news), rows=torch.arange(B, device="cuda"),
                   keep=keep, sink=1, recent=1)
        exec(loop, env)
        lens = calls[-1]
        assert calls[-layers:] == [lens] * layers
        assert cache_len.tolist() == [n if n < 0 else min(n // s, keep) * s + n % s for n in lens]
        assert L.ssa_get_device_error() == L.SSA_OK
    assert max(map(max, calls)) > (keep + 1) * s and cache_len.tolist()[2] == 1  # blocks did leave


@pytest.mark.parametrize("n", [1, 3])
def test_append_keeps_the_sign_of_zero_beside_an_infinity(n):
    """The code of -0 is 0x80 whatever stands beside it, in the single-token form as in the other."""
    dims = L.make_dims(1, 2, 128, D, 64, 0)
    K = torch.zeros(1, 2, n, D, dtype=torch.bfloat16, device="cuda")
    K[..., 1::2] = -0.0
    K[0, 0, 0, 0], K[0, 0, 0, 2], K[0, 0, 0, 3] = float("inf"), float("-inf"), float("nan")
    for at in (0, 63):
        c = filled(dims, [at - 1])
        before = snapshot(c)
        ops.cache_append(dims, c, i32(at), K, K)
        assert L.ssa_get_device_error() == L.SSA_OK
        check_append(dims, c, before, [at], [n], K, K)


def test_rows_off_a_16_byte_boundary_are_refused():
    """Views of the right shape whose strides fit but whose base does not: the library refuses them, by its status."""
    dims = L.make_dims(1, 4, 256, D, 64, 0)
    c = filled(dims, [9])
    before = snapshot(c)
    wide = torch.zeros(1, 4, 30, D + 8, dtype=torch.bfloat16, device="cuda")
    odd, even = wide[..., 1:1 + D], wide[..., 8:]
    assert odd.shape == even.shape and odd.stride() == even.stride() and odd.data_ptr() % 16 == 2
    for K, V in ((odd, even), (even, odd)):
        with pytest.raises(L.SSAError):
            ops.cache_append(dims, c, i32(10), K, V)
    assert unchanged(c, before)
    rope = L.make_dims(1, 4, 30, D, 64, 0)
    pos = torch.zeros(1, 1, 30, dtype=torch.int32, device="cuda")
    for args in ((odd,), (even, odd)):
        with pytest.raises(L.SSAError):
            ops.rope_axes(rope, pos, [64], *args)
    with pytest.raises(L.SSAError):
        ops.rope_axes(rope, pos, [64], even, out=(odd, None))
    ops.cache_append(dims, c, i32(10), even, even)      # the same view on its boundary is taken
    assert torch.equal(ops.rope_axes(rope, pos, [64], even)[0], even)
    assert L.ssa_get_device_error() == L.SSA_OK
