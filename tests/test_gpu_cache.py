"""The 8-bit key/value cache (ssa_cache_append, ssa_cache_decode, ssa_cache_evict)
against its 64-bit definitions (cache_ref.py).

Bounds.  Codes, scales, selections and moved data are equal.  A pooled key is an
fp32 sum of s codes: 32 * 2^-24 of the mean magnitude.  A logit is a sum of 2 d
exact products in fp32 of a query in two terms: 2^-20 of the sum of magnitudes it
is made of, and its exponential carries that as a relative error, as do the
weights and, in absolute terms, lse.  The output's weights are further cut to
three terms of 4 significant bits and it is rounded to bf16 (2^-8 of its value).
A rounding to 4 significant bits is off by at most 2^-4 of the value, and each term
holds what the ones before it left: (2^-4)^3 = 2^-12 of the weight; where the third
term is below 2^-6, half its step of 2^-9 counts, 2^-10 / (256 * 256) = 2^-26 of the
unit that stands for 256.  That is the largest weight of the key's tile of 128 keys
(one block of 128, two of 64) times the tile's larger value scale, at most 2^6 times
the key's own (2^-20 of the value), or else the tile's largest product of weight and
value scale (2^-26 of it times the key's code)."""
import numpy as np
import pytest

from block_top_sparse_b200 import _lib as L
from block_top_sparse_b200 import ops

from . import cache_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _build():
    from block_top_sparse_b200 import build
    build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes_np(t):
    return t.view(torch.uint8).cpu().numpy()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(dims, lens, seed=0, garbage=True):
    """A cache of lens[b] + 1 tokens per sequence whose blocks differ in size; everything behind them is garbage:
    NaN codes and scales, huge pooled keys."""
    B, Hk, T, s, nb = dims.B, dims.kv_heads, dims.T, dims.s, dims.T // dims.s
    g = gen(seed)
    c = ops.Cache8.empty(dims)
    for codes, scale in ((c.K8, c.Kscale), (c.V8, c.Vscale)):
        x = torch.randn(B, Hk, nb, s, D, device="cuda", generator=g)
        x *= torch.exp2(torch.randint(-3, 3, (B, Hk, nb, 1, 1), device="cuda", generator=g).float())
        m, e = torch.frexp(x.abs().amax((-1, -2)))
        sc = torch.ldexp(torch.ones_like(m), torch.where(m > 0.875, e - 8, e - 9))
        codes.copy_((x / sc[..., None, None]).to(torch.float8_e4m3fn).view(B, Hk, T, D))
        scale.copy_(sc)
    c.Kbar.copy_((c.K8.float().view(B, Hk, nb, s, D) * c.Kscale[..., None, None]).mean(3))
    if garbage:
        for b, n in enumerate(lens):
            n = max(int(n), -1) + 1
            for codes, scale in ((c.K8, c.Kscale), (c.V8, c.Vscale)):
                codes.view(torch.uint8)[b, :, n:] = 0x7F
                scale[b, :, -(-n // s):] = float("nan")
            c.Kbar[b, :, n // s:] = 3e38
    return c


def snapshot(c):
    return [t.clone() for t in (c.K8.view(torch.uint8), c.Kscale, c.V8.view(torch.uint8), c.Vscale, c.Kbar)]


def unchanged(c, before, where=slice(None)):
    now = (c.K8.view(torch.uint8), c.Kscale, c.V8.view(torch.uint8), c.Vscale, c.Kbar)
    return all(torch.equal(a[where].view(torch.uint8), b[where].view(torch.uint8)) for a, b in zip(now, before))


# ------------------------------------------------------------------------------------------ append
def check_append(dims, c, before, lens, news, K, V):
    s, nb = dims.s, dims.T // dims.s
    Kbar = before[4].cpu().numpy()
    for keys, codes, scale, was, was_scale, X in ((True, c.K8, c.Kscale, before[0], before[1], K),
                                                  (False, c.V8, c.Vscale, before[2], before[3], V)):
        want, want_scale = was.cpu().numpy().copy(), was_scale.double().cpu().numpy().copy()
        x = X.double().cpu().numpy()
        for b in range(dims.B):
            for h in range(dims.kv_heads):
                done = R.append(x[b, h, :news[b]], want[b, h], want_scale[b, h], lens[b], s)
                if keys:
                    for j in done:
                        rows = R.CODES[want[b, h, j * s:(j + 1) * s]] * want_scale[b, h, j]
                        got = c.Kbar[b, h, j].double().cpu().numpy()
                        np.testing.assert_array_less(np.abs(got - rows.mean(0)), 32 * 2.0 ** -24 * np.abs(rows).mean(0) + 1e-300)
                        Kbar[b, h, j] = c.Kbar[b, h, j].cpu().numpy()
        got = codes_np(codes)
        nan = (got & 0x7F == 0x7F) & (want & 0x7F == 0x7F)
        assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want))
        np.testing.assert_array_equal(scale.double().cpu().numpy(), want_scale)
    np.testing.assert_array_equal(c.Kbar.cpu().numpy(), Kbar)  # rows of no completed block are as they were


@pytest.mark.parametrize("s,T,n,lens,news", [
    (64, 256, 1, [0, 63, 64, 255, 130], None),                 # first token, one that completes a block, the last row
    (128, 512, 1, [0, 127, 128, 511, 300], None),
    (64, 512, 200, [0, 1, 63, 64, 312], None),                 # across blocks, up to the end of the cache
    (128, 1024, 300, [0, 5, 127, 640, 724], [300, 0, 1, 128, 123]),   # ragged, none at all
    (128, 256, 256, [0, 0, 0, 0, 0], None)])
@pytest.mark.parametrize("rows", ["heads", "tokens"])
def test_append_matches_the_definition(s, T, n, lens, news, rows):
    B, Hk = len(lens), 3
    dims = L.make_dims(B, Hk, T, D, s, 0)
    g = gen(s + n)
    c = filled(dims, [x - 1 for x in lens], seed=n, garbage=True)
    if rows == "tokens":
        K, V = (torch.randn(B, n, Hk, D, device="cuda", generator=g).bfloat16().transpose(1, 2) for _ in range(2))
    else:
        K, V = (torch.randn(B, Hk, n, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    K[:, 0] *= 30.0     # the open block's scale grows
    V[:, 1] *= 1e-3     # and stays
    if news is not None:  # rows that are not read
        for b, m in enumerate(news):
            K[b, :, m:] = float("nan")
            V[b, :, m:] = float("inf")
    before = snapshot(c)
    ops.cache_append(dims, c, i32(*lens), K, V, None if news is None else i32(*news))
    assert L.ssa_get_device_error() == L.SSA_OK
    check_append(dims, c, before, lens, news or [n] * B, K, V)


def test_append_special_values():
    s, T = 64, 128
    dims = L.make_dims(1, 4, T, D, s, 0)
    c = filled(dims, [-1])
    x = torch.randn(1, 4, 100, D, device="cuda", generator=gen(1)).bfloat16()
    x[0, 0] = 0.0                                    # nothing but zeros: the smallest scale
    x[0, 1, 3, 5] = float("inf")
    x[0, 1, 70, 6] = float("-inf")
    x[0, 1, 4, 7] = float("nan")
    x[0, 2] = x[0, 2] * 2.0 ** -130                  # subnormal in bf16
    x[0, 3, 0, 0] = torch.finfo(torch.bfloat16).max
    before = snapshot(c)
    ops.cache_append(dims, c, i32(0), x, x)
    check_append(dims, c, before, [0], [100], x, x)
    assert float(c.Kscale[0, 0, 0]) == R.MIN_SCALE


def test_append_token_by_token_is_the_definition_of_every_step():
    s, T = 64, 192
    dims = L.make_dims(2, 2, T, D, s, 0)
    c = filled(dims, [-1, 29])
    x = (torch.randn(2, 2, 140, D, device="cuda", generator=gen(2)) * torch.exp(
        torch.randn(2, 2, 140, 1, device="cuda", generator=gen(3)))).bfloat16()
    for t in range(140):
        before = snapshot(c)
        K = x[:, :, t:t + 1]
        ops.cache_append(dims, c, i32(t, 30 + t), K, -K)
        if t % 9 == 0 or (t + 1) % s == 0 or (t + 31) % s == 0:
            check_append(dims, c, before, [t, 30 + t], [1, 1], K, -K)


def test_append_refuses_a_sequence_and_writes_the_others():
    dims = L.make_dims(5, 2, 256, D, 64, 0)
    c = filled(dims, [9] * 5)
    K = torch.randn(5, 2, 4, D, device="cuda", generator=gen(4)).bfloat16()
    for lens, news in (([10, -1, 253, 10, 10], [4, 1, 4, 5, -1]),):
        before = snapshot(c)
        ops.cache_append(dims, c, i32(*lens), K, K, i32(*news))
        assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
        assert L.ssa_get_device_error() == L.SSA_OK
        assert unchanged(c, before, slice(1, 5))
        check_append(dims, c, before, lens, [4, 0, 0, 0, 0], K, K)


# ------------------------------------------------------------------------------------------ decode
def check_decode(dims, c, lens, q, out, weight_in=None, weight_out=None, rows=None):
    """rows: (sequence, key head) pairs to check; default: all."""
    o, lse, idx = out
    s, k, G, nb = dims.s, dims.k, dims.H // dims.kv_heads, dims.T // dims.s
    K8, V8, Ks, Vs = codes_np(c.K8), codes_np(c.V8), c.Kscale.cpu().numpy(), c.Vscale.cpu().numpy()
    qn, Kbar = q.double().cpu().numpy(), c.Kbar.double().cpu().numpy()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, h in rows or [(b, h) for b in range(dims.B) for h in range(dims.kv_heads)]:
        Lb, heads = int(lens[b]), slice(h * G, (h + 1) * G)
        win = np.zeros(nb) if weight_in is None else weight_in[b, h].double().cpu().numpy()
        if Lb < 0:
            assert np.all(o[b, heads] == 0) and np.all(lse[b, heads] == -np.inf)
            assert k == 0 or np.all(idx[b, h].cpu().numpy() == -1)
            if weight_out is not None:
                np.testing.assert_array_equal(weight_out[b, h].double().cpu().numpy(), win)
            continue
        bt = Lb // s
        if k:
            want = R.select(qn[b, heads], Kbar[b, h], bt, k)
            assert idx[b, h].tolist() == want
            blocks = [j for j in want if j >= 0]
        else:
            blocks = list(range(bt + 1))
        tokens = np.concatenate([np.arange(j * s, min((j + 1) * s, Lb + 1)) for j in blocks])
        Kd, Vd = R.dequantise(K8[b, h, :Lb + 1], Ks[b, h], s), R.dequantise(V8[b, h, :Lb + 1], Vs[b, h], s)
        ro, rl, p, size = R.attend(qn[b, heads], Kd, Vd, tokens, dims.scale)
        e = 2.0 ** -20 * (size + 1.0)[:, None]
        spread = p @ np.abs(Vd[tokens])
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -12 + 2 * e) * spread
        slots = np.concatenate([np.full(min((j + 1) * s, Lb + 1) - j * s, i) for i, j in enumerate(blocks)])
        vs = Vs[b, h].astype(np.float64)[tokens // s]
        for tile in range(slots[-1] // (128 // s) + 1):
            u = np.flatnonzero(slots // (128 // s) == tile)
            V = np.abs(Vd[tokens[u]])
            tol += np.maximum(2.0 ** -20 * p[:, u].max(1, keepdims=True) * V.sum(0),
                              2.0 ** -26 * (p[:, u] * vs[u]).max(1, keepdims=True) * (V / vs[u][:, None]).sum(0))
        assert np.all(np.abs(o[b, heads] - ro) <= tol), (b, h, np.max(np.abs(o[b, heads] - ro) / tol))
        assert np.all(np.abs(lse[b, heads] - rl) <= e[:, 0] + 2.0 ** -22 * np.abs(rl))
        if weight_out is not None:
            add = np.zeros(nb)
            slack = np.zeros(nb)
            for j in blocks:
                m = (tokens >= j * s) & (tokens < (j + 1) * s)
                add[j] = p[:, m].sum()
                slack[j] = (2 * e[:, 0] * p[:, m].sum(1)).sum()
            got = weight_out[b, h].double().cpu().numpy()
            # (weights below 2^-126, the smallest normal fp32, count as 0: at most so much for each of s keys and G heads)
            assert np.all(np.abs(got - (win + add)) <= slack + 2.0 ** -22 * (win + add) + s * G * 2.0 ** -126)


def query(B, H, seed=7, size=2.0):
    return (size * torch.randn(B, H, D, device="cuda", generator=gen(seed))).bfloat16()


def lens_of(s, T):
    return [-1, 0, 1, s - 2, s - 1, s, 5 * s + 17, T - 2, T - 1]


@pytest.mark.parametrize("s", [64, 128])
@pytest.mark.parametrize("H,Hkv,k", [(2, 2, 0), (2, 2, 3), (4, 2, 5), (5, 1, 0), (16, 2, 1), (12, 1, 4), (16, 1, 0),
                                     (34, 2, 0), (32, 1, 2), (3, 3, 16)])
def test_decode_matches_the_definition(H, Hkv, s, k):
    T = 16 * s
    lens = lens_of(s, T)
    B = len(lens)
    dims = L.make_dims(B, H, T, D, s, k, Hkv=Hkv)
    c = filled(dims, lens, seed=H)
    q = query(B, H)
    before = snapshot(c)
    w_in = torch.rand(B, Hkv, T // s, device="cuda", generator=gen(8))
    w_out = torch.empty_like(w_in)
    out = ops.cache_decode(dims, c, i32(*lens), q, weight_in=w_in, weight_out=w_out)
    assert L.ssa_get_device_error() == L.SSA_OK
    check_decode(dims, c, lens, q, out, w_in, w_out)
    assert unchanged(c, before)
    # without weights, with a fresh sum, and added in place: the same values
    again = ops.cache_decode(dims, c, i32(*lens), q)
    assert torch.equal(again[0], out[0]) and torch.equal(again[1], out[1])
    fresh = torch.empty_like(w_in)
    ops.cache_decode(dims, c, i32(*lens), q, weight_out=fresh)
    check_decode(dims, c, lens, q, out, None, fresh)
    ops.cache_decode(dims, c, i32(*lens), q, weight_in=w_in, weight_out=w_in)
    assert torch.equal(w_in, w_out)


@pytest.mark.parametrize("B,H,Hkv,T,s,k", [(1, 4, 1, 131072, 128, 0), (1, 2, 2, 131072, 64, 40), (37, 8, 4, 2048, 64, 0),
                                           (150, 2, 1, 1024, 128, 3), (700, 1, 1, 256, 64, 0), (1, 1, 1, 524288, 64, 300)])
def test_decode_shares_of_work(B, H, Hkv, T, s, k):
    """Long caches split over many CTAs, and many short ones of which a CTA takes several."""
    rng = np.random.default_rng(T)
    lens = rng.integers(-1, T, B) if B > 1 else np.array([T - 77])
    dims = L.make_dims(B, H, T, D, s, k, Hkv=Hkv)
    c = filled(dims, lens, seed=5)
    q = query(B, H, 9)
    w = torch.empty(B, Hkv, T // s, device="cuda")
    out = ops.cache_decode(dims, c, i32(*lens.tolist()), q, weight_out=w)
    assert L.ssa_get_device_error() == L.SSA_OK
    rows = [(int(b), int(rng.integers(Hkv))) for b in rng.choice(B, min(B, 40), replace=False)]
    check_decode(dims, c, lens, q, out, None, w, rows)
    w2 = torch.empty_like(w)
    again = ops.cache_decode(dims, c, i32(*lens.tolist()), q, weight_out=w2)   # bit for bit
    assert all(torch.equal(a, b) for a, b in zip(out, again) if a is not None) and torch.equal(w, w2)


def test_decode_with_every_block_selected_is_the_full_attention():
    s, T, lens = 64, 1024, [1000, 63, 500]
    d0, dk = L.make_dims(3, 8, T, D, s, 0, Hkv=2), L.make_dims(3, 8, T, D, s, T // s, Hkv=2)
    c = filled(d0, lens)
    q = query(3, 8)
    a, b = ops.cache_decode(d0, c, i32(*lens), q), ops.cache_decode(dk, c, i32(*lens), q)
    check_decode(dk, c, lens, q, b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_ties_go_to_the_lower_block():
    s, T = 64, 64 * 40
    dims = L.make_dims(1, 2, T, D, s, 6, Hkv=1)
    c = filled(dims, [T - 1])
    c.Kbar[:] = c.Kbar[:, :, 3:4]
    c.Kbar[:, :, 20] = 0.0
    q = query(1, 2)
    _, _, idx = ops.cache_decode(dims, c, i32(T - 1), q)
    assert idx[0, 0].tolist() == R.select(q[0].double().cpu().numpy(), c.Kbar[0, 0].double().cpu().numpy(), 39, 6)
    c.Kbar.zero_()
    c.Kbar[:, :, 1::2] = -0.0
    _, _, idx = ops.cache_decode(dims, c, i32(T - 1), q)
    assert idx[0, 0].tolist() == [0, 1, 2, 3, 4, 39]


def test_decode_extreme_values():
    """Blocks whose scales lie 2^60 apart in one tile, logits of thousands, queries with elements far apart, NaN."""
    s, T = 64, 512
    lens = [T - 1] * 4
    dims = L.make_dims(4, 4, T, D, s, 0, Hkv=2)
    c = filled(dims, lens)
    c.Vscale[0, :, ::2] *= 2.0 ** -60
    q = query(4, 4)
    q[1] *= 64.0
    q[2, :, 0] *= 2.0 ** 12
    q[3, 2, 5] = float("nan")
    c.K8.view(torch.uint8)[3, 0, 100, 7] = 0x7F
    out = ops.cache_decode(dims, c, i32(*lens), q)
    check_decode(dims, c, lens, q, out, rows=[(b, h) for b in range(3) for h in range(2)])
    o, lse, _ = out
    assert bool(o[3, :3].isnan().all()) and bool(lse[3, :3].isnan().all())  # the head with the NaN key, the NaN query
    assert bool(o[3, 3].isfinite().all()) and bool(lse[3, 3].isfinite())    # its neighbour is untouched


@pytest.mark.parametrize("G", [2, 8, 13, 32])
@pytest.mark.parametrize("s", [64, 128])
def test_decode_value_scales_far_apart(s, G):
    """Value scales from 2^-40 to 2^40 from block to block, and logits up to tens apart: the blocks that carry the
    weight and those that carry the output are others, and both keep their precision."""
    T = 16 * s
    lens = [T - 1, 9 * s + 5, 3 * s - 1, 2 * s]
    dims = L.make_dims(4, 4 * G, T, D, s, 0, Hkv=4)
    c = filled(dims, lens, seed=3)
    c.Vscale.mul_(torch.exp2(torch.randint(-40, 41, c.Vscale.shape, device="cuda", generator=gen(4)).float()))
    for size in (0.5, 2.0, 12.0):
        q = query(4, 4 * G, 5, size)
        w = torch.empty(4, 4, T // s, device="cuda")
        out = ops.cache_decode(dims, c, i32(*lens), q, weight_out=w)
        check_decode(dims, c, lens, q, out, None, w)
    # one block's values vanish beside the other's in the same tile, and it has all the weight
    c.Vscale[:, :, 1::2] = c.Vscale[:, :, ::2] * 2.0 ** 30
    q = query(4, 4 * G, 6, 1.0)
    K8 = torch.zeros(4, 4, T, D, device="cuda")
    K8[:, :, (torch.arange(T, device="cuda") // s) % 2 == 0] = torch.sign(q.float().view(4, 4, G, D).sum(2))[:, :, None]
    c.K8.copy_(K8.to(torch.float8_e4m3fn))
    c.Kscale.fill_(4.0)
    out = ops.cache_decode(dims, c, i32(*lens), q)
    check_decode(dims, c, lens, q, out)


def test_decode_reports_bad_lengths():
    dims = L.make_dims(4, 2, 256, D, 64, 2)
    lens = [255, 256, -2, 10]
    c = filled(dims, [255, -1, -1, 10])
    q = query(4, 2)
    w = torch.rand(4, 2, 4, device="cuda")
    w0 = w.clone()
    out = ops.cache_decode(dims, c, i32(*lens), q, weight_in=w, weight_out=w)
    assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
    assert L.ssa_get_device_error() == L.SSA_OK
    check_decode(dims, c, [255, -1, -1, 10], q, out, w0, w)


def test_decode_workspace_contents_do_not_matter():
    dims = L.make_dims(3, 8, 1024, D, 64, 4, Hkv=2)
    lens = [1023, 70, 300]
    c = filled(dims, lens)
    q = query(3, 8)
    n = L.ssa_workspace_size(dims, L.SSA_OP_CACHE_DECODE)
    outs = []
    for fill in (0, 255):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        w = torch.empty(3, 2, 16, device="cuda")
        outs.append(ops.cache_decode(dims, c, i32(*lens), q, weight_out=w, ws=ws[:n]) + (w,))
        assert bool((ws[n:] == fill).all())
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_decode_captured_graphs_and_streams():
    """Two graphs that share a workspace, replayed in turn with other lengths; and a call on another stream."""
    dims = L.make_dims(4, 8, 1024, D, 128, 0, Hkv=2)
    dk = L.make_dims(4, 8, 1024, D, 128, 3, Hkv=2)
    lens = i32(5, 1000, 640, -1)
    c = filled(dims, [1023] * 4, garbage=False)
    q = query(4, 8)
    n = max(L.ssa_workspace_size(x, L.SSA_OP_CACHE_DECODE) for x in (dims, dk))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    w = torch.zeros(4, 2, 8, device="cuda")
    ops.cache_decode(dims, c, lens, q, ws=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (dims, dk):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.cache_decode(x, c, lens, q, weight_in=w, weight_out=w, ws=ws))
        graphs.append(g)
    for new in ([7, 1023, 0, 300], [1023, -1, 127, 128]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for x, g, out in zip((dims, dk), graphs, outs):
            was = w.clone()
            g.replay()
            torch.cuda.synchronize()
            check_decode(x, c, new, q, out, was, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = ops.cache_decode(dims, c, lens, q)
    s.synchronize()
    check_decode(dims, c, [1023, -1, 127, 128], q, out)
    assert L.ssa_get_device_error() == L.SSA_OK


# ------------------------------------------------------------------------------------------ evict
def check_evict(dims, c, before, lens, keep, sink, recent, weight, kept, new_len, weight_out):
    s, nb = dims.s, dims.T // dims.s
    now = (c.K8.view(torch.uint8), c.Kscale, c.V8.view(torch.uint8), c.Vscale, c.Kbar)
    for b, n in enumerate(lens):
        whole = n // s
        assert int(new_len[b]) == min(whole, keep) * s + n % s
        for h in range(dims.kv_heads):
            want = R.evict_order(weight[b, h].tolist(), whole, keep, sink, recent)
            assert kept[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
            places = want + ([whole] if n % s else [])
            src = list(range(nb))
            src[:len(places)] = places                 # blocks behind stay what they were
            for t, was in zip(now, before):
                a, e = t[b, h].reshape(nb, -1), was[b, h].reshape(nb, -1)[src]
                assert torch.equal(a.view(torch.uint8), e.view(torch.uint8)), (b, h)
            if weight_out is not None:
                e = torch.zeros(nb)
                e[:len(places)] = weight[b, h].cpu()[places]
                assert torch.equal(weight_out[b, h].cpu().view(torch.int32), e.view(torch.int32))


@pytest.mark.parametrize("s,nb,keep,sink,recent", [(64, 17, 16, 1, 2), (64, 12, 1, 0, 0), (128, 9, 4, 2, 2), (64, 40, 7, 0, 3),
                                                   (128, 6, 6, 1, 1), (64, 300, 150, 4, 20), (64, 1, 1, 0, 0),
                                                   (64, 1100, 777, 1, 0)])
def test_evict_matches_the_definition(s, nb, keep, sink, recent):
    T = nb * s
    lens = [T, T - 1, 0, 1, min(T, keep * s), min(T, keep * s + 1), min(T, (keep + 1) * s), T // 2]
    B, Hk = len(lens), 2
    dims = L.make_dims(B, Hk, T, D, s, 0)
    c = filled(dims, [n - 1 for n in lens], seed=nb)
    weight = torch.rand(B, Hk, nb, device="cuda", generator=gen(nb))
    weight[:, 1] = torch.randint(0, 3, (B, nb), device="cuda", generator=gen(1)).float()   # many ties
    before, w0 = snapshot(c), weight.clone()
    w_out = torch.full_like(weight, -5.0)
    kept, new_len = ops.cache_evict(dims, c, i32(*lens), keep, weight, sink, recent, weight_out=w_out)
    assert L.ssa_get_device_error() == L.SSA_OK
    check_evict(dims, c, before, lens, keep, sink, recent, w0, kept, new_len, w_out)
    assert torch.equal(weight, w0)


def test_evict_special_weights_in_place():
    s, nb, keep = 64, 20, 8
    dims = L.make_dims(2, 2, nb * s, D, s, 0)
    lens = [nb * s - 3, 10 * s]
    c = filled(dims, [n - 1 for n in lens])
    weight = torch.randn(2, 2, nb, device="cuda", generator=gen(3))
    weight[0, 0, ::3] = float("nan")
    weight[0, 0, 1::3] = float("-inf")
    weight[0, 1, ::2] = float("inf")
    weight[0, 1, 1::2] = -0.0
    weight[1, 0] = float("nan")
    weight[1, 1] = 0.0
    weight[1, 1, ::2] = -0.0
    before, w0 = snapshot(c), weight.clone()
    cache_len = i32(*lens)
    kept, new_len = ops.cache_evict(dims, c, cache_len, keep, weight, weight_out=weight, new_len=cache_len)
    assert new_len is cache_len
    check_evict(dims, c, before, lens, keep, 0, 0, w0, kept, new_len, weight)


def test_evict_leaves_a_sequence_with_a_bad_length():
    dims = L.make_dims(3, 2, 640, D, 64, 0)
    c = filled(dims, [639] * 3)
    weight = torch.rand(3, 2, 10, device="cuda")
    before, w0 = snapshot(c), weight.clone()
    w_out = torch.empty_like(weight)
    kept, new_len = ops.cache_evict(dims, c, i32(-4, 641, 640), 3, weight, weight_out=w_out)
    assert L.ssa_get_device_error() == L.SSA_ERR_BAD_INPUT
    assert L.ssa_get_device_error() == L.SSA_OK
    assert unchanged(c, before, slice(0, 2)) and new_len.tolist() == [-4, 641, 192]
    assert bool((kept[:2] == -1).all()) and torch.equal(w_out[:2], w0[:2])


def test_evict_largest_number_of_blocks_and_no_pooled_keys():
    s, nb, keep = 64, 8192, 5000
    dims = L.make_dims(1, 1, nb * s, D, s, 0)
    c = filled(dims, [nb * s - 1], garbage=False)
    weight = torch.rand(1, 1, nb, device="cuda", generator=gen(6))
    before, w0 = snapshot(c), weight.clone()
    kept, new_len = ops.cache_evict(dims, ops.Cache8(*c[:4]), i32(nb * s), keep, weight, 1, 100)
    want = R.evict_order(w0[0, 0].tolist(), nb, keep, 1, 100)
    assert kept[0, 0].tolist() == want
    src = torch.tensor(want + list(range(keep, nb)), device="cuda")
    assert torch.equal(c.K8.view(torch.uint8).view(nb, -1), before[0].view(nb, -1)[src])
    assert torch.equal(c.Vscale.view(nb), before[3].view(nb)[src])
    assert torch.equal(c.Kbar, before[4])


def test_evict_captured():
    dims = L.make_dims(2, 2, 1024, D, 64, 0)
    lens = i32(1024, 700)
    c = filled(dims, [1023, 699])
    weight = torch.rand(2, 2, 16, device="cuda", generator=gen(2))
    ws = torch.empty(L.ssa_workspace_size(dims, L.SSA_OP_CACHE_EVICT), dtype=torch.uint8, device="cuda")
    w_out, new_len = torch.empty_like(weight), torch.empty_like(lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, _ = ops.cache_evict(dims, c, lens, 5, weight, 1, 1, weight_out=w_out, new_len=new_len, ws=ws)
    for seed in (1, 2):
        weight.copy_(torch.rand(2, 2, 16, device="cuda", generator=gen(seed)))
        before = snapshot(c)
        g.replay()
        torch.cuda.synchronize()
        check_evict(dims, c, before, [1024, 700], 5, 1, 1, weight, kept, new_len, w_out)


# ------------------------------------------------------------------------------------------ together
def test_serving_loop():
    """Two layers' worth of what a model does: positions, append, decode with weights, eviction at the budget, a
    prompt first and single tokens after it; every call against the definitions, on the state that the one before left."""
    B, H, Hkv, s, T, keep = 3, 8, 2, 64, 512, 5
    dense, sparse = L.make_dims(B, H, T, D, s, 0, Hkv=Hkv), L.make_dims(B, H, T, D, s, 3, Hkv=Hkv)
    sections = [16, 24, 24]
    g = gen(11)
    c = ops.Cache8.empty(dense)
    for t in (c.K8.view(torch.uint8), c.V8.view(torch.uint8)):
        t.fill_(0x7F)
    for t in (c.Kscale, c.Vscale, c.Kbar):
        t.fill_(float("nan"))
    weight = torch.zeros(B, Hkv, T // s, device="cuda")
    cache_len = i32(0, 0, 0)
    where = i32(0, 0, 0)            # rotary position of the next token: goes on when blocks leave
    news = [350, 1, 129]
    for step in range(70):
        n = 350 if step == 0 else 1
        count = i32(*news) if step == 0 else torch.ones(B, dtype=torch.int32, device="cuda")
        pos = (where[None, :, None] + torch.arange(n, device="cuda", dtype=torch.int32)).expand(3, B, n).contiguous()
        dn = L.make_dims(B, H, n, D, s, 0, Hkv=Hkv)
        qkv = torch.randn(B, n, H + 2 * Hkv, D, device="cuda", generator=g).bfloat16()
        q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        q, k = ops.rope_axes(dn, pos, sections, q, k, base=10000.0)
        lens, before = cache_len.tolist(), snapshot(c)
        ops.cache_append(dense, c, cache_len, k, v, count)
        if step % 10 == 0:
            check_append(dense, c, before, lens, count.tolist(), k, v)
        last = (cache_len + count - 1).contiguous()       # the newest token attends
        qlast = q[torch.arange(B, device="cuda"), :, count.long() - 1].contiguous()
        dims = sparse if step % 2 else dense
        was = weight.clone()
        out = ops.cache_decode(dims, c, last, qlast, weight_in=weight, weight_out=weight)
        if step % 7 == 0 or step == 69:
            check_decode(dims, c, last.tolist(), qlast, out, was, weight)
        cache_len += count
        where += count
        if step % 6 == 5 or step == 0:
            before, was, lens = snapshot(c), weight.clone(), cache_len.tolist()
            kept, _ = ops.cache_evict(dense, c, cache_len, keep, weight, 1, 1, weight_out=weight, new_len=cache_len)
            check_evict(dense, c, before, lens, keep, 1, 1, was, kept, cache_len, weight)
    assert L.ssa_get_device_error() == L.SSA_OK
    assert int(cache_len.max()) <= (keep + 1) * s and where.tolist() == [419, 70, 198]


def test_tensor_checks():
    dims = L.make_dims(2, 4, 256, D, 64, 0, Hkv=2)
    c = filled(dims, [100, 100])
    q, lens, w = query(2, 4), i32(100, 100), torch.zeros(2, 2, 4, device="cuda")
    K = torch.zeros(2, 2, 1, D, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: ops.cache_decode(dims, c, lens.long(), q), lambda: ops.cache_decode(dims, c, lens[:1], q),
           lambda: ops.cache_decode(dims, c, lens, q.float()), lambda: ops.cache_decode(dims, c, lens, q[:, :2]),
           lambda: ops.cache_decode(dims, c, lens, q.cpu()), lambda: ops.cache_decode(dims, c, lens, q, weight_out=w[..., :2]),
           lambda: ops.cache_decode(dims, c._replace(V8=c.V8.float()), lens, q),
           lambda: ops.cache_decode(dims, c._replace(Kscale=c.Kscale.transpose(0, 1)), lens, q),
           lambda: ops.cache_append(dims, c, lens, K.float(), K), lambda: ops.cache_append(dims, c, lens, K, K[:, :1]),
           lambda: ops.cache_append(dims, c, lens, K, K, n_new=lens.long()),
           lambda: ops.cache_evict(dims, c, lens, 2, w.double()), lambda: ops.cache_evict(dims, c, lens, 2, w, new_len=lens[:1])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    ws = torch.empty(L.ssa_workspace_size(dims, L.SSA_OP_CACHE_DECODE), dtype=torch.uint8)
    for call in (lambda: ops.cache_decode(dims, c, lens, q, ws=ws), lambda: ops.cache_evict(dims, c, lens, 2, w, ws=ws)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.cache_decode(dims, c, lens, q, ws=ws[:-1].cuda()), lambda: ops.cache_evict(dims, c, lens, 0, w), lambda: ops.cache_evict(dims, c, lens, 2, w, sink=3),
                 lambda: ops.cache_decode(L.make_dims(2, 4, 256, D, 64, 2, Hkv=2), c._replace(Kbar=None), lens, q)):
        with pytest.raises(L.SSAError):
            call()


# ------------------------------------------------------------------------------- sizes, streams, capture
def test_offsets_beyond_32_bits():
    """A cache of 4.3 GB of codes each: the last sequence's rows lie beyond 2^32 bytes."""
    B, Hk, s, T = 33, 8, 128, 131072
    assert B * Hk * T * D > 2 ** 32
    dims, sparse = L.make_dims(B, 16, T, D, s, 0, Hkv=Hk), L.make_dims(B, 16, T, D, s, 4, Hkv=Hk)
    c = ops.Cache8.empty(dims)
    last = L.make_dims(1, 16, T, D, s, 0, Hkv=Hk)
    small = filled(last, [1500], seed=4)
    for whole, one in zip(c, small):
        whole.view(torch.uint8)[-1].copy_(one.view(torch.uint8)[0])
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    lens[-1] = 1500
    q = query(B, 16)
    for dm in (dims, sparse):
        w = torch.empty(B, Hk, T // s, device="cuda")
        out = ops.cache_decode(dm, c, lens, q, weight_out=w)
        one = [x[-1:] if x is not None else None for x in out]
        check_decode(L.make_dims(1, 16, T, D, s, dm.k, Hkv=Hk), small, [1500], q[-1:], one, None, w[-1:])
    # tokens into the last sequence, the same as into the small cache
    K = torch.randn(B, Hk, 100, D, device="cuda", generator=gen(1)).bfloat16()
    n_new = torch.zeros(B, dtype=torch.int32, device="cuda")
    n_new[-1] = 100
    ops.cache_append(dims, c, (lens + 1).contiguous(), K, -K, n_new)
    ops.cache_append(last, small, i32(1501), K[-1:], -K[-1:])
    weight = torch.rand(B, Hk, T // s, device="cuda", generator=gen(2))
    held = (lens + 1 + n_new).contiguous()
    kept, new_len = ops.cache_evict(dims, c, held, 7, weight)
    kept1, new1 = ops.cache_evict(last, small, held[-1:].clone(), 7, weight[-1:].contiguous())
    assert torch.equal(kept[-1:], kept1) and torch.equal(new_len[-1:], new1)
    n = int(new1[0])
    for whole, one in zip(c, small):
        rows = n if whole.shape[2] == T else -(-n // s) if whole.dim() == 3 else n // s
        assert torch.equal(whole[-1, :, :rows].contiguous().view(torch.uint8), one[0, :, :rows].contiguous().view(torch.uint8))
    assert L.ssa_get_device_error() == L.SSA_OK


def test_append_captured():
    """A captured step of one token, replayed from inside a block across its end, and a captured piece."""
    s, T = 64, 256
    dims = L.make_dims(2, 2, T, D, s, 0)
    for n, starts in ((1, (62, 63, 64)), (20, (50, 70, 108))):
        lens = i32(0, 0)
        c = filled(dims, [200, 200], garbage=False)
        K = torch.empty(2, 2, n, D, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.cache_append(dims, c, lens, K, K)
        for i, at in enumerate(starts):
            lens.copy_(torch.tensor([at, at + 17], dtype=torch.int32))
            K.copy_(torch.randn(K.shape, device="cuda", generator=gen(i)) * 4.0 ** i)
            before = snapshot(c)
            g.replay()
            torch.cuda.synchronize()
            check_append(dims, c, before, [at, at + 17], [n, n], K, K)


def test_two_calls_at_once():
    """Decodes of two caches on two streams, each with its workspace, while the other runs."""
    dims = [L.make_dims(8, 32, 4096, D, 128, 0, Hkv=8), L.make_dims(8, 16, 4096, D, 64, 9, Hkv=2)]
    lens = [[4095 - 300 * i for i in range(8)], [100 + 500 * i for i in range(8)]]
    caches = [filled(d, n, seed=i) for i, (d, n) in enumerate(zip(dims, lens))]
    qs = [query(8, 32, 1), query(8, 16, 2)]
    cl = [i32(*n) for n in lens]
    ws = [ops._ws(d, L.SSA_OP_CACHE_DECODE, "cuda") for d in dims]
    alone = [ops.cache_decode(d, c, n, q, ws=w) for d, c, n, q, w in zip(dims, caches, cl, qs, ws)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(ops.cache_decode(dims[i], caches[i], cl[i], qs[i], ws=ws[i]))
    torch.cuda.synchronize()
    for want, got in zip(alone, outs):
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(want, g) if a is not None)
    check_decode(dims[1], caches[1], lens[1], qs[1], alone[1])


def test_decode_of_broadcast_and_strided_new_rows():
    """Keys shared by every head (a stride of 0) are stored once per head; a batch of one with odd strides."""
    dims = L.make_dims(1, 4, 256, D, 64, 0)
    c, e = filled(dims, [9]), filled(dims, [9])
    x = torch.randn(1, 1, 30, D, device="cuda", generator=gen(1)).bfloat16()
    ops.cache_append(dims, c, i32(10), x.expand(1, 4, 30, D), x.expand(1, 4, 30, D))
    y = x.expand(1, 4, 30, D).contiguous()
    odd = torch.as_strided(y, y.shape, (7, 30 * D, D, 1))  # the stride of an extent of one is never used
    ops.cache_append(dims, e, i32(10), odd, odd)
    assert unchanged(c, snapshot(e))
    short = torch.as_strided(y, y.shape, (4 * 30 * D, 30 * D, D, 1), 0)[..., 1:]  # off a 16-byte boundary
    with pytest.raises((ValueError, L.SSAError)):
        ops.cache_append(dims, c, i32(10), short, short)
    wide = torch.zeros(1, 4, 30, 2 * D, dtype=torch.bfloat16, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        ops.cache_append(dims, c, i32(10), wide, wide)
