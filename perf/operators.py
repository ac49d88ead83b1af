"""The operators of serving from an 8-bit key/value cache, as calls to measure.

rope    rotary positions with several axes on the queries and keys (ssa_rope_axes)
append  new keys and values written into the 8-bit cache (ssa_cache_append)
decode  one query token per sequence over the 8-bit cache, all blocks or selected ones (ssa_cache_decode)
evict   blocks with little accumulated attention weight leave the cache (ssa_cache_evict)

``run`` computes them in elementary torch operations where ``own`` is false and
through this package where it is true.  The cache holds e4m3 codes [B, Hkv, T, d]
and a power-of-two fp32 scale per block of s tokens and key/value head.
"""
import math

import torch

own = False

D = 128                       # head size of the cache
BASE, FACTOR = 500000.0, 4.0  # rotary base and scaling factor of the long-context settings
MIN_SCALE = 2.0 ** -126
F8 = torch.float8_e4m3fn


# --------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------
def listed():
    return [
        # single tokens of a batch while decoding: text positions beside image ones, latency counts
        dict(name="rope, a token of 64 sequences", op="rope", B=64, T=1, H=32, Hkv=8, d=128, type="bf16", axes=3,
             ladder="shared", interleaved=False, transpose=False, rows="heads", far=30000),
        # a 32K prompt of video and text: three axes, rows as a projection leaves them ([B, T, heads, d])
        dict(name="rope, a 32K prompt", op="rope", B=1, T=32768, H=32, Hkv=8, d=128, type="bf16", axes=3,
             ladder="shared", interleaved=False, transpose=False, rows="tokens", far=8000),
        # gradients of an image batch's queries and keys: fp32, two axes with a ladder each, odd length
        dict(name="rope, fp32 gradients of images", op="rope", B=4, T=4097, H=16, Hkv=16, d=64, type="fp32", axes=2,
             ladder="own", interleaved=False, transpose=True, rows="heads", far=100),
        # the decode step's write: one token of each sequence
        dict(name="append, a token of 64 sequences", op="append", B=64, Hkv=8, T=4096, s=128, n=1, held="ragged",
             ragged=False),
        # a whole 32K prompt enters the cache
        dict(name="append, a 32K prompt", op="append", B=1, Hkv=8, T=32768, s=128, n=32768, held="none", ragged=False),
        # pieces of several prompts, of different lengths, into caches whose open block is partly filled
        dict(name="append, ragged pieces", op="append", B=8, Hkv=16, T=8192, s=64, n=1000, held="ragged", ragged=True),
        # a single conversation of about a thousand tokens: latency
        dict(name="decode, one short sequence", op="decode", B=1, H=32, Hkv=8, T=2048, s=128, k=0, held="ragged",
             weight=False),
        # mixed lengths, attention weight added up for the eviction
        dict(name="decode, 16 ragged sequences", op="decode", B=16, H=16, Hkv=2, T=32768, s=64, k=0, held="ragged",
             weight=True),
        # the sparse decode of this repository's benchmark, on the 8-bit cache
        dict(name="decode, 64 x 32K, 16 blocks", op="decode", B=64, H=32, Hkv=8, T=32768, s=128, k=16, held="half",
             weight=True),
        # every key of 64 caches of 32K tokens
        dict(name="decode, 64 x 32K, all blocks", op="decode", B=64, H=32, Hkv=8, T=32768, s=128, k=0, held="half",
             weight=False),
        # a small cache at its budget loses one block
        dict(name="evict one of 17 blocks", op="evict", B=4, Hkv=8, T=2048, s=64, held="budget", keep=16, sink=1, recent=2),
        # half of 32 long caches goes
        dict(name="evict half of 32 x 32K", op="evict", B=32, Hkv=8, T=32768, s=128, held="half", keep=96, sink=1, recent=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        H = Hkv * rng.choice([1, 2, 4, 5, 8]) if Hkv < 16 else 16
        B, d = _log_int(rng, 1, 64), rng.choice([64, 128, 128])
        kind = rng.choice(["bf16", "bf16", "fp32"])
        most = 300_000_000 // (B * (H + Hkv) * d * (2 if kind == "bf16" else 4))
        T = _log_int(rng, 1, max(1, min(32768, most)))
        return dict(op=op, B=B, T=T, H=H, Hkv=Hkv, d=d, type=kind, axes=rng.choice([1, 2, 3, 3]),
                    ladder=rng.choice(["shared", "shared", "own"]), interleaved=rng.random() < 0.4,
                    transpose=rng.random() < 0.4, rows=rng.choice(["heads", "tokens"]), far=_log_int(rng, 64, 1_000_000))
    s, Hkv, B = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16]), _log_int(rng, 1, 64)
    nb = _log_int(rng, 4, max(4, min(32768 // s, 500_000_000 // (B * Hkv * s * D))))
    T = nb * s
    if op == "append":
        n = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, T // 2))
        return dict(op=op, B=B, Hkv=Hkv, T=T, s=s, n=n, held=rng.choice(["ragged", "none"]) if n < T // 2 else "none",
                    ragged=n > 1 and rng.random() < 0.6)
    if op == "decode":
        G = rng.choice([1, 2, 4, 4, 5, 8, 12, 16])
        k = 0 if rng.random() < 0.5 else _log_int(rng, 1, min(64, nb))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, T=T, s=s, k=k, held=rng.choice(["ragged", "half"]),
                    weight=rng.random() < 0.6)
    keep = _log_int(rng, 1, nb - 1)
    return dict(op=op, B=B, Hkv=Hkv, T=T, s=s, held=rng.choice(["ragged", "half"]), keep=keep,
                sink=1 if keep >= 8 and rng.random() < 0.7 else 0, recent=keep // 4 if rng.random() < 0.7 else 0)


def _held(c):
    """Tokens that each sequence's cache holds before the call; they depend on the case alone."""
    T, B, s = c["T"], c["B"], c["s"]
    room = c.get("n", 1)
    part = [(0.37 + 0.6180339887 * b) % 1.0 for b in range(B)]
    if c["held"] == "none":
        return [0] * B
    if c["held"] == "budget":  # one block over the budget, the next one begun in some sequences
        return [(c["keep"] + 1) * s + int(f * s) for f in part]
    lo = T // 2 if c["held"] == "half" else 0
    return [lo + int(f * (T - room - lo)) for f in part]


def _new(c):
    """New tokens of each sequence of an append."""
    return [max(0, c["n"] - (b * c["n"]) // c["B"] - b % 3) if c["ragged"] else c["n"] for b in range(c["B"])]


# --------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _smallest_scale(amax):
    """The smallest power of two, at least 2^-126, that brings amax to 448 or less (fp32; amax finite)."""
    m, e = torch.frexp(amax)
    p = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), p.clamp(min=-126)), torch.full_like(amax, MIN_SCALE))


def _quantise(x):
    """Codes and scales of blocks x [..., nb, s, d]."""
    scale = _smallest_scale(x.abs().amax((-2, -1)))
    return (x / scale[..., None, None]).to(F8), scale


def _cache(c, g):
    """A filled cache: normal keys and values, of another size in every block, quantised block by block."""
    B, Hkv, T, s = c["B"], c["Hkv"], c["T"], c["s"]
    nb = T // s
    st = {"K8": torch.empty(B, Hkv, T, D, dtype=F8, device="cuda"), "V8": torch.empty(B, Hkv, T, D, dtype=F8, device="cuda"),
          "K_scale": torch.empty(B, Hkv, nb, device="cuda"), "V_scale": torch.empty(B, Hkv, nb, device="cuda"),
          "Kbar": torch.empty(B, Hkv, nb, D, device="cuda")}
    for b in range(B):
        for x, sc in (("K8", "K_scale"), ("V8", "V_scale")):
            v = torch.randn(Hkv, nb, s, D, device="cuda", generator=g)
            v *= torch.exp(0.3 * torch.randn(Hkv, nb, 1, 1, device="cuda", generator=g))
            codes, scale = _quantise(v)
            st[x][b] = codes.view(Hkv, T, D)
            st[sc][b] = scale
            if x == "K8":
                st["Kbar"][b] = codes.float().mul_(scale[..., None, None]).mean(2)
    return st


def _sections(c):
    half = c["d"] // 2
    if c["axes"] == 1:
        return [half]
    if c["axes"] == 2:
        return [half // 2, half - half // 2]
    first = half // 4
    return [first, (half - first) // 2, half - first - (half - first) // 2]


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "rope":
        t = torch.bfloat16 if c["type"] == "bf16" else torch.float32
        pos = torch.randint(0, c["far"] + 1, (c["axes"], c["B"], c["T"]), device="cuda", generator=g, dtype=torch.int32)
        axis, freq = _axes_and_frequencies(c, "cuda")
        st = {"pos": pos, "axis": axis, "freq": freq}
        for name, heads in (("Q", c["H"]), ("K", c["Hkv"])):
            if c["rows"] == "tokens":
                x = torch.randn(c["B"], c["T"], heads, c["d"], device="cuda", generator=g).to(t).transpose(1, 2)
            else:
                x = torch.randn(c["B"], heads, c["T"], c["d"], device="cuda", generator=g).to(t)
            st[name] = x
    else:
        st = _cache(c, g)
        st["cache_len"] = torch.tensor(_held(c), dtype=torch.int32, device="cuda")
        if c["op"] == "append":
            st["n_new"] = torch.tensor(_new(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
            for name in ("K", "V"):  # rows as a projection leaves them
                st[name] = torch.randn(c["B"], c["n"], c["Hkv"], D, device="cuda", generator=g).bfloat16().transpose(1, 2)
        elif c["op"] == "decode":
            # logits of standard deviation 2: attention over some hundreds of the tokens
            st["q"] = (2.0 * torch.randn(c["B"], c["H"], D, device="cuda", generator=g)).bfloat16()
            st["weight"] = torch.rand(c["B"], c["Hkv"], c["T"] // c["s"], device="cuda", generator=g) if c["weight"] else None
        else:
            st["weight"] = torch.randn(c["B"], c["Hkv"], c["T"] // c["s"], device="cuda", generator=g).square_()
    st["case"] = c
    return st


# --------------------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------------------
def _axes_and_frequencies(c, device):
    """Axis of every pair and its angle per position (64 bits), without the scaling factor."""
    half, sections = c["d"] // 2, _sections(c)
    if c["interleaved"]:  # dealt out in turn, an axis left out once its section is full
        left, axis = list(sections), []
        while len(axis) < half:
            axis += [a for a in range(len(left)) if left[a] > 0]
            left = [max(0, n - 1) for n in left]
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if c["ladder"] == "own":
        power = [axis[:i].count(axis[i]) / sections[axis[i]] for i in range(half)]
    else:
        power = [i / half for i in range(half)]
    freq = torch.tensor([BASE ** -p for p in power], dtype=torch.float64)
    return torch.tensor(axis, device=device), freq.to(device)


def _plain_rope(st):
    c = st["case"]
    angle = st["pos"].double()[st["axis"]].permute(1, 2, 0) * st["freq"] / FACTOR  # [B, T, d/2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sin = -sin if c["transpose"] else sin

    def turn(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(x.dtype)

    return {"Q": turn(st["Q"]), "K": turn(st["K"])}


def _plain_append_one(new, codes, scale, L, n_new, s):
    """One tensor's new rows [B, Hkv, n, d] into codes [B, Hkv, T, d] and scale [B, Hkv, nb], in place."""
    B, Hkv, n, d = new.shape
    nb = scale.shape[2]
    m = min(nb, (n + s - 2) // s + 1)                                 # blocks that n rows can touch
    block = (L[:, None] // s + torch.arange(m, device=L.device)).long()       # [B, m]
    inside = block < nb
    at = block % nb                                                           # distinct, and unchanged where outside
    row = block[:, :, None] * s + torch.arange(s, device=L.device)            # [B, m, s] token of every row
    fresh = (row >= L[:, None, None]) & (row < (L + n_new)[:, None, None]) & inside[..., None]
    older = (row < L[:, None, None]) & inside[..., None]
    at_b = torch.arange(B, device=L.device)[:, None]
    cur = codes.view(B, Hkv, nb, s, d)[at_b, :, at]                           # [B, m, Hkv, s, d]
    old_scale = scale[at_b, :, at]                                            # [B, m, Hkv]
    src = (row - L[:, None, None]).clamp(0, n - 1)
    x = new.transpose(1, 2)[at_b[..., None], src].permute(0, 1, 3, 2, 4).float()  # [B, m, Hkv, s, d]
    amax = torch.where(fresh[:, :, None, :, None] & x.isfinite(), x.abs(), 0.0).amax((-2, -1))
    had = older.any(-1)[..., None]
    want = torch.where(had, torch.maximum(_smallest_scale(amax), old_scale), _smallest_scale(amax))
    touched = fresh.any(-1)[..., None]
    want = torch.where(touched, want, old_scale)
    coded = torch.where(x.isfinite(), x / want[..., None, None], math.nan).to(F8).float()
    again = (cur.float() * old_scale[..., None, None] / want[..., None, None]).to(F8).float()
    out = torch.where(fresh[:, :, None, :, None], coded,
                      torch.where((older & touched)[:, :, None, :, None], again, cur.float())).to(F8)
    codes.view(torch.uint8).view(B, Hkv, nb, s, d)[at_b, :, at] = out.view(torch.uint8)
    scale[at_b, :, at] = want
    return fresh[:, :, -1], at_b, at, out, want                               # fresh: the block's last row is new


def _plain_append(st):
    c, L, s = st["case"], st["cache_len"], st["case"]["s"]
    n_new = st["n_new"] if st["n_new"] is not None else torch.full_like(L, c["n"])
    done, at_b, at, out, want = _plain_append_one(st["K"], st["K8"], st["K_scale"], L, n_new, s)
    _plain_append_one(st["V"], st["V8"], st["V_scale"], L, n_new, s)
    mean = out.float().sum(3) * want[..., None] / s
    st["Kbar"][at_b, :, at] = torch.where(done[:, :, None, None], mean, st["Kbar"][at_b, :, at])
    return {x: st[x] for x in ("K8", "V8", "K_scale", "V_scale", "Kbar")}


def _plain_select(st, bt):
    """Own block and the k - 1 highest of the ones before it, ascending, -1 behind (scores summed in 64 bits)."""
    c = st["case"]
    B, Hkv, nb, k = c["B"], c["Hkv"], c["T"] // c["s"], c["k"]
    q = st["q"].double().view(B, Hkv, -1, D).sum(2)
    score = (st["Kbar"].double() @ q[..., None])[..., 0].float()
    j = torch.arange(nb, device=q.device)
    score = torch.where(j < bt[:, None, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k - 1]
    chosen = torch.where(order < bt[:, None, None], order, nb)
    chosen = torch.cat([chosen, bt[:, None, None].expand(B, Hkv, 1)], -1).sort(-1).values
    return torch.where(chosen < nb, chosen, -1).int()


def _plain_decode(st):
    c, L = st["case"], st["cache_len"].long()
    B, Hkv, s, nb, k = c["B"], c["Hkv"], c["s"], c["T"] // c["s"], c["k"]
    K, V = st["K8"].view(B, Hkv, nb, s, D), st["V8"].view(B, Hkv, nb, s, D)
    ks, vs = st["K_scale"], st["V_scale"]
    q = st["q"].float().view(B, Hkv, -1, D)
    out = {}
    if k:
        idx = _plain_select(st, L // s)
        out["idx"] = idx
        at = idx.long().clamp(min=0)
        b_i, h_i = torch.arange(B, device=L.device)[:, None, None], torch.arange(Hkv, device=L.device)[None, :, None]
        K, V, ks, vs = K[b_i, h_i, at], V[b_i, h_i, at], ks[b_i, h_i, at], vs[b_i, h_i, at]
        token = idx.long()[..., None] * s + torch.arange(s, device=L.device)
        seen = (token >= 0) & (idx[..., None] >= 0) & (token <= L[:, None, None, None])
    else:
        token = torch.arange(nb * s, device=L.device).view(1, 1, nb, s)
        seen = (token <= L[:, None, None, None]).expand(B, Hkv, nb, s)
    n = K.shape[2]
    x = K.float().mul_(ks[..., None, None]).view(B, Hkv, n * s, D)
    logit = torch.matmul(q, x.transpose(-1, -2)) * D ** -0.5
    logit = torch.where(seen.reshape(B, Hkv, 1, n * s), logit, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    p = p / total
    out["lse"] = (top + total.log()).view(B, -1)
    x = V.float().mul_(vs[..., None, None]).view(B, Hkv, n * s, D)
    out["o"] = torch.matmul(p, x).view(B, -1, D).bfloat16()
    if st["weight"] is not None:
        w = p.view(B, Hkv, -1, n, s).sum((2, 4))
        out["weight"] = st["weight"] + (w if not k else torch.zeros_like(st["weight"]).scatter_add_(
            2, at, torch.where(idx >= 0, w, 0.0)))
    return out


def _plain_evict(st):
    c, L = st["case"], st["cache_len"].long()
    B, Hkv, s, nb, keep = c["B"], c["Hkv"], c["s"], c["T"] // c["s"], c["keep"]
    whole = (L // s)[:, None, None]
    j = torch.arange(nb, device=L.device)
    safe = (j < c["sink"]) | (j >= whole - c["recent"])
    w = torch.where(safe, math.inf, torch.nan_to_num(st["weight"], nan=-math.inf))
    w = torch.where(j < whole, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(order < whole, order, nb).sort(-1).values               # ascending, nb behind
    kept = torch.where(whole > keep, kept, torch.where(j[:keep] < whole, j[:keep], nb))
    left = torch.minimum(whole, torch.full_like(whole, keep))                  # complete blocks that stay
    begun = (L % s > 0)[:, None, None]
    move = torch.cat([kept, torch.full_like(kept[..., :1], nb)], -1)
    move = torch.where((torch.arange(keep + 1, device=L.device) == left) & begun, whole, move)
    stays = (move < nb)
    src = j.expand(B, Hkv, nb).clone()
    n = min(nb, keep + 1)
    src[..., :n] = torch.where(stays, move, torch.arange(keep + 1, device=L.device))[..., :n]
    for_rows = src[..., None].expand(B, Hkv, nb, s * D // 8)
    codes = [st[x].view(torch.int64).view(B, Hkv, nb, s * D // 8) for x in ("K8", "V8")]
    codes[0].copy_(torch.gather(codes[0], 2, for_rows))
    codes[1].copy_(torch.gather(codes[1], 2, for_rows))
    st["K_scale"].copy_(torch.gather(st["K_scale"], 2, src))
    st["V_scale"].copy_(torch.gather(st["V_scale"], 2, src))
    st["Kbar"].copy_(torch.gather(st["Kbar"], 2, src[..., None].expand(B, Hkv, nb, D)))
    weight = torch.where(j < left + begun, torch.gather(st["weight"], 2, src), 0.0)
    return {"kept": torch.where(kept < nb, kept, -1).int(), "new_len": (left[:, 0, 0] * s + L % s).int(), "weight": weight,
            **{x: st[x] for x in ("K8", "V8", "K_scale", "V_scale", "Kbar")}}


# --------------------------------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------------------------------
def _own(st):
    from block_top_sparse_b200 import _lib, ops
    c = st["case"]
    if c["op"] == "rope":
        dims = _lib.make_dims(c["B"], c["H"], c["T"], c["d"], 64, 1, c["type"], Hkv=c["Hkv"])
        Q, K = ops.rope_axes(dims, st["pos"], _sections(c), st["Q"], st["K"], base=BASE, factor=FACTOR,
                             interleaved=c["interleaved"], own_ladder=c["ladder"] == "own", transpose=c["transpose"])
        return {"Q": Q, "K": K}
    dims = _lib.make_dims(c["B"], c.get("H", c["Hkv"]), c["T"], D, c["s"], c.get("k", 0), Hkv=c["Hkv"])
    cache = ops.Cache8(st["K8"], st["K_scale"], st["V8"], st["V_scale"], st["Kbar"])
    if c["op"] == "append":
        ops.cache_append(dims, cache, st["cache_len"], st["K"], st["V"], n_new=st["n_new"])
        return {x: st[x] for x in ("K8", "V8", "K_scale", "V_scale", "Kbar")}
    if c["op"] == "decode":
        weight = None if st["weight"] is None else torch.empty_like(st["weight"])
        o, lse, idx = ops.cache_decode(dims, cache, st["cache_len"], st["q"], weight_in=st["weight"], weight_out=weight)
        out = {"o": o, "lse": lse}
        if c["k"]:
            out["idx"] = idx
        if weight is not None:
            out["weight"] = weight
        return out
    weight = torch.empty_like(st["weight"])
    kept, new_len = ops.cache_evict(dims, cache, st["cache_len"], c["keep"], st["weight"], sink=c["sink"],
                                    recent=c["recent"], weight_out=weight)
    return {"kept": kept, "new_len": new_len, "weight": weight,
            **{x: st[x] for x in ("K8", "V8", "K_scale", "V_scale", "Kbar")}}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[
        state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------
# Work and exact values
# --------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["B"] * c["T"] * (c["H"] + c["Hkv"])
        return {"bytes": 2 * rows * c["d"] * (2 if c["type"] == "bf16" else 4) + 4 * c["axes"] * c["B"] * c["T"],
                "flops": 3 * rows * c["d"]}
    s, Hkv, held = c["s"], c["Hkv"], _held(c)
    if c["op"] == "append":
        b = f = 0
        for L, n in zip(held, _new(c)):
            blocks = (L + n - 1) // s - L // s + 1 if n else 0
            b += Hkv * (n * D * (2 * 2 + 2 * 1) + blocks * 2 * 4 + ((L + n) // s - L // s) * D * 4)
            f += Hkv * n * D * 6
        return {"bytes": b, "flops": f}
    if c["op"] == "decode":
        b = c["B"] * c["H"] * (D * 2 * 2 + 4) + (2 * 4 * c["B"] * Hkv * (c["T"] // s) if c["weight"] else 0)
        f = 0
        for L in held:
            keys = L + 1 if not c["k"] else min(c["k"] - 1, L // s) * s + L % s + 1
            b += Hkv * (keys * D * 2 + 2 * 4 * -(-keys // s))
            f += 4 * D * c["H"] * keys
            if c["k"] > 1:
                b += Hkv * (L // s) * D * 4
                f += 2 * D * Hkv * (L // s)
        return {"bytes": b, "flops": f}
    b = 0
    for L in held:
        whole = L // s
        gone = whole - c["keep"]
        b += Hkv * 4 * whole
        if gone > 0:  # the blocks behind the first one that goes move, as does the one begun
            free = whole - c["sink"] - c["recent"]
            moved = c["keep"] - c["sink"] - (free - gone) / (gone + 1) + (1 if L % s else 0)
            b += int(Hkv * moved * 2 * (2 * s * D + 2 * 4 + D * 4))
    return {"bytes": b, "flops": c["B"] * Hkv * c["T"] // s}


def _nearest_e4m3(x):
    """x (64 bits, |x| <= 464) rounded to a number with 4 significant bits that is a multiple of 2^-9, ties to even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_scale(amax):
    """math.ceil(log2(amax / 448)) by trial, as a 64-bit power of two."""
    p = torch.full_like(amax, -126.0)
    for _ in range(300):
        small = amax > 448.0 * torch.exp2(p)
        if not bool(small.any()):
            break
        p = p + small
    return torch.exp2(p)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "rope":
        sections, half, out = _sections(c), c["d"] // 2, {"Q": st["Q"].double(), "K": st["K"].double()}
        rank, owner, i = [0] * len(sections), [], 0
        while len(owner) < half:
            if c["interleaved"]:
                a = i % len(sections)
                i += 1
                if rank[a] >= sections[a]:
                    continue
            else:
                a = next(a for a in range(len(sections)) if rank[a] < sections[a])
            owner.append((a, rank[a]))
            rank[a] += 1
        got = {name: torch.empty_like(x) for name, x in out.items()}
        for pair, (a, r) in enumerate(owner):
            rate = BASE ** (-2.0 * r / (2 * sections[a])) if c["ladder"] == "own" else BASE ** (-2.0 * pair / c["d"])
            turn = st["pos"][a].double() * rate / FACTOR * (-1.0 if c["transpose"] else 1.0)  # [B, T]
            for name, x in out.items():
                z = torch.complex(x[..., pair], x[..., pair + half]) * torch.polar(torch.ones_like(turn), turn)[:, None]
                got[name][..., pair], got[name][..., pair + half] = z.real, z.imag
        return got
    s, B, Hkv, nb = c["s"], c["B"], c["Hkv"], c["T"] // c["s"]
    held = _held(c)
    if c["op"] == "append":
        out = {}
        for x, codes, scales in (("K", "K8", "K_scale"), ("V", "V8", "V_scale")):
            C, S = st[codes].double(), st[scales].double()
            for b, (L, n) in enumerate(zip(held, _new(c))):
                at = L
                while at < L + n:
                    j, to = at // s, min(L + n, (at // s + 1) * s)
                    if at % s == 0:  # all the whole blocks from here on at once
                        to = max(to, (L + n) // s * s)
                    count = -(-(to - at) // s)
                    v = st[x][b, :, at - L:to - L].double()
                    pad = torch.zeros(Hkv, count * s - (to - at), D, dtype=torch.float64, device=v.device)
                    top = torch.cat([v, pad], 1).view(Hkv, count, -1).abs().amax(-1)
                    scale = _exact_scale(top)
                    if at % s:
                        scale = torch.maximum(scale, S[b, :, j:j + 1])
                        C[b, :, j * s:at] = _nearest_e4m3(C[b, :, j * s:at] * (S[b, :, j:j + 1] / scale)[..., None])
                    S[b, :, j:j + count] = scale
                    C[b, :, at:to] = _nearest_e4m3(v / scale.repeat_interleave(s, 1)[:, :to - at, None])
                    at = to
            out[codes], out[scales] = C, S
        out["Kbar"] = st["Kbar"].double()
        for b, (L, n) in enumerate(zip(held, _new(c))):
            lo, hi = L // s, (L + n) // s
            if hi > lo:
                blocks = out["K8"][b, :, lo * s:hi * s].view(Hkv, hi - lo, s, D)
                out["Kbar"][b, :, lo:hi] = blocks.mean(2) * out["K_scale"][b, :, lo:hi, None]
        return out
    if c["op"] == "decode":
        G = c["H"] // Hkv
        o = torch.empty(B, c["H"], D, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, c["H"], dtype=torch.float64, device="cuda")
        weight = None if st["weight"] is None else st["weight"].double()
        for b, L in enumerate(held):
            bt = L // s
            q = st["q"][b].double().view(Hkv, G, D)
            if c["k"]:
                r = (st["Kbar"][b, :, :bt].double() * q.sum(1)[:, None]).sum(-1).float().tolist()
                rows = [sorted(sorted(range(bt), key=lambda j: (-r[h][j], j))[:c["k"] - 1] + [bt]) for h in range(Hkv)]
                blocks = torch.tensor(rows, device="cuda")
            else:
                blocks = torch.arange(bt + 1, device="cuda").expand(Hkv, bt + 1)
            h_i = torch.arange(Hkv, device="cuda")[:, None]
            keys = (blocks.shape[1] - 1) * s + L % s + 1  # the own block comes last
            pick = lambda x, sc: (st[x][b].view(Hkv, nb, s, D)[h_i, blocks].double()  # noqa: E731
                                  * st[sc][b][h_i, blocks].double()[..., None, None]).view(Hkv, -1, D)[:, :keys]
            z = torch.einsum("hgd,hud->hgu", q, pick("K8", "K_scale")) / math.sqrt(D)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - total[..., None])
            o[b] = torch.einsum("hgu,hud->hgd", p, pick("V8", "V_scale")).reshape(c["H"], D)
            lse[b] = total.reshape(-1)
            if weight is not None:
                mass = torch.cat([p.sum(1), torch.zeros(Hkv, blocks.shape[1] * s - keys, dtype=p.dtype, device="cuda")], 1)
                weight[b].scatter_add_(1, blocks, mass.view(Hkv, -1, s).sum(-1))
        out = {"o": o, "lse": lse}
        if c["k"]:
            out["idx"] = None
        if weight is not None:
            out["weight"] = weight
        return out
    names = ("K8", "V8", "K_scale", "V_scale", "Kbar")
    got = {x: st[x].view(torch.uint8).clone().view(F8) if x in ("K8", "V8") else st[x].clone() for x in names}
    weight, w = torch.zeros_like(st["weight"], dtype=torch.float64), st["weight"].tolist()
    for b, L in enumerate(held):
        whole = L // s
        for h in range(Hkv):
            rows = list(range(whole))
            if whole > c["keep"]:
                always = [j for j in rows if j < c["sink"] or j >= whole - c["recent"]]
                rest = sorted((j for j in rows if j not in always), key=lambda j: (-w[b][h][j], j))
                rows = sorted(always + rest[:c["keep"] - len(always)])
            rows += [whole] if L % s else []
            src = torch.tensor(rows, device="cuda")
            for x in names:
                t = st[x][b, h].view(nb, -1)
                t, to = (t.view(torch.uint8), got[x][b, h].view(nb, -1).view(torch.uint8)) if x in ("K8", "V8") else (
                    t, got[x][b, h].view(nb, -1))
                to[:len(rows)] = t[src]
            weight[b, h, :len(rows)] = st["weight"][b, h, src].double()
    return {"kept": None, "new_len": None, "weight": weight, **got}
