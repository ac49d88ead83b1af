"""The 8-bit cache's calls where their contract is narrowest, against the 64-bit
definitions (cache_ref.py); the ordinary shapes are in test_gpu_cache.py, whose
bounds hold here too unless a tighter one is derived at the test."""
import numpy as np
import pytest

from block_top_sparse_b200 import _lib as L
from block_top_sparse_b200 import ops

from . import cache_ref as R
from .test_gpu_cache import D, filled, gen, i32

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
