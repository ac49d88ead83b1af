"""Rotary positions with several axes (ssa_rope_axes) against the 64-bit definition.

Bounds: the angle's turn fraction is exact to about pos * 2^-52 turns, its cosine
and sine are fp32 values with an error of at most 4 * 2^-24, and an output is two
products and a sum in fp32: 8 * 2^-24 of |x_i| + |x_j|; a bf16 output is rounded
once more, by at most 2^-8 of its value."""
import numpy as np
import pytest

from block_top_sparse_b200 import _lib as L
from block_top_sparse_b200 import ops

from . import cache_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from block_top_sparse_b200 import build
    build.build()


def check(y, x, pos, sections, base, factor, **kw):
    ref = R.rope_axes(x.double().cpu().numpy(), pos.cpu().numpy(), sections, base, factor, **kw)
    a = x.double().abs().cpu().numpy()
    h = a.shape[-1] // 2
    size = a + np.concatenate([a[..., h:], a[..., :h]], -1)
    far = float(pos.abs().max()) * 2.0 ** -50 if pos.numel() else 0.0
    tol = (8 * 2.0 ** -24 + far) * size + (2.0 ** -8 * np.abs(ref) if y.dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)


def inputs(B, H, T, d, dtype, rows, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if rows == "tokens":
        return torch.randn(B, T, H, d, device="cuda", generator=g).to(dtype).transpose(1, 2)
    if rows == "fused":  # the middle of a wider projection
        return torch.randn(B, T, H * d + 3 * d, device="cuda", generator=g).to(dtype)[..., d:d + H * d].view(B, T, H, d).transpose(1, 2)
    return torch.randn(B, H, T, d, device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("B,H,Hkv,T,d,dtype,sections,rows", [
    (1, 1, 1, 1, 64, torch.bfloat16, [32], "heads"), (3, 5, 5, 1, 128, torch.bfloat16, [16, 24, 24], "heads"),
    (2, 8, 2, 17, 128, torch.float32, [32, 32], "tokens"), (1, 32, 8, 333, 128, torch.bfloat16, [16, 24, 24], "tokens"),
    (2, 4, 1, 130, 64, torch.float32, [1, 30, 1], "heads"), (64, 3, 1, 1, 64, torch.float32, [8, 8, 8, 8], "fused"),
    (1, 2, 2, 5000, 128, torch.bfloat16, [64], "fused"), (300, 1, 1, 2, 128, torch.float32, [10, 54], "heads")])
@pytest.mark.parametrize("interleaved,own_ladder,transpose", [(False, False, False), (True, False, True), (True, True, False)])
def test_matches_the_definition(B, H, Hkv, T, d, dtype, sections, rows, interleaved, own_ladder, transpose):
    dims = L.make_dims(B, H, T, d, 64, Hkv=Hkv)
    Q, K = inputs(B, H, T, d, dtype, rows, 1), inputs(B, Hkv, T, d, dtype, rows, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 40000, (len(sections), B, T), device="cuda", generator=g, dtype=torch.int32)
    kw = dict(interleaved=interleaved, own_ladder=own_ladder, transpose=transpose)
    Qr, Kr = ops.rope_axes(dims, pos, sections, Q, K, base=500000.0, factor=4.0, **kw)
    check(Qr, Q, pos, sections, 500000.0, 4.0, **kw)
    check(Kr, K, pos, sections, 500000.0, 4.0, **kw)
    # in place, on the views themselves; then the queries alone: the same values
    Q2, K2 = inputs(B, H, T, d, dtype, rows, 1), inputs(B, Hkv, T, d, dtype, rows, 2)
    ops.rope_axes(dims, pos, sections, Q2, K2, base=500000.0, factor=4.0, out=(Q2, K2), **kw)
    assert torch.equal(Q2, Qr) and torch.equal(K2, Kr)
    only, none = ops.rope_axes(dims, pos, sections, Q, base=500000.0, factor=4.0, **kw)
    assert none is None and torch.equal(only, Qr)


def test_far_and_negative_positions():
    dims = L.make_dims(1, 2, 6, 128, 64)
    pos = torch.tensor([[[0, -1, 2 ** 23 + 1, -2 ** 24, 2 ** 31 - 1, -2 ** 31]]], dtype=torch.int32, device="cuda")
    Q = inputs(1, 2, 6, 128, torch.float32, "heads")
    Qr, _ = ops.rope_axes(dims, pos, [64], Q, base=10000.0)
    check(Qr, Q, pos.to(torch.int64), [64], 10000.0, 1.0)


def test_one_axis_is_the_single_axis_call():
    dims = L.make_dims(2, 4, 256, 128, 64)
    Q = inputs(2, 4, 256, 128, torch.bfloat16, "heads")
    pos = (777 + torch.arange(256, device="cuda", dtype=torch.int32)).expand(1, 2, 256).contiguous()
    Qr, _ = ops.rope_axes(dims, pos, [64], Q, base=10000.0, factor=4.0)
    old = ops.rope(dims, Q.clone(), pos0=777, base=10000.0, factor=4.0)
    # both are within one fp32 rounding of the exact value before theirs to bf16: equal, or one step apart
    assert float((Qr.float() - old.float()).abs().max()) <= 2.0 ** -7 * float(old.abs().max())
    assert float((Qr != old).float().mean()) < 1e-3


def test_gradient_is_the_transpose():
    # <dY, rope(x)> has the gradient rope^T(dY); differences of the loss along random directions agree.  The loss
    # is linear in x, so the difference quotient is exact but for rounding: |e| <= 2^-22 sum |dY| (|x| + |step|) / step
    dims = L.make_dims(1, 2, 31, 64, 64)
    g = torch.Generator(device="cuda").manual_seed(5)
    pos = torch.randint(0, 900, (2, 1, 31), device="cuda", generator=g, dtype=torch.int32)
    x, dY, u = (torch.randn(1, 2, 31, 64, device="cuda", generator=g) for _ in range(3))
    f = lambda t, **kw: ops.rope_axes(dims, pos, [12, 20], t, interleaved=True, **kw)[0]  # noqa: E731
    dX = f(dY, transpose=True)
    loss = lambda t: float((f(t).double() * dY.double()).sum())  # noqa: E731
    step = 0.5
    quotient = (loss(x + step * u) - loss(x - step * u)) / (2 * step)
    exact = float((dX.double() * u.double()).sum())
    bound = 2.0 ** -22 * float((dY.abs().sum() * (x.abs().max() + step * u.abs().max()) * 2)) / step
    assert abs(quotient - exact) <= bound
    check(dX, dY, pos, [12, 20], 10000.0, 1.0, interleaved=True, transpose=True)


def test_other_stream_and_captured():
    dims = L.make_dims(4, 8, 1, 128, 64, Hkv=2)
    pos = torch.randint(0, 99, (3, 4, 1), device="cuda", dtype=torch.int32)
    Q, K = inputs(4, 8, 1, 128, torch.bfloat16, "heads", 1), inputs(4, 2, 1, 128, torch.bfloat16, "heads", 2)
    out = (torch.empty_like(Q), torch.empty_like(K))
    want = ops.rope_axes(dims, pos, [16, 24, 24], Q, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.rope_axes(dims, pos, [16, 24, 24], Q, K, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    pos += 5
    graph.replay()
    want = ops.rope_axes(dims, pos, [16, 24, 24], Q, K)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_tensor_checks():
    dims = L.make_dims(1, 2, 4, 128, 64)
    Q = inputs(1, 2, 4, 128, torch.bfloat16, "heads")
    pos = torch.zeros(1, 1, 4, dtype=torch.int32, device="cuda")
    for bad in (lambda: ops.rope_axes(dims, pos.long(), [64], Q), lambda: ops.rope_axes(dims, pos[:, :, :3], [64], Q),
                lambda: ops.rope_axes(dims, pos, [64], Q.half()), lambda: ops.rope_axes(dims, pos, [64], Q.cpu()),
                lambda: ops.rope_axes(dims, pos, [64], Q, Q.float()), lambda: ops.rope_axes(dims, pos, [64], Q[..., :64]),
                lambda: ops.rope_axes(dims, pos, [64], Q, out=(Q, Q))):
        with pytest.raises(ValueError):
            bad()
