"""Rotary positions (mla_rope) against the rotation written out in fp64.

Tolerance: the rotation runs in fp32 on cos and sin that are off by at most 3e-7 (the reduced
half turn's rounding, pi * 2^-25; sincospif; the magnitude's product) and three roundings of
2^-24 each follow, so |error| <= 5e-7 * m * (|x0| + |x1|), plus half a step of the output type
(and of its subnormals)."""

import math

import pytest
import torch

from paged_mla_decode_11_b200 import ops

pytestmark = pytest.mark.gpu


def rotated(x, pos, freq, interleaved, magnitude, inverse):
    """fp64 result and the largest of |x0| + |x1| that each element comes from."""
    y = x.double().clone()
    n = freq.numel()
    r = y[..., y.shape[-1] - 2 * n:]
    a = pos.double()[:, None, None] * freq * (-1 if inverse else 1)
    x0, x1 = (r[..., 0::2].clone(), r[..., 1::2].clone()) if interleaved else (r[..., :n].clone(), r[..., n:].clone())
    y0, y1 = magnitude * (x0 * a.cos() - x1 * a.sin()), magnitude * (x0 * a.sin() + x1 * a.cos())
    size = torch.zeros_like(y)
    s = size[..., size.shape[-1] - 2 * n:]
    for part, lo, hi in ((r, y0, y1), (s, x0.abs() + x1.abs(), x0.abs() + x1.abs())):
        if interleaved:
            part[..., 0::2], part[..., 1::2] = lo, hi
        else:
            part[..., :n], part[..., n:] = lo, hi
    return y, size


def check(x, pos, freq, out, interleaved=True, magnitude=1.0, inverse=False):
    ref, size = rotated(x, pos, freq, interleaved, magnitude, inverse)
    info = torch.finfo(x.dtype)
    front = x.shape[-1] - 2 * freq.numel()
    assert torch.equal(out[..., :front], x[..., :front])
    tol = info.eps / 2 * ref.abs() + 5e-7 * magnitude * size + info.smallest_normal * info.eps
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} elements off, worst {((out.double() - ref).abs() / tol).max():.3f} of the tolerance"


def draw(T, H, D, dtype, seed=0, far=4096):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    return x, torch.randint(-far, far, (T,), generator=g, device="cuda")


CASES = [
    # (T, H, D, pairs)
    (1, 1, 64, 32),          # one token, one head
    (1, 128, 192, 32),       # one token's query heads, 128 columns in front
    (3, 5, 64, 32),
    (130, 16, 64, 32),
    (257, 3, 32, 8),
    (5, 2, 7, 3),            # an odd width: one column passes through, element-wise moves
    (9, 1, 2, 1),            # a single pair
    (2, 3, 1024, 512),       # the widest rotation
    (33, 7, 200, 64),
]


@pytest.mark.parametrize("T,H,D,n", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
def test_rope(T, H, D, n, dtype, interleaved, inverse):
    x, pos = draw(T, H, D, dtype, seed=T + D)
    freq = ops.rope_frequencies(2 * n, device="cuda")
    out = ops.mla_rope(x, pos, freq, interleaved=interleaved, magnitude=1.25, inverse=inverse)
    check(x, pos, freq, out, interleaved, 1.25, inverse)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_far_positions(interleaved, scaling):
    x, pos = draw(64, 4, 64, torch.float32, seed=3)
    pos = pos + 2 ** 40 * (pos % 2) + 10 ** 6
    freq = ops.rope_frequencies(64, scaling=scaling, factor=40.0, device="cuda")
    # fp64 turns: 2^40 * 2^-53 of a turn, times 2 pi and a few roundings
    out = ops.mla_rope(x, pos, freq, interleaved=interleaved)
    ref, size = rotated(x, pos, freq, interleaved, 1.0, False)
    assert ((out.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + (5e-7 + 4e-3) * size).all()
    near = pos < 2 ** 30
    assert ((out.double() - ref).abs()[near] <= 2.0 ** -24 * ref.abs()[near] + 6e-7 * size[near]).all()


@pytest.mark.parametrize("pos_type", [torch.int32, torch.int64])
def test_strided_views_in_place_and_position_types(pos_type):
    # the rope columns of a [T, H, 192] projection, and the same rows with an odd offset
    x, pos = draw(37, 16, 200, torch.bfloat16, seed=9)
    pos = pos.to(pos_type)
    freq = ops.rope_frequencies(64, device="cuda")
    for lo in (128, 136, 131):
        view = x[..., lo:lo + 64]
        out = ops.mla_rope(view, pos, freq)
        check(view, pos, freq, out)
        kept = x.clone()
        place = kept[..., lo:lo + 64]
        assert ops.mla_rope(place, pos, freq, out=place) is place
        assert torch.equal(place, out)
        rest = torch.ones(200, dtype=torch.bool, device="cuda")
        rest[lo:lo + 64] = False
        assert torch.equal(kept[..., rest], x[..., rest])
    # head-major storage, and heads broadcast from one row
    y = x[..., :64].transpose(0, 1).contiguous().transpose(0, 1)
    check(y, pos, freq, ops.mla_rope(y, pos, freq))
    z = x[:, :1, :64].expand(-1, 8, -1)
    check(z, pos, freq, ops.mla_rope(z, pos, freq))


def test_inverse_is_the_gradient_and_undoes_the_rotation():
    x, pos = draw(11, 3, 64, torch.float32, seed=4)
    freq = ops.rope_frequencies(64, device="cuda")
    g = torch.randn_like(x)
    m = 1.5
    # <rope(x), g> = <x, rope^T(g)>: in fp64 from fp32 results, each off by 5e-7 of its terms
    left = (ops.mla_rope(x, pos, freq, magnitude=m).double() * g.double()).sum()
    right = (x.double() * ops.mla_rope(g, pos, freq, magnitude=m, inverse=True).double()).sum()
    terms = 2 * m * (x.abs().double().sum() * g.abs().max())
    assert abs(left - right) <= 1e-6 * terms
    # against differences of the formula: the map is linear, so a difference quotient is exact
    grad = ops.mla_rope(g, pos, freq, magnitude=m, inverse=True).double()
    for k in (0, 1, 40, 63):
        e = torch.zeros_like(x)
        e[2, 1, k] = 1.0
        step = (rotated(x + e, pos, freq, True, m, False)[0] - rotated(x, pos, freq, True, m, False)[0])
        # x + e is rounded to fp32: 2^-23 of values up to 5
        assert abs((step * g.double()).sum() - grad[2, 1, k]) <= 1e-5
    back = ops.mla_rope(ops.mla_rope(x, pos, freq), pos, freq, inverse=True)
    assert ((back - x).abs() <= 2e-6 * (x.abs().amax(-1, keepdim=True) * 2)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
def test_gradient_is_recorded(dtype, interleaved, inverse):
    """Through autograd: the gradient of sum(w * mla_rope(x)) is w turned the other way (the
    formula's, within check's tolerance), also of gradients that arrive as expanded views and into
    an x shared by all heads, whose gradient is the heads' sum."""
    x, pos = draw(37, 6, 96, dtype, seed=3)
    w, _ = draw(37, 6, 96, dtype, seed=4)
    freq = ops.rope_frequencies(64, device="cuda")
    how = (interleaved, 1.25, inverse)
    leaf = x.clone().requires_grad_()
    y = ops.mla_rope(leaf, pos, freq, *how)
    assert y.requires_grad and torch.equal(y.detach(), ops.mla_rope(x, pos, freq, *how))
    y.backward(w)
    check(w, pos, freq, leaf.grad, interleaved, 1.25, not inverse)

    leaf = x.clone().requires_grad_()
    ops.mla_rope(leaf, pos, freq, *how).sum().backward()      # the gradient arrives with strides 0
    check(torch.ones_like(x), pos, freq, leaf.grad, interleaved, 1.25, not inverse)

    if dtype == torch.float32:
        one = x[:, :1].clone().requires_grad_()
        ops.mla_rope(one.expand(-1, 6, -1), pos, freq, *how).backward(w)
        ref, size = rotated(w, pos, freq, interleaved, 1.25, not inverse)
        # each head's gradient as in check, and five sums of fp32 (2^-24 of the heads' sum of sizes each)
        each = 2.0 ** -24 * ref.abs() + 5e-7 * 1.25 * size
        tol = each.sum(1, keepdim=True) + 5 * 2.0 ** -24 * (ref.abs() + each).sum(1, keepdim=True)
        assert ((one.grad.double() - ref.sum(1, keepdim=True)).abs() <= tol).all()

    with torch.no_grad():
        assert not ops.mla_rope(leaf, pos, freq, *how).requires_grad


def test_second_gradient_and_captured_backward():
    """The gradient is linear in its input and recorded itself: turning forth, back and forth again.
    A forward and backward pass captured in a graph gives what the eager one gives."""
    x, pos = draw(9, 3, 64, torch.float32, seed=5)
    w, _ = draw(9, 3, 64, torch.float32, seed=6)
    freq = ops.rope_frequencies(64, device="cuda")
    leaf, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    (gx,) = torch.autograd.grad(ops.mla_rope(leaf, pos, freq), leaf, wl, create_graph=True)
    (gw,) = torch.autograd.grad(gx, wl, x)
    assert torch.equal(gw, ops.mla_rope(x, pos, freq))
    eager = gx.detach().clone()
    del leaf, gx, gw

    static = x.clone().requires_grad_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.autograd.grad(ops.mla_rope(static, pos, freq), static, w)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (grad,) = torch.autograd.grad(ops.mla_rope(static, pos, freq), static, w)
    grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad, eager)


def test_non_finite_values_stay_in_their_pair():
    x, pos = draw(4, 2, 64, torch.float32, seed=6)
    clean = ops.mla_rope(x, pos, ops.rope_frequencies(64, device="cuda"))
    x[1, 1, 10] = float("nan")
    x[2, 0, 31] = float("inf")
    out = ops.mla_rope(x, pos, ops.rope_frequencies(64, device="cuda"))
    same = torch.ones_like(x, dtype=torch.bool)
    same[1, 1, 10:12] = False
    same[2, 0, 30:32] = False
    assert torch.equal(out[same], clean[same]) and not torch.isfinite(out[~same]).any()


def test_empty_streams_and_graphs():
    freq = ops.rope_frequencies(64, device="cuda")
    x, pos = draw(0, 4, 64, torch.bfloat16)
    assert ops.mla_rope(x, pos, freq).shape == (0, 4, 64)
    x, pos = draw(50, 16, 64, torch.bfloat16, seed=1)
    want = ops.mla_rope(x, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.mla_rope(x, pos, freq)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.mla_rope(x, pos, freq, out=out)
        ops.mla_rope(out, pos, freq, out=out, inverse=True)
        ops.mla_rope(x, pos, freq, out=out)
    x2, pos2 = draw(50, 16, 64, torch.bfloat16, seed=2)
    x.copy_(x2)
    pos.copy_(pos2)
    graph.replay()
    torch.cuda.synchronize()
    check(x2, pos2, freq, out)


def test_many_tokens_and_heads():
    # above 2^31 bytes: 64-bit offsets
    x = torch.zeros(70001, 128, 192, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.tensor([0, 1, 35000, 69999, 70000], device="cuda")
    x[rows] = torch.randn(5, 128, 192, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(70001, device="cuda")
    freq = ops.rope_frequencies(64, device="cuda")
    out = ops.mla_rope(x, pos, freq, interleaved=False)
    check(x[rows], pos[rows], freq, out[rows], False)
    assert int((out != 0).any(-1).any(-1).sum()) == 5


def test_frequencies_are_the_formulas():
    f = ops.rope_frequencies(64)
    assert f.dtype == torch.float64 and math.isclose(f[5], 10000.0 ** (-10 / 64))
    assert torch.allclose(ops.rope_frequencies(64, scaling="linear", factor=8.0), f / 8, rtol=1e-14)
    ntk = ops.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 8, rel_tol=1e-12)
    yarn = ops.rope_frequencies(64, scaling="yarn", factor=40.0)
    assert math.isclose(yarn[0], f[0]) and math.isclose(yarn[-1], f[-1] / 40) and (yarn <= f).all() and (yarn >= f / 40 * (1 - 1e-12)).all()


@pytest.mark.parametrize("n", [256, 257, 300, 511, 512])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_wide_rotations_element_by_element(n, dtype, interleaved):
    """Rows that cannot be moved 16 bytes at a time: an odd width, an odd row stride and an odd offset;
    into an output that held NaN, in place and as the gradient."""
    freq = ops.rope_frequencies(2 * n, device="cuda")
    how = dict(interleaved=interleaved, magnitude=1.25)
    g = torch.Generator(device="cuda").manual_seed(n)
    odd_width, pos = draw(3, 2, 2 * n + 3, dtype, seed=n)
    odd_stride = torch.randn(3, 2, 2 * n + 1, generator=g, device="cuda").to(dtype)[..., :2 * n]
    odd_offset = torch.randn(3, 2, 2 * n + 8, generator=g, device="cuda").to(dtype)[..., 1:1 + 2 * n]
    for x in (odd_width, odd_stride, odd_offset):
        out = torch.full_like(x, float("nan"))
        ops.mla_rope(x, pos, freq, out=out, **how)
        check(x, pos, freq, out, **how)
        check(x, pos, freq, ops.mla_rope(x, pos, freq, **how), **how)
        kept = torch.full((3, 2, 2 * n + 9), 7.0, dtype=dtype, device="cuda")
        place = kept[..., 1:1 + x.shape[-1]]
        place.copy_(x)
        ops.mla_rope(place, pos, freq, out=place, **how)
        assert torch.equal(place, out)
        assert (kept[..., :1] == 7).all() and (kept[..., 1 + x.shape[-1]:] == 7).all()
        leaf = x.clone().requires_grad_()
        w = torch.empty(3, 2, 2 * n + 9, dtype=dtype, device="cuda")[..., 1:1 + x.shape[-1]].copy_(x.flip(0))
        ops.mla_rope(leaf, pos, freq, **how).backward(w)
        check(w, pos, freq, leaf.grad, inverse=True, **how)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
def test_tangent_is_carried(interleaved, inverse):
    """Forward mode: the map is linear, so the tangent is turned like x; also beside a gradient."""
    import torch.autograd.forward_ad as fwd
    x, pos = draw(9, 3, 80, torch.float32, seed=5)
    t, _ = draw(9, 3, 80, torch.float32, seed=6)
    w, _ = draw(9, 3, 80, torch.float32, seed=7)
    freq = ops.rope_frequencies(64, device="cuda")
    how = (interleaved, 1.25, inverse)
    want, moved = ops.mla_rope(x, pos, freq, *how), ops.mla_rope(t, pos, freq, *how)
    for tangent in (t, t.transpose(0, 2).contiguous().transpose(0, 2)):     # a strided last dimension
        with fwd.dual_level():
            out = fwd.unpack_dual(ops.mla_rope(fwd.make_dual(x, tangent), pos, freq, *how))
            assert torch.equal(out.primal, want) and torch.equal(out.tangent, moved)
    with fwd.dual_level(), torch.no_grad():
        assert torch.equal(fwd.unpack_dual(ops.mla_rope(fwd.make_dual(x, t), pos, freq, *how)).tangent, moved)
    leaf = x.clone().requires_grad_()
    with fwd.dual_level():
        out = fwd.unpack_dual(ops.mla_rope(fwd.make_dual(leaf, t), pos, freq, *how))
        assert torch.equal(out.tangent, moved)
        (grad,) = torch.autograd.grad(out.primal, leaf, w)
    assert torch.equal(grad, ops.mla_rope(w, pos, freq, interleaved, 1.25, not inverse))
    # differences of the formula: the tangent is that of the 64-bit map at any step
    ref = rotated(t, pos, freq, *how)
    assert ((moved.double() - ref[0]).abs() <= 2.0 ** -24 * ref[0].abs() + 5e-7 * 1.25 * ref[1]).all()


def test_function_transforms_are_refused_by_torch():
    x, pos = draw(5, 4, 64, torch.float32, seed=1)
    turn = lambda v: ops.mla_rope(v, pos, ops.rope_frequencies(64, device="cuda"))
    for call in (lambda: torch.func.grad(lambda v: turn(v).sum())(x), lambda: torch.func.jvp(turn, (x,), (x,)),
                 lambda: torch.func.vmap(turn)(x[None])):
        with pytest.raises(RuntimeError):
            call()
