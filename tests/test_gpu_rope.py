"""Rotary positions on the GPU (basa_rope_fwd, basa_rope_bwd through GridRope) against the
float64 oracle.

Tolerances. The kernel works in float32 and rounds once, so an output is off by at most
half a step of its type (eps / 2 of its value) plus the float32 work, bounded by the sizes
of the terms that are added:
  forward  y = xa cos -/+ xb sin: the row's factor rsqrt(mean + eps) comes from a sum of d
           squares in chains of at most 2 VEC + 4 additions (16 + 4) and a 2-step rsqrt,
           under 2^-19 in all; two products with rounded cos and sin (2^-24 each), one
           addition: under 2^-18 (|xa| + |xb|).
  dx       r (g - xh mean(g xh)) with |g| <= |w| (|dya| + |dyb|): the mean is a sum of d
           products in the same chains; under 2^-17 r (|g| + |xh| mean|g xh|).
  dweight  a sum of M = B heads rows products g xh: each product under 2^-18 of
           |g||xh|, and a chain of at most (units of a thread) + (blocks / 32) + 64
           additions of 2^-24 each; both of sum |g||xh|.
"""
import numpy as np
import pytest
import torch

from oracle import rope_oracle as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


def _fwd_bound(x, pairs, weight, eps, dtype, y):
    xn = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    a, b = R.split_pairs(np.abs(xn), pairs)
    return _half_step(dtype) * np.abs(y) + (1 + _half_step(dtype)) * 2.0**-18 * R.join_pairs(a + b, a + b, pairs)


def _bwd_bound(x, pairs, dy, weight, eps, dtype, dx, chain):
    a, b = R.split_pairs(np.abs(dy), pairs)
    g = R.join_pairs(a + b, a + b, pairs)
    if weight is None:
        return _half_step(dtype) * np.abs(dx) + 2.0**-17 * g, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = np.abs(x * r)
    dw = (2.0**-18 + chain * 2.0**-24) * (g * xh).sum((0, 1, 2))
    gw = g * np.abs(weight)
    return _half_step(dtype) * np.abs(dx) + 2.0**-17 * r * (gw + xh * (gw * xh).mean(-1, keepdims=True)), dw


CASES = [
    # B, heads, d, grid, axes, text, text_pos, pairs, norm, dtype
    (1, 24, 128, (1, 16, 16), (16, 56, 56), 5, True, "adjacent", True, "bf16"),
    (2, 3, 128, (3, 5, 7), (44, 42, 42), 0, False, "adjacent", True, "bf16"),
    (2, 3, 128, (3, 5, 7), (44, 42, 42), 9, False, "halves", True, "bf16"),
    (1, 1, 128, (1, 1, 1), (2, 2, 2), 0, False, "adjacent", True, "bf16"),
    (3, 5, 64, (2, 9, 11), (10, 22, 30), 33, True, "halves", False, "bf16"),
    (1, 7, 64, (5, 19, 23), (16, 24, 22), 7, True, "adjacent", True, "bf16"),
    (2, 2, 64, (5, 19, 23), (16, 24, 22), 7, True, "halves", True, "f32"),
    (1, 3, 128, (1, 1, 37), (0, 0, 128), 1, True, "adjacent", False, "f32"),
    (1, 2, 128, (2, 3, 4), (0, 0, 0), 2, False, "halves", True, "f32"),
    (1, 2, 128, (67, 1, 1), (126, 0, 0), 0, False, "halves", True, "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[8]}-{c[2]}-{c[9]}-{c[7]}-{i}" for i, c in enumerate(CASES)])
def test_forward_and_gradients(case):
    """q, k, v of the grid and of the text from two token-major packed projections to
    head-major tensors and back."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    B, heads, d, grid, axes, text, with_pos, pairs, norm, dtype = case
    g = _rng(hash(case[:3]) % 1000)
    N = grid[0] * grid[1] * grid[2]
    pos = torch.randn(text, 3, generator=g, device="cuda") * 30 if with_pos else None
    eps = 1e-6
    rope = GridRope(d, grid, axes, batch=B, theta=100.0, pairs=pairs, n_text=text, text_pos=pos, dtype=dtype, eps=eps)
    ang = R.angles(R.positions(grid, text, None if pos is None else _np(pos)), axes, d, 100.0)
    qkv, tqkv = _randn(g, B, N, 3, heads, d, dtype=dtype), _randn(g, B, text, 3, heads, d, dtype=dtype)
    weights = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(DT[dtype]) if norm else None for _ in range(4)]
    k, v = (torch.full((B, heads, N + text, d), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    q, qt = torch.full_like(k[:, :, :N].contiguous(), float("nan")), torch.full_like(k[:, :, N:].contiguous(), float("nan"))
    head = lambda x, i: x[:, :, i].permute(0, 2, 1, 3)  # noqa: E731
    parts = [RopePart(head(qkv, 0), q, weights[0]), RopePart(head(qkv, 1), k[:, :, :N], weights[1]),
             RopePart(head(qkv, 2), v[:, :, :N], rotate=False),
             RopePart(head(tqkv, 0), qt, weights[2], N), RopePart(head(tqkv, 1), k[:, :, N:], weights[3], N),
             RopePart(head(tqkv, 2), v[:, :, N:], None, N, False)]
    rope.forward(parts)
    grads = [_randn(g, *p.x.shape, dtype=dtype) for p in parts]
    dqkv, dtqkv = torch.full_like(qkv, float("nan")), torch.full_like(tqkv, float("nan"))
    dx = [head(dqkv, i) for i in range(3)] + [head(dtqkv, i) for i in range(3)]
    dws = rope.backward(parts, grads, dx)
    again = [torch.empty_like(t) for t in dx]
    for a, b in zip(dws, rope.backward(parts, grads, again)):
        assert (a is None and b is None) or torch.equal(a, b)  # the same bits every run
    torch.cuda.synchronize()
    for i, (p, dy, out, dw) in enumerate(zip(parts, grads, dx, dws)):
        assert torch.equal(out, again[i])
        rows = slice(p.first_row, p.first_row + p.x.shape[2])
        x, a, w, dy = _np(p.x), ang[rows] if p.rotate else 0 * ang[rows], None if p.weight is None else _np(p.weight), _np(dy)
        ref = R.forward(x, a, pairs, w, eps)
        assert (np.abs(_np(p.y) - ref) <= _fwd_bound(x, pairs, w, eps, dtype, ref)).all(), f"part {i}"
        ref_dx, ref_dw = R.backward(x, a, pairs, dy, w, eps)
        bound, dw_bound = _bwd_bound(x, pairs, dy, w, eps, dtype, ref_dx, B * heads + N / 8 + 64)
        assert (np.abs(_np(out) - ref_dx) <= bound).all(), f"part {i}"
        assert (dw is None) == (ref_dw is None)
        if dw is not None:
            assert (np.abs(_np(dw) - ref_dw) <= dw_bound + _half_step(dtype) * np.abs(ref_dw)).all(), f"part {i}"
        if not p.rotate:
            assert torch.equal(p.y, p.x) and torch.equal(out, grads[i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_ranges_down_to_one_token(dtype):
    """A range of rows gives the bits of the same rows of the whole sequence, also across
    the end of the grid; rows outside it are left as they were."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(3)
    B, heads, d, grid, text = 2, 3, 128, (3, 5, 7), 6
    n = 105 + text
    rope = GridRope(d, grid, (44, 42, 42), batch=B, n_text=text, text_pos=torch.arange(18.0).view(6, 3), dtype=dtype)
    x, w = _randn(g, B, heads, n, d, dtype=dtype), _randn(g, d, dtype=dtype)
    whole = torch.empty_like(x)
    rope.forward([RopePart(x, whole, w)])
    for first, rows in ((0, 1), (104, 1), (105, 1), (n - 1, 1), (103, 5), (17, 33), (0, n)):
        y = torch.full_like(x, 7.0)
        rope.forward([RopePart(x[:, :, first : first + rows], y[:, :, first : first + rows], w, first)])
        assert torch.equal(y[:, :, first : first + rows], whole[:, :, first : first + rows]), (first, rows)
        y[:, :, first : first + rows] = 7.0
        assert (y == 7.0).all()


def test_shared_heads_broadcast_inputs_and_in_place():
    """Fewer key heads than query heads in one call; an input broadcast over heads and
    batch (its gradient per head, to be summed by the caller); x and dy overwritten."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(4)
    B, d, grid, eps = 2, 64, (1, 6, 9), 1e-6
    rope = GridRope(d, grid, (0, 32, 32), batch=B, pairs="halves", eps=eps)
    ang = R.angles(R.positions(grid), (0, 32, 32), d, 10000.0)
    w = _randn(g, d, dtype="bf16")
    q, k = _randn(g, B, 8, 54, d, dtype="bf16"), _randn(g, B, 2, 54, d, dtype="bf16")
    one = _randn(g, 1, 1, 54, d, dtype="bf16").expand(B, 3, 54, d)
    outs = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k, one)]
    q0 = q.clone()
    rope.forward([RopePart(q, q, w), RopePart(k, outs[1], w), RopePart(one, outs[2], w)])
    for x, y in ((q0, q), (k, outs[1]), (one, outs[2])):
        ref = R.forward(_np(x), ang, "halves", _np(w), eps)
        assert (np.abs(_np(y) - ref) <= _fwd_bound(_np(x), "halves", _np(w), eps, "bf16", ref)).all()
    dy1 = _randn(g, 1, 1, 54, d, dtype="bf16").expand(B, 8, 54, d)
    parts = [RopePart(q0, q, w), RopePart(k, outs[1], w)]
    dk = _randn(g, *k.shape, dtype="bf16")
    dk0, dq = dk.clone(), torch.empty_like(q)
    rope.backward(parts, [dy1, dk], [dq, dk])
    for x, dy, dx in ((q0, dy1, dq), (k, dk0, dk)):
        ref, _ = R.backward(_np(x), ang, "halves", _np(dy), _np(w), eps)
        bound, _ = _bwd_bound(_np(x), "halves", _np(dy), _np(w), eps, "bf16", ref, 0)
        assert (np.abs(_np(dx) - ref) <= bound).all()


def test_far_positions_and_steps():
    """Angles of 10^5 turns keep their fraction; positions may be interpolated."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(5)
    grid, axes = (2, 3, 70), (4, 4, 120)
    origin, step = (700001.0, -3.5, 123456.75), (1.0, 0.25, 0.3125)
    rope = GridRope(128, grid, axes, theta=1e6, origin=origin, step=step, dtype="f32")
    x = _randn(g, 1, 1, 420, 128, dtype="f32")
    y = torch.empty_like(x)
    rope.forward([RopePart(x, y)])
    ref = R.forward(_np(x), R.angles(R.positions(grid, origin=origin, step=step), axes, 128, 1e6), "adjacent")
    # numpy's own angles are products rounded at 2^-53 of up to 10^6: 2^-33 apart
    assert (np.abs(_np(y) - ref) <= _fwd_bound(_np(x), "adjacent", None, 0, "f32", ref) + 2.0**-32 * 8).all()


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(6)
    rope = GridRope(128, (1, 8, 8), (16, 56, 56))
    x, w = _randn(g, 1, 2, 64, 128, dtype="bf16"), _randn(g, 128, dtype="bf16")
    clean = torch.empty_like(x)
    rope.forward([RopePart(x, clean, w)])
    bad = x.clone()
    bad[0, 0, 3] = 0.0
    bad[0, 1, 5, 7] = float("nan")
    bad[0, 0, 9, 0] = float("inf")
    y = torch.empty_like(x)
    rope.forward([RopePart(bad, y, w)])
    assert (y[0, 0, 3] == 0).all() and y[0, 1, 5].isnan().all() and not y[0, 0, 9].isfinite().all()
    keep = torch.ones(1, 2, 64, dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = keep[0, 1, 5] = keep[0, 0, 9] = False
    assert torch.equal(y[keep], clean[keep])


def test_overflowing_rows_in_place_stay_out_of_other_gradients():
    """Rows in blocks that the sequence does not fill: a first row that overflows (and is
    overwritten in place) leaves the weight's gradient of a range without it as it was."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(9)
    rope = GridRope(128, (1, 5, 9), (16, 56, 56))
    x, w, dy = _randn(g, 1, 2, 45, 128, dtype="bf16"), _randn(g, 128, dtype="bf16"), _randn(g, 1, 2, 45, 128, dtype="bf16")
    sub = lambda t: t[:, :, 1:]  # noqa: E731
    want_dx = torch.empty_like(x)
    want, = rope.backward([RopePart(sub(x), sub(x), w, 1)], [sub(dy)], [sub(want_dx)])
    x[:, :, 0], dy[:, :, 0] = float("inf"), float("nan")
    got, = rope.backward([RopePart(sub(x), sub(x), w, 1)], [sub(dy)], [sub(dy)])
    assert torch.equal(got, want) and torch.equal(sub(dy), sub(want_dx))


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart, read and written."""
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(7)
    rope = GridRope(128, (1, 1, 3), (0, 0, 128))
    far = 2**30 + 128
    x = torch.empty(2 * far + 128, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 3, 128), (0, 0, far, 1))
    y = torch.empty(2 * far + 128, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 3, 128), (0, 0, far, 1))
    x.copy_(_randn(g, 1, 1, 3, 128, dtype="bf16"))
    near = torch.empty(1, 1, 3, 128, dtype=torch.bfloat16, device="cuda")
    rope.forward([RopePart(x, y)])
    rope.forward([RopePart(x.contiguous(), near)])
    assert torch.equal(y, near)


def test_other_stream_and_captured_graph():
    from sparse_window_attention_b200.rope import GridRope, RopePart

    g = _rng(8)
    rope = GridRope(128, (2, 8, 8), (44, 42, 42), batch=1)
    x, w = _randn(g, 1, 4, 128, 128, dtype="bf16"), _randn(g, 128, dtype="bf16")
    dy = _randn(g, 1, 4, 128, 128, dtype="bf16")

    def step(stream=None):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        rope.forward([RopePart(x, y, w)], stream)
        dw, = rope.backward([RopePart(x, y, w)], [dy], [dx], stream)
        return y, dx, dw

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(_randn(g, 1, 4, 128, 128, dtype="bf16"))
    graph.replay()
    ref = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
