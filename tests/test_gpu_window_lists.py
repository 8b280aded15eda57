"""The backward's key windows and the windows that see them, at the ends of what a call may
name: more windows than 16 bits count, and a window routed to more than once, also by itself
and by a route out of range, which stands for the own window. Both the window attention and
the differential one, against the float64 oracles.

Tolerance, for bfloat16: P and dS are rounded once each (2^-8 at most, 2^-8 / sqrt(3) on the
average) before sums of several products, the forward's output and the results once more: a few
independent errors of 2.3e-3, 1e-2 of the relative L2 norm. float32: scores are sums of d
products, off by at most s = (d + 4) 2^-23 max |q| |k| / sqrt(d), which moves P by 2 s of its
value and dS by as much of |P| (|dP| + |D|): 16 s."""
import numpy as np
import pytest
import torch

from oracle import diff_oracle as D
from tests.test_gpu_diff import Case, _f64, _rel, _score_error
from tests.test_gpu_long_windows import _plain_layer, _plain_step

pytestmark = pytest.mark.gpu


def _plain_reference(c, q, k, v, dout, kp=None, vp=None, route=None):
    """The same by the differential oracle: its first maps where lambda is 0."""
    zero = torch.zeros(c.heads, dtype=torch.float64, device="cuda")
    args = _f64(q, k, v)
    out = D.forward(*args, zero, None, c.geo, *_f64(kp, vp), route)
    dq, dk, dv, _, _ = D.backward(*args, zero, None, c.geo, dout.double(), *_f64(kp, vp), route)
    return out, dq[:, 0::2], dk[:, 0::2], dv


def _check(c, q, k, got, ref, names, rows=None):
    tol = 1e-2 if c.dtype == "bf16" else 16 * _score_error(q, k, c.d)
    for name, x, y in zip(names, got, ref):
        if rows is not None:
            x, y = x[:, :, rows], y[:, :, rows]
        assert x.isfinite().all(), name
        assert _rel(x, y) <= tol, (name, _rel(x, y), tol)


@pytest.mark.parametrize("shift", [(0, 0, 0), (0, 1, 1)], ids=["straight", "shifted"])
def test_more_windows_than_16_bits_count(shift):
    c = Case("many_windows", "bf16", 1, 1, 128, (1, 364, 364), (1, 2, 2), shift)
    assert c.geo.n_win == 33124
    q, k, v, lam, w, dout, _ = c.inputs(21)
    late = D.window_tokens(c.geo)[32768:].flatten().cuda()  # the tokens of the windows past 32767
    layer = _plain_layer(c)
    got, ref = _plain_step(c, layer, q, k, v, dout), _plain_reference(c, q, k, v, dout)
    assert layer.device_error() == 0
    for rows in (None, late):
        _check(c, q, k, got, ref, ("out", "dq", "dk", "dv"), rows)
    layer = c.layer()
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    got = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    assert layer.device_error() == 0
    ref = D.backward(*_f64(q, k, v, lam, w), c.geo, dout.double(), gain=c.gain, eps=c.eps)
    for rows in (None, late):
        _check(c, q, k, got[:3], ref[:3], ("dq", "dk", "dv"), rows)


def _repeats(c, kind):
    """Routes [B, heads, windows, routed]: every window's own id only; one other window
    throughout; or drawn with repetition from the own window and two others."""
    g, rng = c.geo, np.random.default_rng(5)
    w = np.arange(g.n_win)[:, None]
    if kind == "own":
        r = np.broadcast_to(w, (c.B, c.heads, g.n_win, g.routed_k))
    elif kind == "one":
        r = np.full((c.B, c.heads, g.n_win, g.routed_k), g.n_win // 2)
    else:
        r = (w + rng.integers(0, 3, (c.B, c.heads, g.n_win, g.routed_k))) % g.n_win
    return torch.from_numpy(np.ascontiguousarray(r, dtype=np.int32)).cuda()


REPEATED = [
    Case("odd2", "bf16", 2, 2, 128, (3, 12, 26), (3, 6, 13), (0, 3, 6), (3, 6, 13), 5, 2),
    Case("sixteen", "bf16", 1, 2, 128, (1, 20, 20), (1, 4, 4), (0, 1, 2), (0, 0, 0), 0, 16),
    Case("two_tiles", "bf16", 1, 1, 128, (1, 32, 48), (1, 16, 16), (0, 8, 8), (1, 8, 8), 130, 3, norm=False),
    Case("f32_three", "f32", 1, 2, 128, (1, 16, 16), (1, 8, 8), (0, 4, 4), (1, 4, 4), 9, 3),
]


@pytest.mark.parametrize("kind", ["own", "one", "mixed"])
@pytest.mark.parametrize("c", REPEATED, ids=[c.name for c in REPEATED])
def test_a_window_listed_more_than_once_counts_as_often(c, kind):
    q, k, v, lam, w, dout, _ = c.inputs(22)
    route = _repeats(c, kind)
    layer = c.layer()
    kp, vp = layer.pool_kv(k, v) if layer.has_pool else (None, None)
    keys = dict(kp=kp, vp=vp, route_idx=route)
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w, **keys)
    got = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    again = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    assert layer.device_error() == 0
    assert c.dtype == "f32" or all(torch.equal(a, b) for a, b in zip(got[:4], again[:4]))
    ref = D.backward(*_f64(q, k, v, lam, w), c.geo, dout.double(), *_f64(kp, vp), route, c.gain, c.eps)
    _check(c, q, k, got[:3], ref[:3], ("dq", "dk", "dv"))
    plain = _plain_layer(c)
    got = _plain_step(c, plain, q, k, v, dout, kp, vp, route)
    assert plain.device_error() == 0
    _check(c, q, k, got, _plain_reference(c, q, k, v, dout, kp, vp, route), ("out", "dq", "dk", "dv"))


@pytest.mark.parametrize("c", [REPEATED[0], REPEATED[3]], ids=["bf16", "f32"])
def test_gradients_with_routes_out_of_range_are_those_of_the_own_window(c):
    q, k, v, lam, w, dout, _ = c.inputs(23)
    route = _repeats(c, "mixed")
    fixed = route.clone()
    for at, bad in (((0, 0, 0, 0), -1), ((0, 1, 3, 1), c.geo.n_win), ((0, 1, 2, 0), 2**31 - 1), ((0, 1, 2, 1), -(2**31))):
        route[at], fixed[at] = bad, at[2]
    layer = c.layer()
    kp, vp = layer.pool_kv(k, v)
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w, kp=kp, vp=vp, route_idx=route)
    layer.dev_err.zero_()
    got = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    assert layer.device_error() == 8
    ref = D.backward(*_f64(q, k, v, lam, w), c.geo, dout.double(), *_f64(kp, vp), fixed, c.gain, c.eps)
    _check(c, q, k, got[:3], ref[:3], ("dq", "dk", "dv"))


def test_the_most_windows_with_routes():
    """4096 windows, most of which route to one of two: lists as long as they get."""
    c = Case("most", "bf16", 1, 1, 128, (1, 64, 128), (1, 1, 2), (0, 0, 1), (0, 0, 0), 0, 2, norm=False)
    assert c.geo.n_win == 4096
    q, k, v, lam, w, dout, _ = c.inputs(24)
    route = torch.zeros(1, 1, 4096, 2, dtype=torch.int32, device="cuda")
    route[..., 1] = 4095
    route[0, 0, ::3, 0] = 4095  # twice the last window
    layer = c.layer()
    _, saved = layer.attention_train(q, k, v, lam, c.shift, route_idx=route)
    got = layer.backward(q, k, v, lam, c.shift, saved, dout)
    assert layer.device_error() == 0
    ref = D.backward(*_f64(q, k, v, lam, None), c.geo, dout.double(), None, None, route)
    _check(c, q, k, got[:3], ref[:3], ("dq", "dk", "dv"))
