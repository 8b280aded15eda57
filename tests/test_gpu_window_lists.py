"""The backward's key windows and the windows that see them, at the ends of what a call may
name. Both the window attention and the differential one, against the float64 oracles.

Tolerance, for bfloat16: P and dS are rounded once each (2^-8 at most, 2^-8 / sqrt(3) on the
average) before sums of several products, the forward's output and the results once more: a few
independent errors of 2.3e-3, 1e-2 of the relative L2 norm. float32: scores are sums of d
products, off by at most s = (d + 4) 2^-23 max |q| |k| / sqrt(d), which moves P by 2 s of its
value and dS by as much of |P| (|dP| + |D|): 16 s."""
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
