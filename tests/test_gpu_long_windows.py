"""Windows longer than 32767 along an axis: offsets inside a window past 15 bits."""
import pytest
import torch

from tests.test_gpu_diff import Case, _rel

pytestmark = pytest.mark.gpu


def _plain_layer(c):
    from sparse_window_attention_b200.layer import BasaLayer

    g = c.geo
    return BasaLayer(c.B, c.heads, c.d, g.grid, g.window, g.pool, g.n_text, g.routed_k, c.dtype)


def _plain_step(c, layer, q, k, v, dout, kp=None, vp=None, route=None):
    """(out, dq, dk, dv) of window attention over the first maps."""
    from sparse_window_attention_b200 import binding as B

    q, k = (x[:, 0::2].contiguous() for x in (q, k))
    if kp is not None:
        layer.kp.copy_(kp[:, 0::2])
        layer.vp.copy_(vp)
    if route is not None:
        layer.route_idx.copy_(route)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    layer.attention_lse(q, k, v, out, lse, c.shift, B.BASA_KEYS_ALL)
    return (out, *layer.backward(q, k, v, out, lse, dout, c.shift))


def test_windows_longer_than_32767():
    """One window over a grid of 33024 tokens in a row: every token sees every token, as with
    one window over the same tokens in 129 rows of 256. The two forms cut the window into other
    tiles, so their sums have another order; each is within 1e-2 of the true one."""
    row = Case("row", "bf16", 1, 1, 128, (1, 1, 33024), (1, 1, 33024), (0, 0, 0))
    rect = Case("rect", "bf16", 1, 1, 128, (1, 129, 256), (1, 129, 256), (0, 0, 0))
    q, k, v, lam, w, dout, _ = row.inputs(25)
    steps = []
    for c in (row, rect):
        plain, layer = _plain_layer(c), c.layer()
        out, saved = layer.attention_train(q, k, v, lam, c.shift, w)
        steps.append((*_plain_step(c, plain, q, k, v, dout), out, *layer.backward(q, k, v, lam, c.shift, saved, dout, w)[:3]))
        assert plain.device_error() == 0 and layer.device_error() == 0
    names = ("out", "dq", "dk", "dv", "diff out", "diff dq", "diff dk", "diff dv")
    for rows in (slice(None), slice(32768, None)):
        for name, a, b in zip(names, *steps):
            a, b = a[:, :, rows], b[:, :, rows]
            assert a.isfinite().all() and _rel(a, b.double()) <= 2e-2, (name, _rel(a, b.double()))
    # rows past 32767 against the formula
    at = torch.arange(32760, 33024, 7, device="cuda")
    p = torch.softmax(q[0, 0, at].double() @ k[0, 0].double().T / row.d**0.5, -1)
    assert _rel(steps[0][0][0, 0, at], p @ v[0, 0].double()) <= 1e-2
