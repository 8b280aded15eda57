"""Pins of the differential-attention oracle (CPU): against the window oracle map by map,
and its gradients against central differences."""
import numpy as np
import pytest
import torch

from oracle import basa_oracle as O
from oracle import diff_oracle as D

GEO = O.Geometry(grid=(2, 4, 6), window=(1, 2, 3), shift=(1, 1, 2), pool=(2, 2, 3), n_text=3, routed_k=2)


def _inputs(seed=0, B=2, h=2, d=8):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
    rows = GEO.N + GEO.n_text
    q, k, v = t(B, 2 * h, GEO.N, d), t(B, 2 * h, rows, d), t(B, h, rows, d)
    route = torch.stack([torch.randperm(GEO.n_win - 1, generator=torch.Generator().manual_seed(i))[:2] for i in range(B * h * GEO.n_win)])
    route = route.view(B, h, GEO.n_win, 2)
    route = route + (route >= torch.arange(GEO.n_win)[:, None])
    return q, k, v, torch.tensor([0.3, 0.8]).double(), t(d), route


def test_maps_are_the_window_oracles():
    q, k, v, lam, w, route = _inputs()
    kp, vp = (torch.from_numpy(O.pool_kv(x.numpy(), x.numpy(), GEO)[0]) for x in (k, v))
    maps = [torch.from_numpy(O.basa_attention(q[:, m::2].numpy(), k[:, m::2].numpy(), v.numpy(), GEO,
                                              kp=kp[:, m::2].numpy(), vp=vp.numpy(), route_idx=route.numpy())) for m in (0, 1)]
    out, rows = D.forward(q, k, v, lam, None, GEO, kp, vp, route, sizes=True)
    a = maps[0] - lam[:, None, None] * maps[1]
    np.testing.assert_allclose(out, a, atol=1e-12)
    np.testing.assert_allclose(rows["o2"], maps[1], atol=1e-12)
    assert (rows["a1"] >= rows["o1"].abs() - 1e-12).all()
    normed = D.forward(q, k, v, lam, w, GEO, kp, vp, route, gain=0.7, eps=1e-3)
    np.testing.assert_allclose(normed, D.mix(*maps, lam, w, 0.7, 1e-3), atol=1e-12)
    np.testing.assert_allclose(normed, 0.7 * w * a * torch.rsqrt((a * a).mean(-1, keepdim=True) + 1e-3), atol=1e-12)


def test_text_rows_are_the_dense_oracle():
    q, k, v, lam, w, _ = _inputs()
    qt = q[:, :, : GEO.n_text].contiguous()
    o = [O.text_query_attention(qt[:, m::2].numpy(), k[:, m::2].numpy(), v.numpy(), GEO) for m in (0, 1)]
    np.testing.assert_allclose(D.text_forward(qt, k, v, lam, None), o[0] - lam.numpy()[:, None, None] * o[1], atol=1e-12)


@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(norm):
    q, k, v, lam, w, route = _inputs(1)
    w = w if norm else None
    dout = torch.from_numpy(np.random.default_rng(2).standard_normal((2, 2, GEO.N, 8)))

    def loss(q, k, v, lam, w):
        kp, vp = (torch.from_numpy(O.pool_kv(x.numpy(), x.numpy(), GEO)[0]) for x in (k, v))
        return float((D.forward(q, k, v, lam, w, GEO, kp, vp, route, 0.7, 1e-3) * dout).sum())

    kp, vp = (torch.from_numpy(O.pool_kv(x.numpy(), x.numpy(), GEO)[0]) for x in (k, v))
    grads = D.backward(q, k, v, lam, w, GEO, dout, kp, vp, route, 0.7, 1e-3)
    args, rng, step = [q, k, v, lam, w], np.random.default_rng(3), 1e-5
    for i, g in enumerate(grads):
        if g is None:
            assert i == 4 and not norm
            continue
        for _ in range(6):
            at = tuple(int(rng.integers(n)) for n in g.shape)
            moved = []
            for sign in (1, -1):
                x = args[i].clone()
                x[at] += sign * step
                moved.append(loss(*args[:i], x, *args[i + 1 :]))
            assert abs((moved[0] - moved[1]) / (2 * step) - float(g[at])) < 1e-7, (i, at)
