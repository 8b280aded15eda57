"""Differential attention on the GPU (basa_diff_* through BasaDiffLayer) against the
float64 oracle.

Tolerances. h = half a step of the element type (bf16 2^-8, float32 2^-24).
  maps     scores are float32 sums of d products: off by at most s = (d + 4) 2^-23 max
           (sum |q||k|) / sqrt(d), which moves a probability by 2 s of its value (numerator
           and sum); with bfloat16 it is also rounded once (h). A map's output is then off
           by E = (h' + 2 s + 2^-18) A, A its sum over |v| (h' = h or 0; 2^-18 for exp and
           the float32 sums).
  out      a = O1 - lambda O2 is off by E1 + |lambda| E2 =: Ea. Behind the norm, with
           a' = a + e, |e| <= Ea, r = (mean(a^2) + eps)^-1/2 and r' that of a':
             |a' r' - a r| <= |e| r' + |a| |r' - r|,  |r' - r| = r r' |1/r' - 1/r|
             <= r r' rms(Ea)                    (1/r is a norm of (a, sqrt(eps)): triangle)
             r' <= (max(0, rms(a) - rms(Ea))^2 + eps)^-1/2
           so y is off by gain |w| r'max (Ea + |a| r rms(Ea)), for errors of any size.
           Then h |out|.
  dq dk dv P and dS are rounded once each (h, uniformly distributed: h / sqrt(3) on the
           average) before sums of >= 64 products, and so are a, O2, g and the results:
           a few independent relative errors of h / sqrt(3) = 2.3e-3, each shrinking in
           the sums; 1e-2 in the relative L2 norm. dV is a difference of the maps' sums
           and is held to 1e-2 of the norm of the two parts before they are subtracted.
           float32: 16 s in place of 1e-2.
  dlambda  a sum of g O2 over M rows of d: each term off by about h |g| A2 / sqrt(3) at
           most, independently; 16 standard deviations (of g, O2 and a's errors together),
           and h of the value. dweight likewise with |G| r (A1 + |lambda| A2).
"""
import numpy as np
import pytest
import torch

from oracle import basa_oracle as O
from oracle import diff_oracle as D

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    def __init__(self, name, dtype, B, heads, d, grid, window, shift, pool=(0, 0, 0), n_text=0, routed_k=0, norm=True):
        self.name, self.dtype, self.B, self.heads, self.d, self.norm = name, dtype, B, heads, d, norm
        self.geo = O.Geometry(grid=grid, window=window, shift=shift, pool=pool, n_text=n_text, routed_k=routed_k)
        self.shift = shift
        self.gain, self.eps = 0.8, 1e-5

    def layer(self, **kw):
        from sparse_window_attention_b200.diff_layer import BasaDiffLayer

        g = self.geo
        return BasaDiffLayer(self.B, self.heads, self.d, g.grid, g.window, g.pool, g.n_text, g.routed_k, self.dtype,
                             gain=self.gain, eps=self.eps, **kw)

    def inputs(self, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        dt, rows = DT[self.dtype], self.geo.N + self.geo.n_text
        q, k = rnd(self.B, 2 * self.heads, self.geo.N, self.d).to(dt), rnd(self.B, 2 * self.heads, rows, self.d).to(dt)
        v = rnd(self.B, self.heads, rows, self.d).to(dt)
        lam = (0.2 + 0.6 * torch.rand(self.heads, generator=gen, device="cuda")).to(dt)
        w = (1 + 0.3 * rnd(self.d)).to(dt) if self.norm else None
        return q, k, v, lam, w, rnd(self.B, self.heads, self.geo.N, self.d).to(dt), gen


CASES = [
    Case("one_token", "bf16", 1, 1, 128, (1, 1, 1), (1, 1, 1), (0, 0, 0)),
    Case("one_token_text", "bf16", 2, 3, 128, (1, 1, 1), (1, 1, 1), (0, 0, 0), (1, 1, 1), 1, norm=False),
    Case("small", "bf16", 1, 2, 128, (1, 32, 32), (1, 8, 8), (0, 4, 4), (1, 4, 4)),
    Case("wrap3d", "bf16", 2, 3, 128, (4, 8, 12), (2, 4, 4), (1, 2, 3), (2, 4, 4), 77, 3),
    Case("odd_windows", "bf16", 2, 2, 128, (3, 12, 26), (3, 6, 13), (0, 3, 6), (3, 6, 13), 5, 2),
    Case("own_only", "bf16", 1, 3, 128, (1, 32, 32), (1, 16, 16), (0, 8, 8), norm=False),
    Case("two_tiles_odd", "bf16", 1, 1, 128, (1, 15, 34), (1, 15, 17), (0, 7, 16), (1, 5, 17), 1),
    Case("ragged", "bf16", 1, 2, 128, (1, 48, 48), (1, 16, 16), (0, 8, 8), (1, 4, 4), 200, 0, norm=False),
    Case("routes16", "bf16", 1, 1, 128, (1, 20, 20), (1, 4, 4), (0, 1, 2), (0, 0, 0), 0, 16),
    Case("many_key_tiles", "bf16", 1, 1, 128, (1, 62, 66), (1, 31, 66), (0, 5, 0), (1, 2, 2), 300, 1),
    Case("f32_d64", "f32", 2, 3, 64, (1, 16, 16), (1, 8, 8), (0, 4, 4), (1, 4, 4), 9, 1),
    Case("f32_d128", "f32", 1, 2, 128, (2, 6, 10), (1, 3, 5), (1, 2, 3), (2, 3, 5), 0, 2, norm=False),
    Case("f32_one_token", "f32", 1, 2, 64, (1, 1, 1), (1, 1, 1), (0, 0, 0)),
]


def _ids(cs):
    return [c.name for c in cs]


def _f64(*ts):
    return [None if t is None else t.double() for t in ts]


def _score_error(q, k, d):
    most = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max())  # >= any sum |q||k|
    return (d + 4) * 2.0**-23 * most / d**0.5


def _map_errors(c, q, k, a1, a2):
    h = torch.finfo(DT[c.dtype]).eps / 2
    rel = (h if c.dtype == "bf16" else 0.0) + 2 * _score_error(q, k, c.d) + 2.0**-18
    return rel * a1, rel * a2


def _assert_forward(c, out, ref, o1, o2, a1, a2, q, k, lam, w):
    h = torch.finfo(DT[c.dtype]).eps / 2
    lam = lam[:, None, None]
    e1, e2 = _map_errors(c, q, k, a1, a2)
    a, ea = o1 - lam * o2, e1 + lam.abs() * e2
    bound = ea + 2.0**-22 * (o1.abs() + (lam * o2).abs())
    if w is not None:
        rms, rms_e = (x.square().mean(-1, keepdim=True).sqrt() for x in (a, bound))
        r, r_max = (rms.square() + c.eps).rsqrt(), ((rms - rms_e).clamp(min=0).square() + c.eps).rsqrt()
        bound = c.gain * w.abs() * r_max * (bound + a.abs() * r * rms_e)
    bound = bound + h * (ref.abs() + bound) + 2.0**-21 * ref.abs()
    err = (out.double() - ref).abs()
    assert out.isfinite().all() and (err <= bound).all(), f"{c.name}: {float((err / bound).max()):.3f} of the bound"


def _keys(layer, q, k, v, shift):
    kp = vp = route = None
    if layer.has_pool:
        kp, vp = layer.pool_kv(k, v)
    if layer.routed_k:
        route = layer.route(q, k, shift)
    return kp, vp, route


@pytest.mark.parametrize("c", CASES, ids=_ids(CASES))
def test_forward(c):
    q, k, v, lam, w, _, _ = c.inputs()
    layer = c.layer()
    kp, vp, route = _keys(layer, q, k, v, c.shift)
    out = torch.full((c.B, c.heads, c.geo.N, c.d), float("nan"), dtype=DT[c.dtype], device="cuda")
    layer.attention(q, k, v, lam, c.shift, w, out=out)
    assert layer.device_error() == 0
    q64, k64, v64, lam64, w64, kp64, vp64 = _f64(q, k, v, lam, w, kp, vp)
    ref, rows = D.forward(q64, k64, v64, lam64, w64, c.geo, kp64, vp64, route, c.gain, c.eps, sizes=True)
    _assert_forward(c, out, ref, rows["o1"], rows["o2"], rows["a1"], rows["a2"], q, k, lam64, w64)
    assert torch.equal(out, layer.attention(q, k, v, lam, c.shift, w, kp=kp, vp=vp, route_idx=route))
    got, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    assert torch.equal(got, out)  # what a backward needs is stored beside the same result
    pre, second, lse = saved[:3]
    _, e2 = _map_errors(c, q, k, rows["a1"], rows["a2"])
    h = torch.finfo(DT[c.dtype]).eps / 2
    assert ((second.double() - rows["o2"]).abs() <= e2 + h * (rows["o2"].abs() + e2)).all()
    if w is not None:
        _assert_forward(c, pre, rows["o1"] - lam64[:, None, None] * rows["o2"], rows["o1"], rows["o2"], rows["a1"], rows["a2"],
                        q, k, lam64, None)
    else:
        assert pre is got


def _rel(a, b, size=None):
    return float((a.double() - b).norm() / (b.norm() if size is None else size))


@pytest.mark.parametrize("c", CASES, ids=_ids(CASES))
def test_gradients(c):
    q, k, v, lam, w, dout, _ = c.inputs(1)
    layer = c.layer()
    out, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    kp, vp, route = saved[3:]
    got = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    assert layer.device_error() == 0
    again = layer.backward(q, k, v, lam, c.shift, saved, dout, w, kp=kp, vp=vp, route_idx=route)
    for name, a, b in zip(("dq", "dk", "dv", "dlam", "dweight"), got, again):
        if c.dtype == "bf16" or name not in ("dk", "dv"):  # float32 adds dk, dv with atomics
            assert (a is None and b is None) or torch.equal(a, b), name
    q64, k64, v64, lam64, w64, kp64, vp64, do64 = _f64(q, k, v, lam, w, kp, vp, dout)
    args = (c.geo, do64, kp64, vp64, route, c.gain, c.eps)
    ref = D.backward(q64, k64, v64, lam64, w64, *args)
    _, rows = D.forward(q64, k64, v64, lam64, w64, c.geo, kp64, vp64, route, c.gain, c.eps, sizes=True)
    # g, the gradient behind the norm, and the maps' parts of dV
    a = rows["o1"] - lam64[:, None, None] * rows["o2"]
    g, weight_terms = do64, None
    if w is not None:
        r = (a.square().mean(-1, keepdim=True) + c.eps).rsqrt()
        G, xh = c.gain * do64, a * r
        weight_terms = G.abs() * r * (rows["a1"] + lam64[:, None, None].abs() * rows["a2"])
        g = r * (G * w64 - xh * (G * w64 * xh).mean(-1, keepdim=True))
    zero = torch.zeros_like(lam64)
    part1 = D.backward(q64, k64, v64, zero, None, c.geo, g, kp64, vp64, route)[2]
    part2 = part1 - D.backward(q64, k64, v64, zero + lam64, None, c.geo, g, kp64, vp64, route)[2]
    tol = 1e-2 if c.dtype == "bf16" else 16 * _score_error(q, k, c.d)
    for name, x, y in zip(("dq", "dk"), got, ref):
        assert x.isfinite().all()
        # one key: the scores have no gradient, and what is left is the error of D against dout V^T
        floor = tol * float(g.norm()) * float(v64.norm(dim=-1).max()) if c.geo.N == 1 else 0.0
        assert _rel(x, y, float(y.norm()) + floor) <= tol, (name, _rel(x, y))
    assert got[2].isfinite().all()
    dv_error = _rel(got[2], ref[2], float((part1.square() + part2.square()).sum().sqrt()))
    assert dv_error <= tol, ("dv", dv_error)
    h = torch.finfo(DT[c.dtype]).eps / 2
    unit = (h if c.dtype == "bf16" else 2 * _score_error(q, k, c.d) + 2.0**-18) / 3**0.5
    size = g.abs() * (rows["a2"] + (rows["a1"] + lam64[:, None, None] * rows["a2"]))
    bound = 16 * unit * size.square().sum((0, 2, 3)).sqrt() + (h + 2.0**-20) * ref[3].abs()
    if c.dtype == "f32":  # not independent: the worst case
        bound = bound + 4 * unit * size.sum((0, 2, 3))
    assert ((got[3].double() - ref[3]).abs() <= bound).all(), ("dlam", got[3], ref[3], bound)
    assert (got[4] is None) == (w is None)
    if w is not None:
        bound = 16 * unit * weight_terms.square().sum((0, 1, 2)).sqrt() + (h + 2.0**-20) * ref[4].abs()
        if c.dtype == "f32":
            bound = bound + 4 * unit * weight_terms.sum((0, 1, 2))
        assert ((got[4].double() - ref[4]).abs() <= bound).all(), "dweight"


TEXT = [
    Case("text1", "bf16", 1, 3, 128, (2, 16, 24), (1, 8, 8), (1, 4, 4), n_text=1),
    Case("text77", "bf16", 2, 2, 128, (1, 48, 48), (1, 16, 16), (0, 8, 8), (1, 4, 4), 77, norm=False),
    Case("text300", "bf16", 1, 12, 128, (1, 40, 40), (1, 8, 8), (0, 4, 4), n_text=300),
    Case("text_many_heads", "bf16", 2, 40, 128, (1, 16, 16), (1, 8, 8), (0, 4, 4), n_text=130),
    Case("text_f32", "f32", 2, 3, 64, (1, 24, 16), (1, 8, 8), (0, 5, 3), (1, 4, 4), 33, 1),
    Case("text_f32_d128", "f32", 1, 1, 128, (1, 8, 8), (1, 8, 8), (0, 0, 0), n_text=3, norm=False),
]


@pytest.mark.parametrize("c", TEXT, ids=_ids(TEXT))
def test_text_rows(c):
    _, k, v, lam, w, _, gen = c.inputs(2)
    qt = torch.randn(c.B, 2 * c.heads, c.geo.n_text, c.d, generator=gen, device="cuda").to(DT[c.dtype])
    layer = c.layer()
    out = layer.text_attention(qt, k, v, lam, w)
    assert layer.device_error() == 0 and torch.equal(out, layer.text_attention(qt, k, v, lam, w))
    q64, k64, v64, lam64, w64 = _f64(qt, k, v, lam, w)
    p = torch.softmax(q64 @ k64.transpose(-1, -2) / c.d**0.5, -1)
    o1, o2 = p[:, 0::2] @ v64, p[:, 1::2] @ v64
    a1, a2 = D.text_forward(q64, k64, v64, lam64, None, magnitudes=True)
    ref = D.text_forward(q64, k64, v64, lam64, w64, c.gain, c.eps)
    _assert_forward(c, out, ref, o1, o2, a1, a2, qt, k, lam64, w64)


def test_gradient_of_lambda_where_the_maps_are_nearly_alike():
    """Behind the norm only the part of O2 that is orthogonal to a counts. Each of its
    channels is off by the probabilities' roundings (h / sqrt(3) of sqrt(sum P^2 v^2),
    independent, of both maps over 1 - lambda) and by h / sqrt(3) of itself; 16 standard
    deviations of the sum of g O2."""
    c = Case("alike", "bf16", 1, 3, 128, (1, 32, 32), (1, 16, 16), (0, 8, 8))
    q, k, v, lam, w, dout, gen = c.inputs(3)
    rnd = lambda x, s: (x[:, 0::2] + s * torch.randn(x[:, 0::2].shape, generator=gen, device="cuda")).to(x.dtype)  # noqa: E731
    q[:, 1::2], k[:, 1::2] = rnd(q, 0.05), rnd(k, 0.05)
    v += 1  # a common part
    layer = c.layer()
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    dlam = layer.backward(q, k, v, lam, c.shift, saved, dout, w)[3]
    q64, k64, v64, lam64, w64, do64 = _f64(q, k, v, lam, w, dout)
    ref = D.backward(q64, k64, v64, lam64, w64, c.geo, do64, gain=c.gain, eps=c.eps)[3]
    _, rows = D.forward(q64, k64, v64, lam64, w64, c.geo, sizes=True)
    ids = D.window_tokens(c.geo).cuda()
    quad = torch.zeros_like(rows["o1"])
    for b in range(c.B):
        for j in range(c.heads):
            for m in (0, 1):
                p = torch.softmax(q64[b, 2 * j + m][ids] @ k64[b, 2 * j + m][ids].transpose(1, 2) / c.d**0.5, -1)
                quad[b, j, ids.flatten()] += (p.square() @ v64[b, j][ids].square()).sqrt().flatten(0, 1)
    a = rows["o1"] - lam64[:, None, None] * rows["o2"]
    r = (a.square().mean(-1, keepdim=True) + c.eps).rsqrt()
    xh, G = a * r, c.gain * do64 * w64
    g = r * (G - xh * (G * xh).mean(-1, keepdim=True))
    rest = rows["o2"] - (rows["o2"] * a).sum(-1, keepdim=True) / a.square().sum(-1, keepdim=True) * a
    size = g.abs() * (quad / (1 - lam64)[:, None, None] + rest.abs())
    bound = 16 * 2.0**-8 / 3**0.5 * size.square().sum((0, 2, 3)).sqrt() + 2.0**-8 * ref.abs()
    assert ((dlam.double() - ref).abs() <= bound).all(), (dlam, ref, bound)


def test_pooled_and_routed_keys():
    """The layer's own pooled keys and routes are those of the window layer's operators."""
    from sparse_window_attention_b200.layer import BasaLayer

    c = CASES[3]
    q, k, v, _, _, _, _ = c.inputs()
    kp, vp, route = _keys(c.layer(), q, k, v, c.shift)
    g = c.geo
    other = BasaLayer(c.B, 2 * c.heads, c.d, g.grid, g.window, g.pool, g.n_text, g.routed_k, c.dtype)
    vv = v.repeat_interleave(2, 1)
    other.pool_kv(k, vv)
    other.route(q, k, c.shift)
    assert torch.equal(kp, other.kp) and torch.equal(vp, other.vp[:, 0::2]) and torch.equal(route, other.route_idx[:, 0::2])


@pytest.mark.parametrize("c", [CASES[3], CASES[7]], ids=["wrap3d", "ragged"])
def test_without_the_second_map_it_is_window_attention(c):
    """lambda 0 gives the first maps' window attention, bit for bit; equal maps with
    lambda 1 cancel to zero rows, which stay zero behind the norm."""
    from sparse_window_attention_b200.layer import BasaLayer

    q, k, v, lam, _, _, _ = c.inputs()
    g, layer = c.geo, c.layer()
    out = layer.attention(q, k, v, torch.zeros_like(lam), c.shift)
    kp, vp, route = _keys(layer, q, k, v, c.shift)
    plain = BasaLayer(c.B, c.heads, c.d, g.grid, g.window, g.pool, g.n_text, g.routed_k, c.dtype)
    first = lambda x: x[:, 0::2].contiguous()  # noqa: E731
    want = torch.empty_like(out)
    plain.attention(first(q), first(k), v, want, c.shift, kp=first(kp), vp=vp, route_idx=route)
    assert torch.equal(out, want)
    twice = lambda x: first(x).repeat_interleave(2, 1)  # noqa: E731
    w = torch.ones(c.d, dtype=DT[c.dtype], device="cuda")
    out, saved = layer.attention_train(twice(q), twice(k), v, torch.ones_like(lam), c.shift, w, kp=twice(kp), vp=vp,
                                       route_idx=route)
    assert (out == 0).all()
    grads = layer.backward(twice(q), twice(k), v, torch.ones_like(lam), c.shift, saved, torch.ones_like(out), w)
    assert all(x.isfinite().all() for x in grads) and (grads[4] == 0).all()


def test_nan_stays_in_its_head_and_window():
    c = CASES[5]
    q, k, v, lam, _, _, _ = c.inputs()
    clean = c.layer().attention(q, k, v, lam, c.shift)
    q[0, 3, 37], k[0, 0, 500, 5] = float("nan"), float("inf")
    out = c.layer().attention(q, k, v, lam, c.shift)
    ids = D.window_tokens(c.geo)
    hit = torch.zeros(c.B, c.heads, c.geo.N, dtype=torch.bool)
    hit[0, 1, 37] = True
    hit[0, 0, ids[(ids == 500).any(1)][0]] = True
    assert out[0, 1, 37].isnan().all()
    assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()])


def test_nan_and_infinity_leave_other_heads_alone():
    """Windows whose tiles have rows that no load writes, more of them than the GPU runs at
    once: nothing that a bad head leaves behind reaches another one."""
    c = Case("bad_heads", "bf16", 2, 24, 128, (3, 12, 26), (3, 6, 13), (0, 3, 6), (3, 6, 13), 5, 2)
    q, k, v, lam, w, dout, _ = c.inputs(9)
    layer = c.layer()
    kp, vp, route = _keys(layer, q, k, v, c.shift)

    def step():
        out, saved = layer.attention_train(q, k, v, lam, c.shift, w, kp=kp, vp=vp, route_idx=route)
        return (out, *layer.backward(q, k, v, lam, c.shift, saved, dout, w)[:4])

    clean = step()
    for b, h in ((0, 5), (1, 20)):
        q[b, 2 * h, ::7], k[b, 2 * h + 1, ::5] = float("nan"), float("inf")
        v[b, h, ::3], dout[b, h, ::11], vp[b, h] = float("nan"), float("-inf"), float("nan")
    bad = step()
    assert layer.device_error() == 0
    heads = torch.ones(2, 24, dtype=torch.bool, device="cuda")
    heads[0, 5] = heads[1, 20] = False
    maps = heads.repeat_interleave(2, 1)
    for name, x, y, keep in zip(("out", "dq", "dk", "dv"), bad, clean, (heads, maps, maps, heads)):
        assert torch.equal(x[keep], y[keep]), name
    keep = heads.all(0)
    assert torch.equal(bad[4][keep], clean[4][keep]) and bad[4][~keep].isnan().all()


def test_out_of_range_route_is_reported():
    c = CASES[4]
    q, k, v, lam, w, dout, _ = c.inputs()
    layer = c.layer()
    kp, vp, route = _keys(layer, q, k, v, c.shift)
    own = route.clone()
    own[1, 0, 3, 1] = 3
    want = layer.attention(q, k, v, lam, c.shift, w, kp=kp, vp=vp, route_idx=own)
    for bad in (-1, c.geo.n_win, 2**31 - 1):
        route[1, 0, 3, 1] = bad
        out, saved = layer.attention_train(q, k, v, lam, c.shift, w, kp=kp, vp=vp, route_idx=route)
        assert torch.equal(out, want)  # the own window in its place: nothing is read out of range
        assert layer.device_error() == 8
        layer.dev_err.zero_()
        layer.backward(q, k, v, lam, c.shift, saved, dout, w)
        assert layer.device_error() == 8
        layer.dev_err.zero_()


def test_bounded_waits_expire_and_the_context_survives():
    from sparse_window_attention_b200 import binding as B

    c = Case("timeout", "bf16", 1, 2, 128, (1, 32, 32), (1, 16, 16), (0, 8, 8), (1, 8, 8), 256)
    q, k, v, lam, w, dout, _ = c.inputs()
    layer = c.layer()
    want, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    grads = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    skip = dict(flags=B.BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD, wait_timeout_us=20000)
    out = torch.zeros_like(want)
    layer.attention(q, k, v, lam, c.shift, w, out=out, **skip)
    assert layer.device_error() & 7 and not layer.device_error() & ~7
    assert not out.any()
    layer.dev_err.zero_()
    layer.backward(q, k, v, lam, c.shift, saved, dout, w, **skip)
    assert layer.device_error() & 7 and not layer.device_error() & ~7
    layer.dev_err.zero_()
    assert torch.equal(want, layer.attention(q, k, v, lam, c.shift, w))
    assert all(torch.equal(a, b) for a, b in zip(grads, layer.backward(q, k, v, lam, c.shift, saved, dout, w)))
    assert layer.device_error() == 0


def test_other_streams_and_captured_graphs():
    """A training step on another stream, two captured graphs of one layer replayed at
    once on two streams, and new inputs in a replay."""
    c = CASES[3]
    q, k, v, lam, w, dout, _ = c.inputs(4)
    layer = c.layer()

    def step(stream=None):
        out, saved = layer.attention_train(q, k, v, lam, c.shift, w, stream=stream)
        return (out, *layer.backward(q, k, v, lam, c.shift, saved, dout, w, stream=stream))

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    q2, k2, v2, _, _, _, _ = c.inputs(5)
    for t, new in ((q, q2), (k, k2), (v, v2)):
        t.copy_(new)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    ref = step()
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_offsets_past_32_bits():
    """More than 2^31 elements of q, k and their gradients: the last heads give the bits
    that they give by themselves (no pooled or text keys, whose sums are split by size)."""
    many = Case("many", "bf16", 1, 520, 128, (1, 128, 128), (1, 16, 16), (0, 8, 8))
    few = Case("few", "bf16", 1, 2, 128, (1, 128, 128), (1, 16, 16), (0, 8, 8))
    q1, k1, v1, lam1, w, dout1, _ = few.inputs(6)
    new = lambda h: torch.zeros(1, h, many.geo.N, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, v, dout, lam = new(1040), new(1040), new(520), new(520), torch.zeros(520, dtype=torch.bfloat16, device="cuda")
    for big, small in ((q, q1), (k, k1), (v, v1), (dout, dout1)):
        big[:, -small.shape[1] :] = small
    lam[-2:] = lam1
    results = []
    for c, args, g in ((few, (q1, k1, v1, lam1), dout1), (many, (q, k, v, lam), dout)):
        layer = c.layer()
        out, saved = layer.attention_train(*args, c.shift, w)
        dq, dk, dv, dlam, _ = layer.backward(*args, c.shift, saved, g, w)
        assert layer.device_error() == 0
        results.append((out[:, -2:], dq[:, -4:], dk[:, -4:], dv[:, -2:], dlam[-2:]))
        del out, saved, dq, dk, dv
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("c", [CASES[2], CASES[3], CASES[-2]], ids=["small", "wrap3d", "f32"])
def test_tensors_on_16_byte_boundaries(c):
    """Every tensor 16 bytes past a 32-byte boundary: the same bits."""

    def moved(*shape, dtype):
        n, pad = int(np.prod(shape)), 16 // torch.empty((), dtype=dtype).element_size()
        t = torch.empty(n + pad, dtype=dtype, device="cuda")[pad:].view(shape)
        assert t.data_ptr() % 32 == 16
        return t

    q, k, v, lam, w, dout, _ = c.inputs(7)

    def step(args, layer):
        out, saved = layer.attention_train(*args[:4], c.shift, args[4])
        return (out, *layer.backward(*args[:4], c.shift, saved, args[5], args[4]))

    args = [q, k, v, lam, w, dout]
    ref = step(args, c.layer())
    args = [None if t is None else moved(*t.shape, dtype=t.dtype).copy_(t) for t in args]
    layer = c.layer()
    plain = layer._new
    layer._new = lambda *shape, dtype=None: plain(*shape, dtype=dtype) if dtype is torch.uint8 else moved(*shape, dtype=dtype or layer.dtype)
    got = step(args, layer)
    assert layer.device_error() == 0
    for name, a, b in zip(("out", "dq", "dk", "dv", "dlam", "dweight"), got, ref):
        if c.dtype == "bf16" or name not in ("dk", "dv"):  # float32 adds dk, dv with atomics
            assert (a is None and b is None) or torch.equal(a, b), name


def test_refused_tensors():
    c = CASES[2]
    q, k, v, lam, w, dout, _ = c.inputs()
    layer = c.layer()
    with pytest.raises(ValueError):
        layer.attention(q[:, :2], k, v, lam, c.shift, w)
    with pytest.raises(ValueError):
        layer.attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, lam, c.shift, w)
    with pytest.raises(ValueError):
        layer.attention(q.float(), k, v, lam, c.shift, w)
    with pytest.raises(ValueError):
        layer.attention(q, k, v, lam.cpu(), c.shift, w)
    with pytest.raises(ValueError):
        layer.attention(q, k, v, lam, c.shift, w, kp=layer.pool_kv(k, v)[0])
    with pytest.raises(ValueError):
        layer.attention(q, k, v, lam, c.shift, w, route_idx=torch.zeros(1, 2, 16, 1, dtype=torch.int32, device="cuda"))


def test_rotary_positions_then_differential_attention():
    """The two operators as a layer runs them: packed projections -> norm and rotation ->
    pooled, routed and text keys -> differential attention, and the gradients back to the
    projections. In float32, against the two oracles in float64."""
    from oracle import rope_oracle as R
    from sparse_window_attention_b200.rope import GridRope, RopePart

    c = Case("joined", "f32", 1, 2, 64, (2, 4, 6), (1, 2, 3), (1, 1, 2), (2, 2, 3), 5, 1)
    g, h, N, text = c.geo, c.heads, c.geo.N, c.geo.n_text
    _, _, _, lam, w, dout, gen = c.inputs(8)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rnd(1, N, 5, h, 64)  # q1 q2 k1 k2 v of every head
    tx = rnd(1, text, 3, h, 64)  # k1 k2 v
    wq, wk = 1 + 0.2 * rnd(64), 1 + 0.2 * rnd(64)
    axes = (20, 22, 22)
    rope = GridRope(64, g.grid, axes, n_text=text, dtype="f32")
    q, k, v = torch.empty(1, 2 * h, N, 64, device="cuda"), torch.empty(1, 2 * h, N + text, 64, device="cuda"), torch.empty(1, h, N + text, 64, device="cuda")
    head = lambda t, i: t[:, :, i].permute(0, 2, 1, 3)  # noqa: E731
    parts = [RopePart(head(x, m), q[:, m::2], wq) for m in (0, 1)]
    parts += [RopePart(head(x, 2 + m), k[:, m::2, :N], wk) for m in (0, 1)]
    parts += [RopePart(head(tx, m), k[:, m::2, N:], wk, N) for m in (0, 1)]
    parts += [RopePart(head(x, 4), v[:, :, :N], rotate=False), RopePart(head(tx, 2), v[:, :, N:], None, N, False)]
    rope.forward(parts)
    layer = c.layer()
    out, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    dq, dk, dv, _, _ = layer.backward(q, k, v, lam, c.shift, saved, dout, w)
    grads = [dq[:, 0::2], dq[:, 1::2], dk[:, 0::2, :N], dk[:, 1::2, :N], dk[:, 0::2, N:], dk[:, 1::2, N:], dv[:, :, :N], dv[:, :, N:]]
    dx, dtx = torch.empty_like(x), torch.empty_like(tx)
    rope.backward(parts, grads, [head(dx, i) for i in range(4)] + [head(dtx, 0), head(dtx, 1), head(dx, 4), head(dtx, 2)])
    # the same in float64 on the CPU
    ang = R.angles(R.positions(g.grid, text), axes, 64, 10000.0)
    turn = lambda p: R.forward(p.x.double().cpu().numpy(), ang[p.first_row : p.first_row + p.x.shape[2]] * p.rotate,  # noqa: E731
                               "adjacent", None if p.weight is None else p.weight.double().cpu().numpy(), 1e-6)
    y = [torch.from_numpy(turn(p)) for p in parts]
    pair = lambda a, b: torch.stack([a, b], 2).flatten(1, 2)  # noqa: E731
    q64, v64 = pair(y[0], y[1]), torch.cat([y[6], y[7]], 2)
    k64 = torch.cat([pair(y[2], y[3]), pair(y[4], y[5])], 2)
    kp64, vp64 = (torch.from_numpy(O.pool_kv(t.numpy(), t.numpy(), g)[0]) for t in (k64, v64))
    route = saved[5].cpu()
    lam64, w64, do64 = lam.double().cpu(), w.double().cpu(), dout.double().cpu()
    ref = D.forward(q64, k64, v64, lam64, w64, g, kp64, vp64, route, c.gain, c.eps)
    tol = 16 * _score_error(q, k, 64)
    assert _rel(out.cpu(), ref) <= tol
    rq, rk, rv, _, _ = D.backward(q64, k64, v64, lam64, w64, g, do64, kp64, vp64, route, c.gain, c.eps)
    rg = [rq[:, 0::2], rq[:, 1::2], rk[:, 0::2, :N], rk[:, 1::2, :N], rk[:, 0::2, N:], rk[:, 1::2, N:], rv[:, :, :N], rv[:, :, N:]]
    for i, (p, dy) in enumerate(zip(parts, rg)):
        got = [head(dx, 0), head(dx, 1), head(dx, 2), head(dx, 3), head(dtx, 0), head(dtx, 1), head(dx, 4), head(dtx, 2)][i]
        want, _ = R.backward(p.x.double().cpu().numpy(), ang[p.first_row : p.first_row + p.x.shape[2]] * p.rotate, "adjacent",
                             dy.numpy(), None if p.weight is None else p.weight.double().cpu().numpy(), 1e-6)
        assert _rel(got.cpu(), torch.from_numpy(np.ascontiguousarray(want))) <= 2 * tol, i
