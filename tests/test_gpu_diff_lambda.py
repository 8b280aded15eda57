"""lambda's gradient where a head's rows are small against the norm's sqrt(eps): maps that are
nearly alike, lambda at or next to 1, small values. Against the float64 oracle.

Tolerance. h = 2^-8, half a step of bfloat16. Let delta be what the kernels' a, rounded and from
rounded probabilities, is off the true one: per channel and independently with a standard
deviation of s = h / sqrt(3) (Q1 + |lambda| Q2 + |a|), Q = sqrt(sum P^2 v^2). With u = gain w
dout, r = (mean a^2 + eps)^-1/2 and g = r (u - a r^2 mean(u a)), a first-order change of g . O2
is  -r^3 / d [(a.delta) (u.O2) + (delta.O2) (u.a) + (a.O2) (u.delta) - 3 r^2 / d (a.delta) (u.a)
(a.O2)].  The maps' row sums R = sum P dP, which the dq pass takes in float32, tell g . delta =
R1 - lambda R2 - g . a, and with c = a.O2 r^2 / d that times c takes out the third term and one
of the three in the fourth. What is left per row is
  r^3 / d delta . [a (u.O2) + O2 (u.a) - 2 r^2 / d a (u.a) (a.O2)],
independent between rows: 16 standard deviations. Beside it stand the second order in delta,
at most r^3 / d |delta|^2 |u.O2| on the average, the product of g's rounding with O2's, the
float32 sums (2^-18 of their terms) and the result's rounding, h of it. The other choice of c,
a.O2 / a.a, is the same where eps is small against mean a^2, and is off by up to the whole
value here."""
import pytest
import torch

from oracle import diff_oracle as D
from tests.test_gpu_diff import Case, _f64

pytestmark = pytest.mark.gpu


def _bound(c, q64, k64, v64, lam64, w64, do64):
    h, d, ids = 2.0**-8, c.d, D.window_tokens(c.geo).cuda()
    total = torch.zeros_like(lam64)
    for j in range(c.heads):
        P = [torch.softmax(q64[0, 2 * j + m][ids] @ k64[0, 2 * j + m][ids].transpose(1, 2) / d**0.5, -1) for m in (0, 1)]
        v, u = v64[0, j][ids], c.gain * w64 * do64[0, j][ids]
        o, quad, size = [p @ v for p in P], [(p.square() @ v.square()).sqrt() for p in P], [p @ v.abs() for p in P]
        a = o[0] - lam64[j] * o[1]
        dot = lambda x, y: (x * y).sum(-1, keepdim=True)  # noqa: E731
        r2 = 1 / (a.square().mean(-1, keepdim=True) + c.eps)
        r3 = r2**1.5 / d
        g = r2.sqrt() * (u - a * r2 / d * dot(u, a))
        s = h / 3**0.5 * (quad[0] + lam64[j].abs() * quad[1] + a.abs())
        left = r3 * (a * dot(u, o[1]) + o[1] * dot(u, a) - 2 * r2 / d * a * dot(u, a) * dot(a, o[1]))
        var = (s * left).square().sum() + (h * h / 3 * g * (quad[1] + o[1].abs())).square().sum()
        second = (r3 * dot(s, s) * dot(u, o[1]).abs()).sum()
        cc = (dot(a, o[1]) * r2 / d).abs()
        sums = (g.abs() * (size[1] + cc * (size[0] + lam64[j].abs() * size[1]))).sum()
        total[j] = 16 * var.sqrt() + second + 2.0**-18 * sums
    return total


@pytest.mark.parametrize("step,size,eps", [(0.003, 0.02, 1e-6), (0.05, 0.02, 1e-5), (0.05, 0.005, 1e-5)])
def test_gradient_of_lambda_where_the_rows_are_small(step, size, eps):
    c = Case("small_rows", "bf16", 1, 4, 128, (1, 32, 32), (1, 16, 16), (0, 8, 8))
    c.eps = eps
    q, k, v, _, w, dout, gen = c.inputs(31)
    near = lambda x: (x[:, 0::2] + step * torch.randn(x[:, 0::2].shape, generator=gen, device="cuda")).to(x.dtype)  # noqa: E731
    q[:, 1::2], k[:, 1::2] = near(q), near(k)
    v = (size * (v.float() + 1)).to(v.dtype)  # a common part
    lam = torch.tensor([1.0, 0.996, 1.0, 0.996], device="cuda").to(q.dtype)
    layer = c.layer()
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    dlam = layer.backward(q, k, v, lam, c.shift, saved, dout, w)[3]
    q64, k64, v64, lam64, w64, do64 = _f64(q, k, v, lam, w, dout)
    ref = D.backward(q64, k64, v64, lam64, w64, c.geo, do64, gain=c.gain, eps=c.eps)[3]
    bound = _bound(c, q64, k64, v64, lam64, w64, do64) + 2.0**-8 * ref.abs()
    assert ((dlam.double() - ref).abs() <= bound).all(), (dlam, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_almost_nothing(dtype):
    """Rows of a whose squares leave float32's range: finite gradients."""
    c = Case("nothing", dtype, 1, 2, 128, (1, 16, 16), (1, 8, 8), (0, 4, 4))
    q, k, v, lam, w, dout, _ = c.inputs(32)
    q[:, 1::2], k[:, 1::2] = q[:, 0::2], k[:, 0::2]
    lam = torch.ones_like(lam)
    layer = c.layer()
    _, saved = layer.attention_train(q, k, v, lam, c.shift, w)
    for tiny in (0.0, 1e-38, 1e-24, 1e-19, 1e-12):
        pre = torch.full_like(saved[0], tiny)
        grads = layer.backward(q, k, v, lam, c.shift, (pre, *saved[1:]), dout, w)
        assert all(x.isfinite().all() for x in grads), tiny
