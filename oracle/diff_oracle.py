"""Float64 oracle of differential attention over the shifted-window key lists (test
infrastructure only): every window's keys gathered by token index computed from
coordinates, gradients by differentiation. Shares no code with the CUDA path."""
from __future__ import annotations

import torch


def window_tokens(geo):
    """[n_win, win_tokens] raster token ids of the shifted windows, from coordinates."""
    (T, H, W), (wt, wh, ww), (st, sy, sx) = geo.grid, geo.window, geo.shift
    ny, nx = H // wh, W // ww
    w = torch.arange((T // wt) * ny * nx)[:, None]
    i = torch.arange(wt * wh * ww)[None]
    t = (w // (ny * nx) * wt + i // (wh * ww) + st) % T
    y = (w // nx % ny * wh + i // ww % wh + sy) % H
    x = (w % nx * ww + i % ww + sx) % W
    return (t * H + y) * W + x


def patch_of_token(geo):
    (T, H, W), (pt, ph, pw) = geo.grid, geo.pool
    n = torch.arange(T * H * W)
    return (n // (H * W) // pt * (H // ph) + n // W % H // ph) * (W // pw) + n % W // pw


def mix(o1, o2, lam, weight, gain, eps):
    """The difference of the maps' outputs and its norm, lam [heads] on axis -3."""
    a = o1 - lam[:, None, None] * o2
    return a if weight is None else gain * weight * a / (a.square().mean(-1, keepdim=True) + eps).sqrt()


def forward(q, k, v, lam, weight, geo, kp=None, vp=None, route=None, gain=1.0, eps=1e-6, sizes=False):
    """out [B, h, N, d] from q [B, 2h, N, d], k [B, 2h, N + n_text, d], v [B, h, ..., d]
    (float64 tensors). With ``sizes`` also the two maps' outputs and the same sums over
    |v| (what rounding errors are relative to), each [B, h, N, d]."""
    B, h, N, d = q.shape[0], v.shape[1], q.shape[2], q.shape[3]
    ids = window_tokens(geo).to(q.device)
    rows = {n: torch.zeros(B, h, N, d, dtype=torch.float64, device=q.device) for n in ("o1", "o2", "a1", "a2")}
    outs = []
    for b in range(B):
        for j in range(h):
            seen = ids
            if geo.routed_k:
                seen = torch.cat([seen, ids[route[b, j].long()].flatten(1)], 1)
            if geo.n_text:
                seen = torch.cat([seen, torch.arange(N, N + geo.n_text, device=q.device).expand(ids.shape[0], -1)], 1)

            def keys(x, xp):
                x = x[seen]
                return x if xp is None else torch.cat([x, xp.expand(ids.shape[0], -1, -1)], 1)

            vv = keys(v[b, j], None if vp is None else vp[b, j])
            o = []
            for m in (0, 1):
                kk = keys(k[b, 2 * j + m], None if kp is None else kp[b, 2 * j + m])
                p = torch.softmax(q[b, 2 * j + m][ids] @ kk.transpose(1, 2) / d**0.5, -1)
                o.append(p @ vv)
                if sizes:
                    rows["o%d" % (m + 1)][b, j, ids.flatten()] = o[m].detach().flatten(0, 1)
                    rows["a%d" % (m + 1)][b, j, ids.flatten()] = (p.detach() @ vv.detach().abs()).flatten(0, 1)
            a = o[0] - lam[j] * o[1]
            if weight is not None:
                a = gain * weight * a / (a.square().mean(-1, keepdim=True) + eps).sqrt()
            back = torch.empty(N, dtype=torch.long, device=q.device)
            back[ids.flatten()] = torch.arange(N, device=q.device)
            outs.append(a.flatten(0, 1)[back])
    out = torch.stack(outs).view(B, h, N, d)
    return (out, rows) if sizes else out


def text_forward(q_text, k, v, lam, weight, gain=1.0, eps=1e-6, magnitudes=False):
    """The text queries' rows: every map dense over all rows of k, v. With
    ``magnitudes`` the sums run over |v| and are added up instead: a bound's size."""
    p = torch.softmax(q_text @ k.transpose(-1, -2) / q_text.shape[-1] ** 0.5, -1)
    if magnitudes:
        return p[:, 0::2] @ v.abs(), p[:, 1::2] @ v.abs()
    return mix(p[:, 0::2] @ v, p[:, 1::2] @ v, lam, weight, gain, eps)


def backward(q, k, v, lam, weight, geo, dout, kp=None, vp=None, route=None, gain=1.0, eps=1e-6):
    """(dq, dk, dv, dlam, dweight): pooled keys and values pass their gradients on
    evenly to their patch's tokens."""
    leaf = {"q": q, "k": k, "v": v, "lam": lam}
    if kp is not None:
        leaf.update(kp=kp, vp=vp)
    if weight is not None:
        leaf["weight"] = weight
    leaf = {n: x.detach().clone().requires_grad_() for n, x in leaf.items()}
    out = forward(leaf["q"], leaf["k"], leaf["v"], leaf["lam"], leaf.get("weight"), geo, leaf.get("kp"), leaf.get("vp"),
                  route, gain, eps)
    g = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), dout)))
    if kp is not None:
        patch, size = patch_of_token(geo).to(q.device), geo.pool[0] * geo.pool[1] * geo.pool[2]
        for n in ("k", "v"):
            g[n][:, :, : geo.N] += g[n + "p"][:, :, patch] / size
    return g["q"], g["k"], g["v"], g["lam"], g.get("weight")
