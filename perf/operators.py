"""Cases of two operators around the shifted-window attention, with their plain forms.

rope   rotary positions along the t, y and x axes of the token grid, with the per-head
       RMS norm of queries and keys before it, from token-major packed projections
       [B, rows, 3, heads, d] to the head-major tensors the attention reads; and its
       gradients.
diff   differential attention over the shifted-window key lists: the difference of two
       softmax maps with a learned weight per head, and an RMS norm of each head's rows;
       and its gradients.

`run` computes them with elementary torch operations in float32 (angles in float64), or,
where `own` is set, through the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------- cases
def _rope(name, B, heads, d, grid, axes, text=0, first=0, rows=0, pairs="adjacent", norm=True, dtype="bf16", grad=False,
          theta=10000.0):
    return {"name": name, "op": "rope", "B": B, "heads": heads, "d": d, "T": grid[0], "H": grid[1], "W": grid[2],
            "dt": axes[0], "dh": axes[1], "dw": axes[2], "text": text, "first": first, "rows": rows, "pairs": pairs,
            "norm": norm, "dtype": dtype, "grad": grad, "theta": theta}


def _diff(name, B, heads, d, grid, window, shift, pool, text=0, routed=0, norm=True, dtype="bf16", grad=False):
    return {"name": name, "op": "diff", "B": B, "heads": heads, "d": d, "T": grid[0], "H": grid[1], "W": grid[2],
            "wt": window[0], "wh": window[1], "ww": window[2], "st": shift[0], "sy": shift[1], "sx": shift[2],
            "pt": pool[0], "ph": pool[1], "pw": pool[2], "text": text, "routed": routed, "norm": norm, "dtype": dtype,
            "grad": grad}


def listed():
    return [
        # one token of a stream of frames: latency
        _rope("rope one token", 1, 24, 128, (1, 64, 64), (16, 56, 56), first=1000, rows=1),
        # an image layer at 1024^2 with its text rows
        _rope("rope image 64x64 + 512 text", 1, 24, 128, (1, 64, 64), (16, 56, 56), text=512),
        # an image layer at 2048^2 with its text rows: the largest
        _rope("rope image 128x128 + 512 text", 1, 24, 128, (1, 128, 128), (16, 56, 56), text=512),
        # a video layer's training step; axis sizes that are no multiple of a vector
        _rope("rope video train", 1, 12, 128, (21, 30, 52), (44, 42, 42), grad=True),
        # float32, odd extents, pairs of the two halves, some channels not rotated, no norm
        _rope("rope f32 odd halves train", 2, 3, 64, (5, 19, 23), (16, 24, 22), text=7, pairs="halves", norm=False,
              dtype="f32", grad=True),
        # few short windows: latency
        _diff("diff small", 1, 2, 128, (1, 32, 32), (1, 8, 8), (0, 4, 4), (1, 4, 4)),
        # an image layer at 1024^2, 12 differential heads (24 maps)
        _diff("diff image 64x64", 1, 12, 128, (1, 64, 64), (1, 16, 16), (0, 8, 8), (1, 8, 8), text=512),
        # an image layer at 2048^2: the largest forward
        _diff("diff image 128x128", 1, 12, 128, (1, 128, 128), (1, 32, 32), (0, 16, 16), (1, 8, 8), text=512),
        # a video layer with routed windows; windows of 234 tokens end inside a tile
        _diff("diff video routed", 1, 6, 128, (21, 30, 52), (3, 6, 13), (0, 3, 6), (3, 6, 13), routed=4),
        # training steps: the image layer at 1024^2, and a batch of odd video windows
        _diff("diff image 64x64 train", 1, 12, 128, (1, 64, 64), (1, 16, 16), (0, 8, 0), (1, 8, 8), text=512, grad=True),
        _diff("diff video odd train", 2, 3, 128, (6, 18, 26), (3, 6, 13), (1, 2, 5), (3, 6, 13), text=77, routed=2,
              grad=True),
        # float32 windows
        _diff("diff f32", 1, 2, 64, (1, 32, 32), (1, 8, 8), (0, 4, 4), (1, 4, 4), norm=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([64, 128, 128])
        grad = rng.random() < 0.5
        B = rng.choice([1, 1, 2])
        T = rng.choice([1, 1, _log(rng, 2, 21)])
        heads = _log(rng, 1, 24)
        room = 380_000 // (B * T * heads)
        H = _log(rng, 1, max(1, min(128, room)))
        W = _log(rng, 1, max(1, min(128, room // H)))
        n = T * H * W
        left, axes = d, []
        for k in (3, 2, 1):
            a = min(left, 2 * rng.randint(1, max(1, left // k // 2 + 4)))
            axes.append(a)
            left -= a
        text = rng.choice([0, 0, rng.randint(1, 512)])
        first, rows = 0, 0
        if not text and rng.random() < 0.3:
            rows = _log(rng, 1, n)
            first = rng.randint(0, n - rows)
        c = _rope("", B, heads, d, (T, H, W), axes, text, first, rows, rng.choice(["adjacent", "halves"]),
                  rng.random() < 0.7, dtype, grad, rng.choice([10000.0, 256.0, 1e6]))
    else:
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        small = dtype == "f32"
        d = 64 if small else 128
        grad = not small and rng.random() < 0.5
        B, heads = rng.choice([1, 1, 2]), _log(rng, 1, 2 if small else 12)
        video = rng.random() < 0.5
        wt = rng.choice([1, 2, 3, 4]) if video else 1
        wh, ww = _log(rng, 4, 8 if small else 24), _log(rng, 4, 8 if small else 24)
        nt = rng.randint(1, 3) if video else 1
        ny, nx = rng.randint(1, 5), rng.randint(1, 5)
        grid, window = (wt * nt, wh * ny, ww * nx), (wt, wh, ww)
        shift = tuple(rng.randrange(g) if rng.random() < 0.7 else 0 for g in grid)
        pool = (0, 0, 0)
        if rng.random() < 0.7:
            pool = tuple(rng.choice([q for q in range(1, min(g, 16) + 1) if g % q == 0 and (q > 1 or g < 4)]
                                    or [g]) for g in grid)
        routed = rng.choice([0, 0, 1, 2, 3])
        routed = min(routed, nt * ny * nx - 1)
        text = rng.choice([0, rng.randint(1, 40 if small else 520)])
        c = _diff("", B, heads, d, grid, window, shift, pool, text, routed, rng.random() < 0.7, dtype, grad)
    del c["name"]
    # no more than the largest listed case of the operator
    cost = work(c)["bytes" if c["op"] == "rope" else "flops"]
    return c if cost <= (1.2e9 if c["op"] == "rope" else 3.6e11) else draw(rng)


# --------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _field(g, heads, T, H, W, d, amp):
    """A smooth field over the grid, one wave per (head, channel): [heads, T*H*W, d]."""
    a = torch.randint(-3, 4, (heads, 1, 1, 1, d), generator=g, device="cuda").float()
    b = torch.randint(-3, 4, (heads, 1, 1, 1, d), generator=g, device="cuda").float()
    ph = 2 * math.pi * torch.rand((heads, 1, 1, 1, d), generator=g, device="cuda")
    y = (torch.arange(H, device="cuda") / H).view(1, 1, H, 1, 1)
    x = (torch.arange(W, device="cuda") / W).view(1, 1, 1, W, 1)
    f = amp * torch.sin(2 * math.pi * (a * y + b * x) + ph)
    return f.expand(heads, T, H, W, d).reshape(heads, T * H * W, d)


def _prepare_rope(c, g):
    dt = DTYPES[c["dtype"]]
    n = c["T"] * c["H"] * c["W"]
    rows = c["rows"] or n
    s = {"case": c}
    proj = lambda r: _randn(g, c["B"], r, 3, c["heads"], c["d"]).mul_(1.5).to(dt)  # noqa: E731
    weight = lambda: (1 + 0.2 * _randn(g, c["d"])).to(dt)  # noqa: E731
    s["qkv"] = proj(rows)
    s["wq"], s["wk"] = (weight(), weight()) if c["norm"] else (None, None)
    if c["text"]:
        s["text_qkv"] = proj(c["text"])
        s["text_wq"], s["text_wk"] = (weight(), weight()) if c["norm"] else (None, None)
        # positions of the text rows: behind the grid on every axis
        far = max(c["T"], c["H"], c["W"])
        s["text_pos"] = (far + torch.arange(c["text"], device="cuda", dtype=torch.float32))[:, None].repeat(1, 3)
    if c["grad"]:
        grad = lambda r: _randn(g, c["B"], c["heads"], r, c["d"]).to(dt)  # noqa: E731
        s["dq"], s["dk"], s["dv"] = grad(rows), grad(rows + c["text"]), grad(rows + c["text"])
        if c["text"]:
            s["dq_text"] = grad(c["text"])
    if own:
        from sparse_window_attention_b200.rope import GridRope

        s["rope"] = GridRope(c["d"], (c["T"], c["H"], c["W"]), (c["dt"], c["dh"], c["dw"]), batch=c["B"],
                             theta=c["theta"], pairs=c["pairs"], n_text=c["text"], text_pos=s.get("text_pos"),
                             dtype=c["dtype"], eps=EPS)
    return s


def _windows_of(c):
    return (c["T"] // c["wt"]) * (c["H"] // c["wh"]) * (c["W"] // c["ww"])


def _prepare_diff(c, g):
    dt = DTYPES[c["dtype"]]
    B, h, d = c["B"], c["heads"], c["d"]
    n = c["T"] * c["H"] * c["W"]

    def tensor(heads, text):
        x = _randn(g, B, heads, n, d).mul_(0.6) + _field(g, heads, c["T"], c["H"], c["W"], d, 1.0)[None]
        if text:
            x = torch.cat([x, _randn(g, B, heads, text, d)], 2)
        return x.to(dt)

    s = {"case": c, "q": tensor(2 * h, 0), "k": tensor(2 * h, c["text"]), "v": tensor(h, c["text"])}
    s["lam"] = (0.2 + 0.6 * torch.rand(h, generator=g, device="cuda")).to(dt)
    s["weight"] = (1 + 0.2 * _randn(g, d)).to(dt) if c["norm"] else None
    s["kp"] = s["vp"] = s["route"] = None
    if c["pt"]:
        pooled = lambda x: x[:, :, :n].float().view(  # noqa: E731
            B, -1, c["T"] // c["pt"], c["pt"], c["H"] // c["ph"], c["ph"], c["W"] // c["pw"], c["pw"], d).mean((3, 5, 7)).reshape(
                B, x.shape[1], -1, d).to(dt)
        s["kp"], s["vp"] = pooled(s["k"]), pooled(s["v"])
    if c["routed"]:
        w = _windows_of(c)
        order = torch.rand((B, h, w, w - 1), generator=g, device="cuda").argsort(-1)[..., : c["routed"]]
        me = torch.arange(w, device="cuda").view(1, 1, w, 1)
        s["route"] = (order + (order >= me)).int()  # any other window
    if c["grad"]:
        s["dout"] = _randn(g, B, h, n, d).to(dt)
    if own:
        from sparse_window_attention_b200.diff_layer import BasaDiffLayer

        s["layer"] = BasaDiffLayer(B, h, d, (c["T"], c["H"], c["W"]), (c["wt"], c["wh"], c["ww"]), (c["pt"], c["ph"], c["pw"]),
                                   c["text"], c["routed"], c["dtype"], gain=GAIN, eps=EPS)
    return s


GAIN = 0.8  # factor behind the norm of a differential head


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return _prepare_rope(case, g) if case["op"] == "rope" else _prepare_diff(case, g)


# --------------------------------------------------------------------------- rope
def _tables(s):
    """cos and sin [rows, d/2] in float32 of the grid's tokens and of the text rows, from float64 angles."""
    c = s["case"]
    dims, ext = (c["dt"], c["dh"], c["dw"]), (c["T"], c["H"], c["W"])
    freq = [c["theta"] ** (-torch.arange(0, a, 2, device="cuda", dtype=torch.float64) / a) for a in dims]
    rest = c["d"] // 2 - sum(dims) // 2

    def joined(parts, fn, one):
        parts = [fn(x).float() for x in parts]
        return torch.cat(parts + [torch.full((*parts[0].shape[:-1], rest), one, device="cuda")], -1)

    angle = [torch.arange(e, device="cuda", dtype=torch.float64)[:, None] * f for e, f in zip(ext, freq)]
    view = [angle[0][:, None, None], angle[1][None, :, None], angle[2][None, None]]
    grid = lambda fn, one: joined([a.expand(*ext, -1) for a in view], fn, one).reshape(-1, c["d"] // 2)  # noqa: E731
    cos, sin = grid(torch.cos, 1.0), grid(torch.sin, 0.0)
    if c["rows"]:
        cos, sin = cos[c["first"] : c["first"] + c["rows"]], sin[c["first"] : c["first"] + c["rows"]]
    text = None
    if c["text"]:
        a = [s["text_pos"].double()[:, i : i + 1] * freq[i] for i in range(3)]
        text = joined(a, torch.cos, 1.0), joined(a, torch.sin, 0.0)
    return (cos, sin), text


def _rotated(x, cos, sin, pairs):
    if pairs == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_rope_fwd(x, weight, table, pairs):
    """x: [B, rows, heads, d] -> head-major, normalised and rotated, in float32."""
    x = x.permute(0, 2, 1, 3).float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    return _rotated(x, *table, pairs)


def _plain_rope_bwd(x, weight, table, pairs, dy):
    """Gradients of _plain_rope_fwd w.r.t. x (token-major) and the weight."""
    g = _rotated(dy.float(), table[0], -table[1], pairs)
    dweight = None
    if weight is not None:
        x = x.permute(0, 2, 1, 3).float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dweight = (g * xh).sum((0, 1, 2)).to(weight.dtype)
        g = g * weight.float()
        g = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return g.permute(0, 2, 1, 3), dweight


def _run_rope_plain(s):
    c, dt = s["case"], s["qkv"].dtype
    table, text_table = _tables(s)
    p, n = c["pairs"], s["qkv"].shape[1]
    x, t = s["qkv"], s.get("text_qkv")
    q = _plain_rope_fwd(x[:, :, 0], s["wq"], table, p).to(dt)
    k = _plain_rope_fwd(x[:, :, 1], s["wk"], table, p)
    v = x[:, :, 2].permute(0, 2, 1, 3)
    out = {}
    if t is not None:
        out["q_text"] = _plain_rope_fwd(t[:, :, 0], s["text_wq"], text_table, p).to(dt)
        k = torch.cat([k, _plain_rope_fwd(t[:, :, 1], s["text_wk"], text_table, p)], 2)
        v = torch.cat([v, t[:, :, 2].permute(0, 2, 1, 3)], 2)
    out.update(q=q, k=k.to(dt), v=v.contiguous())
    if not c["grad"]:
        return out

    def back(x, wq, wk, table, dq, dk, dv):
        gq, dwq = _plain_rope_bwd(x[:, :, 0], wq, table, p, dq)
        gk, dwk = _plain_rope_bwd(x[:, :, 1], wk, table, p, dk)
        return torch.stack([gq, gk, dv.permute(0, 2, 1, 3).float()], 2).to(dt), dwq, dwk

    out["dqkv"], out["dwq"], out["dwk"] = back(x, s["wq"], s["wk"], table, s["dq"], s["dk"][:, :, :n], s["dv"][:, :, :n])
    if t is not None:
        out["dtext_qkv"], out["dtext_wq"], out["dtext_wk"] = back(t, s["text_wq"], s["text_wk"], text_table, s["dq_text"],
                                                                  s["dk"][:, :, n:], s["dv"][:, :, n:])
    return {k: v for k, v in out.items() if v is not None}


def _run_rope_own(s):
    from sparse_window_attention_b200.rope import RopePart

    c, dt = s["case"], s["qkv"].dtype
    n, N = s["qkv"].shape[1], c["T"] * c["H"] * c["W"]
    new = lambda r: torch.empty(c["B"], c["heads"], r, c["d"], dtype=dt, device="cuda")  # noqa: E731
    heads = lambda x, i: x[:, :, i].permute(0, 2, 1, 3)  # noqa: E731
    q, k, v = new(n), new(n + c["text"]), new(n + c["text"])
    out = {"q": q, "k": k, "v": v}
    first = c["first"]
    x, t = s["qkv"], s.get("text_qkv")
    vis = slice(0, n)
    parts = [RopePart(heads(x, 0), q, s["wq"], first), RopePart(heads(x, 1), k[:, :, vis], s["wk"], first),
             RopePart(heads(x, 2), v[:, :, vis], None, first, rotate=False)]
    if t is not None:
        out["q_text"] = new(c["text"])
        parts += [RopePart(heads(t, 0), out["q_text"], s["text_wq"], N), RopePart(heads(t, 1), k[:, :, n:], s["text_wk"], N),
                  RopePart(heads(t, 2), v[:, :, n:], None, N, rotate=False)]
    s["rope"].forward(parts)
    if not c["grad"]:
        return out
    out["dqkv"] = torch.empty_like(x)
    grads = [s["dq"], s["dk"][:, :, vis], s["dv"][:, :, vis]]
    dx = [heads(out["dqkv"], i) for i in range(3)]
    if t is not None:
        out["dtext_qkv"] = torch.empty_like(t)
        grads += [s["dq_text"], s["dk"][:, :, n:], s["dv"][:, :, n:]]
        dx += [heads(out["dtext_qkv"], i) for i in range(3)]
    dw = s["rope"].backward(parts, grads, dx)
    for name, w in zip(("dwq", "dwk", None, "dtext_wq", "dtext_wk"), dw):
        if w is not None:
            out[name] = w
    return out


def _exact_rope(s):
    """Every row by itself: complex rotation of its channel pairs, gradients by differentiation, in 64 bits."""
    c = s["case"]
    N, half = c["T"] * c["H"] * c["W"], c["d"] // 2
    owner = torch.tensor([0] * (c["dt"] // 2) + [1] * (c["dh"] // 2) + [2] * (c["dw"] // 2), device="cuda", dtype=torch.long)
    power = torch.cat([torch.arange(a // 2, device="cuda", dtype=torch.float64) * 2 / a for a in (c["dt"], c["dh"], c["dw"]) if a])
    freq = torch.exp(-power * math.log(c["theta"]))

    def phase(pos):  # [rows, 3] -> unit complex numbers [rows, d/2]
        turn = torch.zeros(pos.shape[0], half, device="cuda", dtype=torch.float64)
        turn[:, : owner.numel()] = pos[:, owner] * freq
        return torch.polar(torch.ones_like(turn), turn)

    tok = torch.arange(N, device="cuda")[c["first"] : c["first"] + (c["rows"] or N)]
    grid = torch.stack([tok // (c["H"] * c["W"]), tok // c["W"] % c["H"], tok % c["W"]], -1).double()

    def forward(x, w, turn):  # x: [B, rows, heads, d]
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS) * w
        z = x.unflatten(-1, (half, 2)) if c["pairs"] == "adjacent" else x.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * turn[None, :, None]
        z = torch.view_as_real(z)
        return (z if c["pairs"] == "adjacent" else z.transpose(-1, -2)).flatten(-2).transpose(1, 2)

    def group(qkv, wq, wk, turn, grads):
        leaf = [t.double().requires_grad_() for t in qkv.unbind(2)]
        ws = [None if w is None else w.double().requires_grad_() for w in (wq, wk)]
        y = [forward(leaf[0], ws[0], turn), forward(leaf[1], ws[1], turn), leaf[2].transpose(1, 2)]
        if grads is None:
            return [t.detach() for t in y], None, None
        want = leaf + [w for w in ws if w is not None]
        got = torch.autograd.grad(y, want, [t.double() for t in grads])
        return [t.detach() for t in y], torch.stack(got[:3], 2), got[3:]

    n = s["qkv"].shape[1]
    cut = lambda sl: [s["dk"][:, :, sl], s["dv"][:, :, sl]] if c["grad"] else None  # noqa: E731
    y, dx, dw = group(s["qkv"], s["wq"], s["wk"], phase(grid), [s["dq"]] + cut(slice(0, n)) if c["grad"] else None)
    out = {"q": y[0], "k": y[1], "v": y[2]}
    if c["grad"]:
        out["dqkv"] = dx
        if c["norm"]:
            out["dwq"], out["dwk"] = dw
    if c["text"]:
        y, dx, dw = group(s["text_qkv"], s["text_wq"], s["text_wk"], phase(s["text_pos"].double()),
                          [s["dq_text"]] + cut(slice(n, None)) if c["grad"] else None)
        out["q_text"] = y[0]
        out["k"], out["v"] = torch.cat([out["k"], y[1]], 2), torch.cat([out["v"], y[2]], 2)
        if c["grad"]:
            out["dtext_qkv"] = dx
            if c["norm"]:
                out["dtext_wq"], out["dtext_wk"] = dw
    return out


# --------------------------------------------------------------------------- differential attention
def _to_windows(c, x):
    """[B, heads, N, d] -> [B, heads, windows, tokens of a window, d] of the shifted grid."""
    B, h, _, d = x.shape
    x = x.reshape(B, h, c["T"], c["H"], c["W"], d).roll((-c["st"], -c["sy"], -c["sx"]), (2, 3, 4))
    x = x.view(B, h, c["T"] // c["wt"], c["wt"], c["H"] // c["wh"], c["wh"], c["W"] // c["ww"], c["ww"], d)
    return x.permute(0, 1, 2, 4, 6, 3, 5, 7, 8).reshape(B, h, _windows_of(c), -1, d)


def _from_windows(c, x):
    B, h, d = x.shape[0], x.shape[1], x.shape[-1]
    x = x.view(B, h, c["T"] // c["wt"], c["H"] // c["wh"], c["W"] // c["ww"], c["wt"], c["wh"], c["ww"], d)
    x = x.permute(0, 1, 2, 5, 3, 6, 4, 7, 8).reshape(B, h, c["T"], c["H"], c["W"], d)
    return x.roll((c["st"], c["sy"], c["sx"]), (2, 3, 4)).reshape(B, h, -1, d)


def _route_index(s, maps):
    """Flat window ids [B * heads * maps * windows * routed] into [B * heads * maps * windows]."""
    r = s["route"].long().repeat_interleave(maps, 1)
    B, h, w, _ = r.shape
    return (r + (torch.arange(B * h, device="cuda") * w).view(B, h, 1, 1)).flatten()


def _key_lists(s, x, pooled, maps):
    """The key (or value) rows that each window's queries see: [B, heads, windows, keys, d]."""
    c = s["case"]
    n = c["T"] * c["H"] * c["W"]
    x = x.float()
    win = _to_windows(c, x[:, :, :n])
    parts = [win]
    if c["routed"]:
        parts.append(win.flatten(0, 2)[_route_index(s, maps)].view(*win.shape[:3], -1, win.shape[-1]))
    if pooled is not None:
        parts.append(pooled.float()[:, :, None].expand(-1, -1, win.shape[2], -1, -1))
    if c["text"]:
        parts.append(x[:, :, None, n:].expand(-1, -1, win.shape[2], -1, -1))
    return torch.cat(parts, 3)


def _key_grads(s, g, maps):
    """Gradients of the rows behind _key_lists' output: the tokens (a pooled row's shared evenly by its patch) and the text."""
    c = s["case"]
    B, h, w, _, d = g.shape
    own_n = c["wt"] * c["wh"] * c["ww"]
    at = own_n
    win = g[:, :, :, :own_n].contiguous()
    if c["routed"]:
        routed = g[:, :, :, at : at + c["routed"] * own_n].reshape(-1, own_n, d)
        win = win.flatten(0, 2).index_add(0, _route_index(s, maps), routed).view(B, h, w, own_n, d)
        at += c["routed"] * own_n
    tok = _from_windows(c, win)
    if c["pt"]:
        grid = (c["T"] // c["pt"], c["H"] // c["ph"], c["W"] // c["pw"])
        np_ = grid[0] * grid[1] * grid[2]
        gp = g[:, :, :, at : at + np_].sum(2) / (c["pt"] * c["ph"] * c["pw"])
        gp = gp.view(B, h, grid[0], 1, grid[1], 1, grid[2], 1, d).expand(B, h, grid[0], c["pt"], grid[1], c["ph"], grid[2], c["pw"], d)
        tok = tok + gp.reshape(B, h, -1, d)
        at += np_
    return torch.cat([tok, g[:, :, :, at:].sum(2)], 2) if c["text"] else tok


def _run_diff_plain(s):
    c, dt = s["case"], s["q"].dtype
    scale = 1 / math.sqrt(c["d"])
    q = _to_windows(c, s["q"].float())
    k, v = _key_lists(s, s["k"], s["kp"], 2), _key_lists(s, s["v"], s["vp"], 1)
    lam = s["lam"].float().view(1, -1, 1, 1, 1)
    two = lambda x: x.unflatten(1, (-1, 2)).unbind(2)  # noqa: E731
    score = q @ k.transpose(-1, -2) * scale
    prob = torch.exp(score - score.amax(-1, keepdim=True))
    prob = prob / prob.sum(-1, keepdim=True)
    p1, p2 = two(prob)
    mix = p1 - lam * p2
    a = mix @ v
    if c["norm"]:
        r = torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS)
        ah = a * r
        out = ah * s["weight"].float() * GAIN
    else:
        out = a
    out = {"out": _from_windows(c, out).to(dt)}
    if not c["grad"]:
        return out
    g = _to_windows(c, s["dout"].float())
    if c["norm"]:
        g = g * GAIN
        out["dweight"] = (g * ah).sum((0, 1, 2, 3)).to(dt)
        g = g * s["weight"].float()
        g = r * (g - ah * (g * ah).mean(-1, keepdim=True))
    gv = g @ v.transpose(-1, -2)  # of the mixed map
    out["dlam"] = -(p2 * gv).sum((0, 2, 3, 4)).to(dt)
    dv = mix.transpose(-1, -2) @ g
    back = lambda p: p * (gv - (p * gv).sum(-1, keepdim=True))  # noqa: E731
    ds = torch.stack([back(p1), -lam * back(p2)], 2).flatten(1, 2) * scale
    out["dq"] = _from_windows(c, ds @ k).to(dt)
    out["dk"] = _key_grads(s, ds.transpose(-1, -2) @ q, 2).to(dt)
    out["dv"] = _key_grads(s, dv, 1).to(dt)
    return out


def _run_diff_own(s):
    c, layer = s["case"], s["layer"]
    shift = (c["st"], c["sy"], c["sx"])
    args = (s["q"], s["k"], s["v"], s["lam"], shift)
    keys = {"kp": s["kp"], "vp": s["vp"], "route_idx": s["route"]}
    if not c["grad"]:
        return {"out": layer.attention(*args, s["weight"], **keys)}
    out, saved = layer.attention_train(*args, s["weight"], **keys)
    dq, dk, dv, dlam, dweight = layer.backward(*args, saved, s["dout"], s["weight"], **keys)
    r = {"out": out, "dq": dq, "dk": dk, "dv": dv, "dlam": dlam}
    if dweight is not None:
        r["dweight"] = dweight
    return r


def _exact_diff(s):
    """Head by head in 64 bits: keys gathered by token index, gradients by differentiation."""
    c = s["case"]
    B, h, d = c["B"], c["heads"], c["d"]
    T, H, W = c["T"], c["H"], c["W"]
    N, nw = T * H * W, _windows_of(c)
    # token ids of every shifted window, by coordinates
    ny, nx = H // c["wh"], W // c["ww"]
    w = torch.arange(nw, device="cuda")[:, None]
    i = torch.arange(c["wt"] * c["wh"] * c["ww"], device="cuda")[None]
    t = (w // (ny * nx) * c["wt"] + i // (c["wh"] * c["ww"]) + c["st"]) % T
    y = (w // nx % ny * c["wh"] + i // c["ww"] % c["wh"] + c["sy"]) % H
    x = (w % nx * c["ww"] + i % c["ww"] + c["sx"]) % W
    ids = (t * H + y) * W + x  # [windows, tokens]
    patch = None
    if c["pt"]:
        tok = torch.arange(N, device="cuda")
        patch = (tok // (H * W) // c["pt"] * (H // c["ph"]) + tok // W % H // c["ph"]) * (W // c["pw"]) + tok % W // c["pw"]
        size = c["pt"] * c["ph"] * c["pw"]
    out = {"out": torch.empty(B, h, N, d, dtype=torch.float64, device="cuda")}
    if c["grad"]:
        for name in ("q", "k", "v"):
            out["d" + name] = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
        out["dlam"] = torch.zeros(h, dtype=torch.float64, device="cuda")
        if c["norm"]:
            out["dweight"] = torch.zeros(d, dtype=torch.float64, device="cuda")
    for b in range(B):
        for j in range(h):
            leaf = {"q1": s["q"][b, 2 * j], "q2": s["q"][b, 2 * j + 1], "k1": s["k"][b, 2 * j], "k2": s["k"][b, 2 * j + 1],
                    "v": s["v"][b, j], "lam": s["lam"][j]}
            if c["pt"]:
                leaf.update(kp1=s["kp"][b, 2 * j], kp2=s["kp"][b, 2 * j + 1], vp=s["vp"][b, j])
            if c["norm"]:
                leaf["weight"] = s["weight"]
            leaf = {n: z.double().requires_grad_(c["grad"]) for n, z in leaf.items()}
            seen = ids
            if c["routed"]:
                seen = torch.cat([ids, ids[s["route"][b, j].long()].flatten(1)], 1)
            if c["text"]:
                seen = torch.cat([seen, torch.arange(N, N + c["text"], device="cuda").expand(nw, -1)], 1)

            def rows(z, zp):
                z = z[seen]
                return z if zp is None else torch.cat([z, zp.expand(nw, -1, -1)], 1)

            v = rows(leaf["v"], leaf.get("vp"))
            o = [torch.softmax(torch.einsum("wqd,wkd->wqk", leaf["q" + m][ids], rows(leaf["k" + m], leaf.get("kp" + m))) / d**0.5, -1) @ v
                 for m in "12"]
            a = o[0] - leaf["lam"] * o[1]
            if c["norm"]:
                a = a / (a.square().mean(-1, keepdim=True) + EPS).sqrt() * leaf["weight"] * GAIN
            out["out"][b, j, ids.flatten()] = a.detach().flatten(0, 1)
            if not c["grad"]:
                continue
            names = list(leaf)
            got = dict(zip(names, torch.autograd.grad(a, [leaf[n] for n in names], s["dout"][b, j].double()[ids])))
            for m in (0, 1):
                out["dq"][b, 2 * j + m] = got["q%d" % (m + 1)]
                out["dk"][b, 2 * j + m] = got["k%d" % (m + 1)]
                if c["pt"]:
                    out["dk"][b, 2 * j + m, :N] += got["kp%d" % (m + 1)][patch] / size
            out["dv"][b, j] = got["v"]
            if c["pt"]:
                out["dv"][b, j, :N] += got["vp"][patch] / size
            out["dlam"][j] += got["lam"]
            if c["norm"]:
                out["dweight"] += got["weight"]
    return out


# --------------------------------------------------------------------------- what the tools call
def run(state):
    if state["case"]["op"] == "rope":
        return _run_rope_own(state) if own else _run_rope_plain(state)
    return _run_diff_own(state) if own else _run_diff_plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_diff(s)


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["T"] * c["H"] * c["W"]
    if c["op"] == "rope":
        values = 3 * c["B"] * c["heads"] * ((c["rows"] or n) + c["text"]) * c["d"]
        # x read and y written; for a training step dy read and dx written too (x is read once)
        return {"bytes": (4 if c["grad"] else 2) * values * size, "flops": (9 if c["grad"] else 4) * values}
    keys = c["wt"] * c["wh"] * c["ww"] * (1 + c["routed"]) + c["text"]
    pooled = 0
    if c["pt"]:
        pooled = (c["T"] // c["pt"]) * (c["H"] // c["ph"]) * (c["W"] // c["pw"])
    product = 2 * c["B"] * c["heads"] * n * (keys + pooled) * c["d"]
    q, kv = 2 * n, 3 * (n + c["text"] + pooled)
    b = (q + kv + n) * c["B"] * c["heads"] * c["d"] * size
    if not c["grad"]:
        return {"bytes": b, "flops": 4 * product}  # two maps' scores, two products with v
    b += (q + 3 * (n + c["text"]) + n) * c["B"] * c["heads"] * c["d"] * size  # dq, dk, dv written, dout read
    # backward: the scores again (2), dout v^T and the mixed map's v gradient (1 each), dq and dk of each map (4)
    return {"bytes": b, "flops": 12 * product}
