"""Differential attention over the shifted-window key lists: the layer of ``BasaLayer``
with the difference of two softmax maps per head.

``BasaDiffLayer`` holds one layer shape and calls the C entry points basa_diff_*. It
computes nothing itself; a call's buffers are allocated for that call, on its stream, so
calls and captured graphs share nothing but the device error word.
"""
from __future__ import annotations

import torch

from . import binding as B
from . import streams


class BasaDiffLayer:
    """``heads`` differential heads: map pairs (2 h, 2 h + 1) of q and k share v's head h.

    q [batch, 2 heads, N, head_dim]; k [batch, 2 heads, N + n_text, head_dim];
    v [batch, heads, N + n_text, head_dim]; ``lam`` [heads] the second maps' weights;
    ``weight`` [head_dim] (None: no norm) of the RMS norm of each head's rows, times
    ``gain``. Values and maps have the same width, ``head_dim``, which the norm spans. All
    tensors are contiguous. Pooled keys and values and routed windows are taken from ``kp``,
    ``vp``, ``route_idx`` where given and computed otherwise (``pool_kv``, ``route``).
    """

    def __init__(self, batch, heads, head_dim, grid, window, pool=(0, 0, 0), n_text=0, routed_k=0, dtype="bf16",
                 device="cuda", route_radius=0, gain=1.0, eps=1e-6):
        if dtype not in ("bf16", "f32"):
            raise ValueError("dtype: bf16 or f32")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("BasaDiffLayer clears its error word when it is made: make it before a capture")
        self.batch, self.heads, self.head_dim = batch, heads, head_dim
        self.grid, self.window, self.pool = tuple(grid), tuple(window), tuple(pool)
        self.n_text, self.routed_k, self.route_radius = n_text, routed_k, route_radius
        self.dtype_name, self.dtype = dtype, torch.bfloat16 if dtype == "bf16" else torch.float32
        self.gain, self.eps = float(gain), float(eps)
        self.device = streams.resolve_device(device)
        self.index = self.device.index
        T, H, W = self.grid
        self.N = T * H * W
        self.n_win = (T // window[0]) * (H // window[1]) * (W // window[2])
        self.has_pool = all(p > 0 for p in self.pool)
        self.n_pool = (T // pool[0]) * (H // pool[1]) * (W // pool[2]) if self.has_pool else 0
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=self.device)
        # the error word may be used on any stream from here on
        torch.cuda.current_stream(self.device).synchronize()
        self._params = {}

    def params(self, shift, heads=None, **extra) -> B.basa_params:
        key = (tuple(shift), heads, tuple(sorted(extra.items())) if extra else ())
        if key not in self._params:
            self._params[key] = B.make_params(self.batch, heads or self.heads, self.head_dim, self.grid, self.window,
                                              shift, self.pool, self.n_text, self.routed_k, self.dtype_name,
                                              dev_err=self.dev_err, route_radius=self.route_radius, **extra)
        return self._params[key]

    def _check(self, name, t, *shape, dtype=None):
        dtype = dtype or self.dtype
        if t.dtype is not dtype or t.get_device() != self.index:
            raise ValueError(f"{name}: {dtype} on {self.device}, got {t.dtype} on {t.device}")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous {shape}, got {tuple(t.shape)} with strides {t.stride()}")

    def _check_inputs(self, q, k, v, lam, weight, kp, vp, route_idx):
        b, h, d = self.batch, self.heads, self.head_dim
        self._check("q", q, b, 2 * h, self.N, d)
        self._check_kv(k, v)
        self._check("lam", lam, h)
        if weight is not None:
            self._check("weight", weight, d)
        if (kp is None) != (vp is None) or (kp is not None and not self.has_pool):
            raise ValueError("kp, vp: both or neither, and only with a pool patch")
        if kp is not None:
            self._check("kp", kp, b, 2 * h, self.n_pool, d)
            self._check("vp", vp, b, h, self.n_pool, d)
        if route_idx is not None:
            if self.routed_k == 0:
                raise ValueError("route_idx: this layer routes no windows")
            self._check("route_idx", route_idx, b, h, self.n_win, self.routed_k, dtype=torch.int32)

    def _check_kv(self, k, v):
        rows = self.N + self.n_text
        self._check("k", k, self.batch, 2 * self.heads, rows, self.head_dim)
        self._check("v", v, self.batch, self.heads, rows, self.head_dim)

    def _new(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def _workspace(self, nbytes):
        return self._new(nbytes, dtype=torch.uint8) if nbytes else None

    def pool_kv(self, k, v, stream=None):
        """Pooled keys [batch, 2 heads, n_pool, head_dim] and values of v's heads."""
        self._check_kv(k, v)
        with streams.on(self.device, stream):
            return self._pool_kv(k, v)

    def _pool_kv(self, k, v):
        kp = self._new(self.batch, 2 * self.heads, self.n_pool, self.head_dim)
        vp = self._new(self.batch, self.heads, self.n_pool, self.head_dim)
        B.basa_diff_pool_kv(k, v, kp, vp, self.params((0, 0, 0)))
        return kp, vp

    def route(self, q, k, shift, stream=None):
        """Routed windows [batch, heads, n_win, routed_k] of each head, chosen by its first
        map (basa_route_windows over the maps)."""
        self._check("q", q, self.batch, 2 * self.heads, self.N, self.head_dim)
        self._check("k", k, self.batch, 2 * self.heads, self.N + self.n_text, self.head_dim)
        with streams.on(self.device, stream):
            return self._route(q, k, shift)

    def _route(self, q, k, shift):
        params = self.params(shift, 2 * self.heads)
        idx = self._new(self.batch, self.heads, 2, self.n_win, self.routed_k, dtype=torch.int32)
        ws = self._workspace(max(B.basa_route_workspace_bytes(params), 16))
        B.basa_route_windows(q, k, idx, None, ws, params)
        return idx[:, :, 0].contiguous()

    def _keys(self, q, k, v, shift, kp, vp, route_idx):
        if self.has_pool and kp is None:
            kp, vp = self._pool_kv(k, v)
        if self.routed_k > 0 and route_idx is None:
            route_idx = self._route(q, k, shift)
        return kp, vp, route_idx

    def _forward(self, q, k, v, lam, shift, weight, kp, vp, route_idx, out, pre, second, lse, extra):
        params = self.params(shift, **extra)
        dp = B.make_diff_params(lam, weight, self.gain, self.eps)
        B.basa_diff_attn_fwd(q, k, v, kp, vp, route_idx, dp, out, pre, second, lse, params)

    def attention(self, q, k, v, lam, shift, weight=None, kp=None, vp=None, route_idx=None, out=None, stream=None,
                  **extra):
        """[batch, heads, N, head_dim]. ``extra`` goes into the parameters (e.g.
        ``wait_timeout_us``)."""
        self._check_inputs(q, k, v, lam, weight, kp, vp, route_idx)
        if out is not None:
            self._check("out", out, self.batch, self.heads, self.N, self.head_dim)
            at, end = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
            for t in (q, k, v, lam, weight, kp, vp, route_idx):  # contiguous, as checked
                if t is not None and t.data_ptr() < end and at < t.data_ptr() + t.numel() * t.element_size():
                    raise ValueError("out: overlaps an input, which other rows still read")
        with streams.on(self.device, stream):
            kp, vp, route_idx = self._keys(q, k, v, shift, kp, vp, route_idx)
            if out is None:
                out = self._new(self.batch, self.heads, self.N, self.head_dim)
            self._forward(q, k, v, lam, shift, weight, kp, vp, route_idx, out, None, None, None, extra)
        return out

    def attention_train(self, q, k, v, lam, shift, weight=None, kp=None, vp=None, route_idx=None, stream=None, **extra):
        """(out, saved): ``saved`` is what ``backward`` needs beside the inputs, the
        difference before the norm, the second maps' output, the log-sum-exps and the
        pooled and routed keys that were used."""
        self._check_inputs(q, k, v, lam, weight, kp, vp, route_idx)
        with streams.on(self.device, stream):
            kp, vp, route_idx = self._keys(q, k, v, shift, kp, vp, route_idx)
            shape = (self.batch, self.heads, self.N, self.head_dim)
            out, second = self._new(*shape), self._new(*shape)
            pre = out if weight is None else self._new(*shape)
            lse = self._new(self.batch, 2 * self.heads, self.N, dtype=torch.float32)
            self._forward(q, k, v, lam, shift, weight, kp, vp, route_idx, out, None if weight is None else pre, second,
                          lse, extra)
        return out, (pre, second, lse, kp, vp, route_idx)

    def backward(self, q, k, v, lam, shift, saved, dout, weight=None, kp=None, vp=None, route_idx=None, stream=None,
                 **extra):
        """(dq, dk, dv, dlam, dweight) of ``attention_train`` with the same arguments;
        dweight None without a norm. Without a norm ``out`` is part of ``saved`` and must
        not have been overwritten. Pooled and routed keys default to those in ``saved``."""
        self._check_inputs(q, k, v, lam, weight, kp, vp, route_idx)
        pre, second, lse, kp0, vp0, route0 = saved
        shape = (self.batch, self.heads, self.N, self.head_dim)
        self._check("dout", dout, *shape)
        self._check("saved", pre, *shape)
        self._check("saved", second, *shape)
        self._check("saved", lse, self.batch, 2 * self.heads, self.N, dtype=torch.float32)
        if kp is None:
            kp, vp = kp0, vp0
        if route_idx is None:
            route_idx = route0
        with streams.on(self.device, stream):
            params = self.params(shift, **extra)
            dp = B.make_diff_params(lam, weight, self.gain, self.eps)
            dq, dk, dv = (self._new(*t.shape) for t in (q, k, v))
            dlam = self._new(self.heads)
            dweight = None if weight is None else self._new(self.head_dim)
            ws = self._workspace(B.basa_diff_attn_bwd_workspace_bytes(dp, params))
            B.basa_diff_attn_bwd(q, k, v, kp, vp, route_idx, dp, pre, second, lse, dout, dq, dk, dv, dlam, dweight, ws,
                                 params)
        return dq, dk, dv, dlam, dweight

    def text_attention(self, q_text, k, v, lam, weight=None, stream=None):
        """Output rows [batch, heads, n_text, head_dim] of the text queries q_text [batch,
        2 heads, n_text, head_dim], dense over every row of k and v."""
        self._check("q_text", q_text, self.batch, 2 * self.heads, self.n_text, self.head_dim)
        self._check_kv(k, v)
        self._check("lam", lam, self.heads)
        if weight is not None:
            self._check("weight", weight, self.head_dim)
        with streams.on(self.device, stream):
            params = self.params((0, 0, 0))
            out = self._new(self.batch, self.heads, self.n_text, self.head_dim)
            ws = self._workspace(B.basa_diff_text_attn_workspace_bytes(params))
            dp = B.make_diff_params(lam, weight, self.gain, self.eps)
            B.basa_diff_text_attn_fwd(q_text, k, v, dp, out, ws, params)
        return out

    def device_error(self) -> int:
        return int(self.dev_err.item())
