"""Rotary positions along the t, y and x axes of the token grid, with the per-head RMS
norm of queries and keys before them: what stands between a layer's projections and
``BasaLayer``.

``GridRope`` holds the angle tables of one grid (computed once) and calls the C entry
points basa_rope_fwd and basa_rope_bwd. It computes nothing itself.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B
from . import streams

PAIRS = {"adjacent": B.BASA_ROPE_PAIRS_ADJACENT, "halves": B.BASA_ROPE_PAIRS_HALVES}


class RopePart(NamedTuple):
    """One tensor of a call: ``x`` [batch, heads, rows, head_dim] in any strides whose
    channels are contiguous and whose other steps are multiples of 16 bytes (a slice of a
    token-major packed projection, permuted), written to ``y`` (same shape, its own
    strides; x itself for in place). Row r is row ``first_row`` + r of the key sequence:
    grid tokens in raster order, then the text rows. With ``weight`` [head_dim] the rows
    are RMS-normalised first; without ``rotate`` they are only laid out."""

    x: torch.Tensor
    y: torch.Tensor
    weight: Optional[torch.Tensor] = None
    first_row: int = 0
    rotate: bool = True


class GridRope:
    """Rotary positions of a T x H x W grid and ``n_text`` text rows behind it.

    ``axes`` = channels turned by the t, y and x position (even, sum <= head_dim; the
    other channels pass). Pair i of an axis with m channels turns by position *
    theta^(-2 i / m). ``pairs``: "adjacent" channels (2 i, 2 i + 1) or the "halves" of a
    head (i, i + head_dim / 2). Grid token (i, j, l) is at ``origin`` + ``step`` * (i, j,
    l). ``text_pos`` [n_text, 3]: positions of the text rows (None: not turned).
    """

    def __init__(self, head_dim, grid, axes, batch=1, theta=10000.0, pairs="adjacent", origin=(0.0, 0.0, 0.0),
                 step=(1.0, 1.0, 1.0), n_text=0, text_pos=None, dtype="bf16", eps=1e-6, device="cuda"):
        if pairs not in PAIRS:
            raise ValueError(f"pairs: one of {sorted(PAIRS)}")
        if dtype not in ("bf16", "f32"):
            raise ValueError("dtype: bf16 or f32")
        if text_pos is not None and tuple(text_pos.shape) != (n_text, 3):
            raise ValueError("text_pos: [n_text, 3]")
        self.head_dim, self.grid, self.axes, self.batch = head_dim, tuple(grid), tuple(axes), batch
        self.n_text, self.eps = n_text, float(eps)
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.params = B.make_params(batch, 1, head_dim, self.grid, (1, 1, 1), n_text=n_text, dtype=dtype)
        self.rope_params = B.make_rope_params(self.axes, float(theta), PAIRS[pairs], origin, step)
        self.device = streams.resolve_device(device)
        self.index, self.weight_shape = self.device.index, (head_dim,)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("GridRope computes its tables when it is made: make it before a capture")
        nbytes = B.basa_rope_table_bytes(self.rope_params, self.params)
        with streams.on(self.device):
            self.table = torch.empty(max(nbytes, 16) // 4, dtype=torch.float32, device=self.device)
            if text_pos is not None:
                text_pos = text_pos.to(self.device, torch.float32).contiguous()
            B.basa_rope_table(text_pos, self.table, self.rope_params, self.params)
            # the tables may be used on any stream from here on
            torch.cuda.current_stream().synchronize()

    def _refuse(self, name, t, shape=None):
        """Raises for a tensor that _fits turned down."""
        if t.dtype != self.dtype or t.device != self.device:
            raise ValueError(f"{name}: {self.dtype} on {self.device}, got {t.dtype} on {t.device}")
        if shape is None:
            shape = (self.batch, "heads", "rows", self.head_dim)
        raise ValueError(f"{name}: {tuple(shape)} with contiguous channels, got {tuple(t.shape)} with strides {t.stride()}")

    def _record(self, part: RopePart, dy=None, dx=None, dweight=None):
        """The C record of a part, checked. Written out flat: it runs for every tensor of
        every call, and a call of one token is bound by it."""
        x, y, weight, first_row, rotate = part
        dtype, index, shape, xs = self.dtype, self.index, x.shape, x.stride()
        if (x.dtype is not dtype or x.get_device() != index or len(shape) != 4 or shape[0] != self.batch
                or shape[3] != self.head_dim or xs[3] != 1):
            self._refuse("x", x)
        wp = 0
        if weight is not None:
            if weight.dtype is not dtype or weight.get_device() != index or weight.shape != self.weight_shape or weight.stride(0) != 1:
                self._refuse("weight", weight, self.weight_shape)
            wp = weight.data_ptr()
        dp = ds0 = ds1 = ds2 = 0
        name = "y"
        if dy is not None:
            ds0, ds1, ds2, ds3 = dy.stride() if dy.dim() == 4 else (0, 0, 0, 0)
            if dy.dtype is not dtype or dy.get_device() != index or dy.shape != shape or ds3 != 1:
                self._refuse("grads", dy, shape)
            dp, y, name = dy.data_ptr(), dx, "dx"
        ys = y.stride()
        if y.dtype is not dtype or y.get_device() != index or y.shape != shape or ys[3] != 1:
            self._refuse(name, y, shape)
        return B.rope_record(x.data_ptr(), xs[0], xs[1], xs[2], y.data_ptr(), ys[0], ys[1], ys[2], dp, ds0, ds1, ds2, wp,
                             0 if dweight is None else dweight.data_ptr(), shape[1], shape[2], first_row, 1 if rotate else 0)

    def forward(self, parts, stream=None):
        """Norm and rotation of every part in one launch; returns their ``y``."""
        records = [self._record(p) for p in parts]
        with streams.on(self.device, stream):
            B.basa_rope_fwd(records, self.table, self.eps, self.rope_params, self.params)
        return [p.y for p in parts]

    def backward(self, parts, grads, dx, stream=None):
        """Gradients for the parts of a forward call: ``grads`` of their outputs (any
        strides, as x), written to ``dx``. A part's ``x`` must still hold the forward's
        input where it has a weight (``y`` is not read). Returns the weights' gradients
        (None for a part without weight)."""
        if not len(parts) == len(grads) == len(dx):
            raise ValueError("one gradient and one output for each part")
        with streams.on(self.device, stream):
            dweights = [None if p.weight is None else torch.empty(self.head_dim, dtype=self.dtype, device=self.device)
                        for p in parts]
            records = [self._record(*r) for r in zip(parts, grads, dx, dweights)]
            nbytes = B.basa_rope_bwd_workspace_bytes(records, self.params)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
            B.basa_rope_bwd(records, self.table, self.eps, ws, self.rope_params, self.params)
        return dweights
