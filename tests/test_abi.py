"""Host-only checks of the C ABI: the library loads, exports what include/basa.h
declares, and rejects invalid calls with the documented status before any CUDA
call (so these run without a GPU)."""
import ctypes
import os
import re

import pytest

from sparse_window_attention_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _declared():
    text = open(os.path.join(ROOT, "include", "basa.h")).read()
    return sorted(set(re.findall(r"^\w[\w\s\*]*?\b(basa_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_symbol_is_exported():
    names = _declared()
    assert set(names) == set(B.EXPORTED), names
    lib = ctypes.CDLL(os.path.join(ROOT, "sparse_window_attention_b200", "libbasa.so"))
    for n in names:
        assert hasattr(lib, n), n


def test_status_strings():
    for code, name in B.STATUS_NAMES.items():
        assert B.basa_status_string(code) == name
    assert B.basa_device_error_status(0) == B.BASA_OK
    assert B.basa_device_error_status(2) == 5
    assert B.basa_device_error_status(B.BASA_DEVERR_BAD_ROUTE) == 6
    assert B.basa_device_error_status(B.BASA_DEVERR_BAD_ROUTE | 1) == 6


def test_params_struct_layout_matches_header():
    # 18 ints, a pointer, two uint32, an int -> 72 + 8 + 8 + 4 (+4 padding) bytes on LP64
    assert ctypes.sizeof(B.basa_params) == 96
    assert B.basa_params.dev_err.offset == 72
    assert B.basa_params.route_radius.offset == 88


def _p(**kw):
    base = dict(B=1, heads=2, head_dim=128, grid=(1, 64, 64), window=(1, 16, 16), shift=(0, 8, 8), pool=(1, 8, 8),
                n_text=16, routed_k=0, dtype="bf16", route_radius=0)
    base.update(kw)
    return B.make_params(base["B"], base["heads"], base["head_dim"], base["grid"], base["window"], base["shift"],
                         base["pool"], base["n_text"], base["routed_k"], base["dtype"], route_radius=base["route_radius"])


FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced: every case fails its checks first


@pytest.mark.parametrize(
    "kw,status",
    [
        (dict(head_dim=96), 3),
        (dict(grid=(1, 60, 64)), 2),
        (dict(window=(1, 16, 20)), 2),
        (dict(shift=(0, 64, 0)), 2),
        (dict(shift=(0, -1, 0)), 2),
        (dict(pool=(1, 8, 0)), 2),
        (dict(pool=(1, 7, 8)), 2),
        (dict(n_text=-1), 1),
        (dict(routed_k=16), 1),  # nWin - 1 = 15
        (dict(routed_k=17, grid=(1, 128, 128)), 1),
        (dict(B=-1), 1),
        (dict(dtype=7), 1),
        (dict(route_radius=-1), 1),
        # a corner window of the 1x4x4 window grid has 3 neighbours within radius 1
        (dict(routed_k=4, route_radius=1), 1),
        (dict(routed_k=9, route_radius=2, grid=(1, 128, 128)), 1),
    ],
)
def test_invalid_params_rejected_before_launch(kw, status):
    p = _p(**kw)
    if kw.get("dtype") == 7:
        p.dtype = 7
    got = B.basa_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE if p.routed_k > 0 else None, FAKE, p,
                                 stream=0, check=False)
    assert got == status


def test_pointer_rules():
    p = _p()
    # pooled pointers must be given iff a pool patch is set
    assert B.basa_window_attn_fwd(FAKE, FAKE, FAKE, None, None, None, FAKE, p, stream=0, check=False) == 1
    # misaligned
    assert B.basa_window_attn_fwd(FAKE + 8, FAKE, FAKE, FAKE, FAKE, None, FAKE, p, stream=0, check=False) == 1
    # null output
    assert B.basa_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, p, stream=0, check=False) == 1
    # route ids must be given iff routed_k > 0
    pr = _p(routed_k=2)
    assert B.basa_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, pr, stream=0, check=False) == 1
    assert B.basa_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, p, stream=0, check=False) == 1
    # bfloat16 attention is built for head_dim 128 only
    assert B.basa_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, _p(head_dim=64), stream=0, check=False) == 3
    # pooling needs a patch; routing needs routed_k >= 1
    assert B.basa_pool_kv(FAKE, FAKE, FAKE, FAKE, _p(pool=(0, 0, 0)), stream=0, check=False) == 1
    assert B.basa_route_windows(FAKE, FAKE, FAKE, None, FAKE, p, stream=0, check=False) == 1
    assert B.basa_route_windows(FAKE, FAKE, FAKE + 2, None, FAKE, pr, stream=0, check=False) == 1


def test_empty_batch_is_a_no_op():
    for kw in (dict(B=0), dict(heads=0)):
        p = _p(**kw)
        assert B.basa_window_attn_fwd(None, None, None, None, None, None, None, p, stream=0, check=False) == 0
        assert B.basa_pool_kv(None, None, None, None, p, stream=0, check=False) == 0


def test_route_radius_limits_routed_k():
    """routed_k may reach the fewest candidates any window has under the radius."""
    assert B.basa_route_workspace_bytes(_p(routed_k=3, route_radius=1)) > 0
    assert B.basa_route_workspace_bytes(_p(routed_k=4, route_radius=1)) == 0
    # 8x8 window grid, radius 2: a corner sees 3 x 3 positions, itself included
    assert B.basa_route_workspace_bytes(_p(routed_k=8, route_radius=2, grid=(1, 128, 128))) > 0
    assert B.basa_route_workspace_bytes(_p(routed_k=9, route_radius=2, grid=(1, 128, 128))) == 0
    # the full video configuration: 4x4 spatial window grid, one routed window
    p = B.make_params(1, 12, 128, (21, 60, 104), (21, 15, 26), (0, 7, 13), (1, 4, 4), 0, 1, "bf16", route_radius=1)
    assert B.basa_route_workspace_bytes(p) == 2 * 12 * 16 * 128 * 4


def test_fused_pool_route_checks():
    """basa_pool_route: needs pooling and routing; shapes whose boxes would hold too
    many pieces (pool patch ∩ window) are refused before any launch."""
    pr = _p(routed_k=2)
    n = B.basa_pool_route_workspace_bytes(pr)
    # window means (2 x heads x 16 windows x 128 floats) + at least one partial slot each
    assert n >= 2 * (2 * 2 * 16 * 128 * 4)
    assert B.basa_pool_route_workspace_bytes(_p()) == 0  # no routing
    assert B.basa_pool_route_workspace_bytes(_p(routed_k=2, pool=(0, 0, 0))) == 0
    assert B.basa_pool_route(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, _p(), stream=0, check=False) == 1
    # a 32x32 patch cut by 2x2 windows into 256 cells: more than one CTA may hold
    big = _p(routed_k=2, pool=(1, 32, 32), window=(1, 2, 2), shift=(0, 1, 1))
    assert B.basa_pool_route_workspace_bytes(big) == 0
    assert B.basa_pool_route(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, big, stream=0, check=False) == 3
    # null and misaligned pointers
    assert B.basa_pool_route(FAKE, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, pr, stream=0, check=False) == 1
    assert B.basa_pool_route(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE + 4, pr, stream=0, check=False) == 1
    # the video configuration fits
    p = B.make_params(1, 12, 128, (21, 60, 104), (21, 15, 26), (0, 7, 13), (1, 4, 4), 0, 1, "bf16", route_radius=1)
    assert B.basa_pool_route_workspace_bytes(p) > 2 * 12 * 16 * 128 * 4


def test_branch_form_checks():
    p = _p()  # pool and 16 text rows, no routing
    call = lambda keys, pp=p: B.basa_window_attn_fwd_lse(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, keys, pp,
                                                         stream=0, check=False)
    assert call(0) == 1 and call(8) == 1
    nop = _p(pool=(0, 0, 0))
    assert B.basa_window_attn_fwd_lse(FAKE, FAKE, FAKE, None, None, None, FAKE, None, B.BASA_KEYS_POOLED, nop,
                                      stream=0, check=False) == 1
    assert call(B.BASA_KEYS_TEXT, _p(n_text=0)) == 1
    assert B.basa_window_attn_fwd_lse(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE + 2, B.BASA_KEYS_ALL, p,
                                      stream=0, check=False) == 1  # misaligned lse
    merge = lambda outs, lses, out=FAKE: B.basa_merge_branches(outs, lses, out, None, p, stream=0, check=False)
    assert merge([], []) == 1
    assert merge([FAKE] * 5, [FAKE] * 5) == 1
    assert merge([FAKE, None], [FAKE, FAKE]) == 1
    assert merge([FAKE, FAKE + 8], [FAKE, FAKE]) == 1
    assert merge([FAKE], [FAKE], out=None) == 1


def test_text_attn_checks():
    p = _p()
    assert B.basa_text_attn_fwd(FAKE, FAKE, FAKE, FAKE, None, _p(n_text=0), stream=0, check=False) == 1
    assert B.basa_text_attn_fwd(FAKE + 8, FAKE, FAKE, FAKE, None, p, stream=0, check=False) == 1
    assert B.basa_text_attn_fwd(FAKE, FAKE, FAKE, None, None, p, stream=0, check=False) == 1
    assert B.basa_text_attn_fwd(FAKE, FAKE, FAKE, FAKE, None, _p(head_dim=64), stream=0, check=False) == 3
    assert B.basa_text_attn_workspace_bytes(_p(n_text=0)) == 0


def test_backward_checks():
    pf = _p(dtype="f32")
    args = [FAKE] * 5 + [None] + [FAKE] * 7
    assert B.basa_window_attn_bwd(*args, _p(dtype="f32", head_dim=64), stream=0, check=False) == 3
    assert B.basa_window_attn_bwd(*args, _p(head_dim=64), stream=0, check=False) == 3  # bfloat16 needs 128
    bad = list(args)
    bad[12] = FAKE + 16  # bfloat16: the workspace must be 256-byte aligned
    assert B.basa_window_attn_bwd(*bad, _p(), stream=0, check=False) == 1
    bad[12] = None
    assert B.basa_window_attn_bwd(*bad, _p(), stream=0, check=False) == 1
    bad = list(args)
    bad[8] = None  # no dout
    assert B.basa_window_attn_bwd(*bad, pf, stream=0, check=False) == 1
    bad = list(args)
    bad[9] = FAKE + 4  # misaligned dq
    assert B.basa_window_attn_bwd(*bad, pf, stream=0, check=False) == 1
    # pooled gradients: 2 x heads x 64 patches x 128 floats
    assert B.basa_window_attn_bwd_workspace_bytes(pf) == 2 * 2 * 64 * 128 * 4
    # bfloat16 (computed on the host, the same on every device): per-token records
    # (2 heads x 4096 tokens x 16 B), chunk partials of the pooled and text key tiles
    # (2 heads x 2 tiles x 8 chunks of the 32 query tiles x [dK | dV] x 128 x 128 floats),
    # pooled-key gradients (2 x 2 heads x 64 x 128 floats)
    rec, part, pooled = 2 * 4096 * 16, 2 * 2 * 8 * 2 * 128 * 128 * 4, 2 * 2 * 64 * 128 * 4
    assert B.basa_window_attn_bwd_workspace_bytes(_p()) == rec + part + pooled


def test_route_workspace_bytes():
    p = _p(routed_k=2)
    assert B.basa_route_workspace_bytes(p) == 2 * 1 * 2 * 16 * 128 * 4
    assert B.basa_route_workspace_bytes(_p(head_dim=100)) == 0


def _bwd_chunks(wl, shift):
    """Chunk count of the bfloat16 backward's pooled/text key pass, read back from
    the workspace size (records + chunk partials + pooled-key gradients)."""
    p = B.make_params(wl.B, wl.heads, wl.d, wl.grid, wl.window, shift, wl.pool, wl.n_text, wl.routed_k, wl.dtype,
                      route_radius=wl.route_radius)
    bh = wl.B * wl.heads
    n = wl.grid[0] * wl.grid[1] * wl.grid[2]
    pt, ph, pw = wl.pool
    n_pool = (wl.grid[0] // pt) * (wl.grid[1] // ph) * (wl.grid[2] // pw)
    n_long = -(-n_pool // 128) + -(-wl.n_text // 128)
    up = lambda x: (x + 255) // 256 * 256
    part = B.basa_window_attn_bwd_workspace_bytes(p) - up(bh * n * 16) - up(bh * n_pool * 128 * 4 * 2)
    assert part % (bh * n_long * 2 * 128 * 128 * 4) == 0
    return part // (bh * n_long * 2 * 128 * 128 * 4), bh * n_long


def test_backward_chunking_fills_whole_waves():
    """The pooled/text pass splits each head's query tiles into the chunk count that
    minimises waves x (tiles per chunk + a CTA's fixed cost) on 148 SMs: one chunk
    (144 CTAs, one wave) at FLUX 2048^2 and 1024^2, six on Wan (144 CTAs), where
    the earlier rule of about two waves gave 2.9 and 2.1 waves."""
    from sparse_window_attention_b200 import synth

    for name, want in (("flux2k", 1), ("flux1k", 1), ("wan", 6)):
        wl = synth.WORKLOADS[name]
        chunks, units = _bwd_chunks(wl, synth.SHIFT_CYCLES[name][-1])
        assert chunks == want, (name, chunks)
        assert units * chunks <= 148, (name, units * chunks)  # one wave


def _rope(dt=16, dh=56, dw=56, pairs=0, theta=10000.0, **kw):
    return B.make_rope_params((dt, dh, dw), theta, pairs, **kw)


def _rope_tensor(x=FAKE, y=FAKE + (1 << 20), heads=2, rows=4, first_row=0, rotate=1, weight=None, dy=None, dweight=None):
    strides = {name: (2 * 4 * 128, 4 * 128, 128) for name in ("x", "y", "dy")}
    return B.rope_tensor(x, y, heads, rows, first_row, rotate, weight, dy, dweight, strides=strides)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=15), 1), (dict(dw=58), 1), (dict(dt=-2), 1), (dict(pairs=2), 1), (dict(theta=0.0), 1),
    (dict(theta=float("inf")), 1), (dict(origin=(0.0, float("nan"), 0.0)), 1),
])
def test_rope_params_rejected(kw, status):
    p = _p()
    assert B.basa_rope_fwd([_rope_tensor()], FAKE, 1e-6, _rope(**kw), p, stream=0, check=False) == status
    assert B.basa_rope_table(None, FAKE, _rope(**kw), p, stream=0, check=False) == status
    assert B.basa_rope_table_bytes(_rope(**kw), p) == 0


def test_rope_table_bytes():
    # pairs 8, 28, 28 of 1, 64, 64 positions and 64 pairs of 16 text rows, 8 bytes each
    assert B.basa_rope_table_bytes(_rope(), _p()) == 8 * (8 + 28 * 64 + 28 * 64 + 64 * 16)
    assert B.basa_rope_table(None, FAKE + 8, _rope(), _p(), stream=0, check=False) == 1
    assert B.basa_rope_table(FAKE + 2, FAKE, _rope(), _p(), stream=0, check=False) == 1


def test_rope_checks():
    p = _p()  # 64 x 64 grid, 16 text rows

    def fwd(*t, table=FAKE, eps=1e-6, pp=p):
        return B.basa_rope_fwd(list(t), table, eps, _rope(), pp, stream=0, check=False)

    T = _rope_tensor
    assert fwd() == 1 and fwd(*[T(rows=0)] * 9) == 1  # 1..8 tensors
    assert fwd(T(first_row=-1)) == 1 and fwd(T(heads=-1)) == 1 and fwd(T(rows=-1)) == 1 and fwd(T(rotate=2)) == 1
    assert fwd(T(first_row=4096 + 13)) == 2  # rows past the sequence
    assert fwd(T(), pp=_p(head_dim=96)) == 3
    assert fwd(T(x=0)) == 1 and fwd(T(y=0)) == 1 and fwd(T(x=FAKE + 8)) == 1 and fwd(T(y=FAKE + 8)) == 1
    assert fwd(T(weight=FAKE + 8)) == 1
    assert fwd(T(weight=FAKE), eps=0.0) == 1 and fwd(T(weight=FAKE), eps=float("nan")) == 1
    assert fwd(T(), table=None) == 1 and fwd(T(), table=FAKE + 8) == 1
    # in place needs the same strides; no tensor writes what another one uses
    assert fwd(T(y=FAKE, x=FAKE), T(x=FAKE, y=FAKE + (2 << 20))) == 1
    assert fwd(T(), T(x=FAKE + (3 << 20))) == 1  # the same output twice


def test_rope_strides_checked():
    p = _p()

    def fwd(xs, ys, x=FAKE, y=FAKE + (1 << 20), pp=p):
        t = B.rope_tensor(x, y, 2, 4, strides={"x": xs, "y": ys})
        return B.basa_rope_fwd([t], FAKE, 1e-6, _rope(), pp, stream=0, check=False)

    good = (1024, 512, 128)
    assert fwd((1024, 512, 132), good) == 1  # not a multiple of 16 bytes
    assert fwd((1024, -512, 128), good) == 1
    assert fwd((1024, 512, 1 << 60), good) == 1
    assert fwd(good, (1024, 512, 120)) == 1 and fwd(good, (1024, 384, 128)) == 1 and fwd(good, (1024, 0, 128)) == 1
    assert fwd(good, (1024, 128, 256), x=FAKE, y=FAKE) == 1  # in place with other strides


def test_rope_backward_checks():
    p = _p()

    def bwd(*t, ws=FAKE):
        return B.basa_rope_bwd(list(t), FAKE, 1e-6, ws, _rope(), p, stream=0, check=False)

    def T(**kw):
        return _rope_tensor(dy=kw.pop("dy", FAKE + (4 << 20)), **kw)

    dw = FAKE + (8 << 20)
    assert bwd(T(dy=None)) == 1
    assert bwd(T(dweight=dw)) == 1  # a gradient without its weight
    assert bwd(T(weight=FAKE, dweight=dw), ws=None) == 1 and bwd(T(weight=FAKE, dweight=dw), ws=FAKE + 8) == 1
    assert bwd(T(weight=FAKE, dweight=dw + 8)) == 1
    assert bwd(T(weight=FAKE, dweight=dw), T(y=FAKE + (2 << 20), weight=FAKE, dweight=dw)) == 1  # the same gradient twice
    assert bwd(T(x=0, weight=FAKE)) == 1
    # one block of 32 rows in groups of one unit each: 2 partial rows of 128 floats
    assert B.basa_rope_bwd_workspace_bytes([T(weight=FAKE, dweight=dw)], p) == 2 * 128 * 4
    assert B.basa_rope_bwd_workspace_bytes([T(weight=FAKE)], p) == 0
    assert B.basa_rope_bwd_workspace_bytes([T(weight=FAKE, dweight=dw, rows=0)], p) == 0


def test_rope_empty_is_a_no_op():
    for t, kw in ((_rope_tensor(x=0, y=0, rows=0), {}), (_rope_tensor(x=0, y=0, heads=0), {}), (_rope_tensor(x=0, y=0), dict(B=0))):
        assert B.basa_rope_fwd([t], None, 1e-6, _rope(), _p(**kw), stream=0, check=False) == 0


def _diff(lam=FAKE, weight=FAKE, gain=1.0, eps=1e-6):
    return B.make_diff_params(lam, weight, gain, eps)


def _diff_fwd(dp=None, p=None, q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, route=None, out=FAKE, pre=None, second=None,
              lse=None):
    return B.basa_diff_attn_fwd(q, k, v, kp, vp, route, dp or _diff(), out, pre, second, lse, p or _p(), stream=0,
                                check=False)


def test_diff_forward_checks():
    assert ctypes.sizeof(B.basa_diff_params) == 24 and B.basa_diff_params.gain.offset == 16
    for kw in (dict(head_dim=96), dict(head_dim=64), dict(B=1 << 15, heads=1 << 15)):
        assert _diff_fwd(p=_p(**kw)) == 3
    assert _diff_fwd(p=_p(window=(1, 16, 20))) == 2 and _diff_fwd(p=_p(shift=(0, 64, 0))) == 2
    for kw in (dict(lam=None), dict(lam=FAKE + 1), dict(weight=FAKE + 8), dict(gain=float("inf")), dict(eps=0.0),
               dict(eps=float("nan"))):
        assert _diff_fwd(_diff(**kw)) == 1, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(out=None), dict(route=FAKE),
               dict(q=FAKE + 8), dict(kp=FAKE + 8), dict(out=FAKE + 8), dict(pre=FAKE + 8), dict(second=FAKE + 8),
               dict(lse=FAKE + 2)):
        assert _diff_fwd(**kw) == 1, kw
    assert _diff_fwd(p=_p(routed_k=2)) == 1 and _diff_fwd(p=_p(routed_k=2), route=FAKE + 2) == 1
    assert _diff_fwd(p=_p(pool=(0, 0, 0))) == 1  # pooled keys without a pool patch
    f32 = _p(dtype="f32")
    assert _diff_fwd(_diff(lam=FAKE + 2), f32) == 1
    for heads in (dict(B=0), dict(heads=0)):
        assert _diff_fwd(_diff(None, None), _p(**heads), *[None] * 5) == 0


def test_diff_pool_checks():
    call = lambda p=None, **kw: B.basa_diff_pool_kv(*[kw.get(n, FAKE) for n in ("k", "v", "kp", "vp")], p or _p(), stream=0, check=False)  # noqa: E731
    assert call(_p(pool=(0, 0, 0))) == 1
    for name in ("k", "v", "kp", "vp"):
        assert call(**{name: None}) == 1 and call(**{name: FAKE + 8}) == 1
    assert call(_p(B=0), k=None) == 0


def test_diff_backward_checks():
    names = ("pre", "second", "lse", "dout", "dq", "dk", "dv", "dlam", "dweight", "ws")

    def call(dp=None, p=None, route=None, **kw):
        return B.basa_diff_attn_bwd(*[kw.get(n, FAKE) for n in ("q", "k", "v", "kp", "vp")], route, dp or _diff(),
                                    *[kw.get(n, FAKE) for n in names], p or _p(), stream=0, check=False)

    for name in ("q", "k", "v", "kp", "vp") + names:
        assert call(**{name: None}) == 1, name
    for name in ("q", "k", "v", "kp", "vp", "pre", "second", "dout", "dq", "dk", "dv", "dweight", "ws"):
        assert call(**{name: FAKE + 8}) == 1, name
    assert call(lse=FAKE + 2) == 1 and call(dlam=FAKE + 1) == 1 and call(ws=FAKE + 16) == 1
    assert call(_diff(weight=None)) == 1  # a gradient without its weight
    assert call(p=_p(head_dim=64)) == 3 and call(p=_p(routed_k=1)) == 1
    assert call(p=_p(window=(1, 1, 1), pool=(0, 0, 0), grid=(1, 128, 64), routed_k=1), kp=None, vp=None, route=FAKE) == 3
    # the gradients of nothing: there is no call that leaves weights' gradients unwritten
    assert call(p=_p(B=0)) == 1 and call(_diff(weight=None), _p(heads=0), dweight=None) == 0


def test_diff_backward_workspace():
    norm, plain = _diff(), _diff(weight=None)
    for dtype, size in (("bf16", 2), ("f32", 4)):
        p = _p(dtype=dtype)
        got = B.basa_diff_attn_bwd_workspace_bytes(norm, p), B.basa_diff_attn_bwd_workspace_bytes(plain, p)
        assert got[0] - got[1] == 2 * 4096 * 128 * size and got[1] > 0
    assert B.basa_diff_attn_bwd_workspace_bytes(norm, _p(head_dim=64)) == 0
    assert B.basa_diff_attn_bwd_workspace_bytes(norm, _p(head_dim=64, dtype="f32")) > 0
    assert B.basa_diff_attn_bwd_workspace_bytes(_diff(eps=0.0), _p()) == 0


def test_diff_text_checks():
    def call(p=None, dp=None, **kw):
        return B.basa_diff_text_attn_fwd(*[kw.get(n, FAKE) for n in ("q", "k", "v")], dp or _diff(), kw.get("out", FAKE),
                                         kw.get("ws", FAKE), p or _p(), stream=0, check=False)

    for name in ("q", "k", "v", "out", "ws"):
        assert call(**{name: None}) == 1 and call(**{name: FAKE + 8}) == 1, name
    assert call(_p(n_text=0)) == 1 and call(_p(head_dim=64)) == 3 and call(dp=_diff(lam=None)) == 1
    assert call(_p(B=0), q=None) == 0
    assert B.basa_diff_text_attn_workspace_bytes(_p(n_text=0)) == 0
    assert B.basa_diff_text_attn_workspace_bytes(_p(dtype="f32")) == 0


def test_backward_window_limits():
    """The bfloat16 backward names windows in 27 bits, and lists 4096 of them with routes."""
    plain = [FAKE] * 3 + [None] * 3 + [FAKE] * 7
    diff = [FAKE] * 3 + [None] * 3 + [_diff()] + [FAKE] * 10
    for grid, kw in (((1, 8192, 16385), {}), ((1, 64, 65), dict(routed_k=1))):
        p = _p(grid=grid, window=(1, 1, 1), shift=(0, 0, 0), pool=(0, 0, 0), **kw)
        assert B.basa_window_attn_bwd(*plain, p, stream=0, check=False) == 3
        assert B.basa_diff_attn_bwd(*diff, p, stream=0, check=False) == 3
