"""Layouts that interleave in memory without meeting: rotary calls that are accepted, and give
the bits of the same call on buffers of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_shared_buffers(dtype):
    from sparse_window_attention_b200.rope import GridRope, RopePart

    B, h, hk, d, n, text = 2, 4, 2, 128, 15, 7
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    rope = GridRope(d, (1, 3, 5), (16, 56, 56), batch=B, n_text=text, text_pos=rnd(text, 3).float(), dtype=dtype)
    w = (1 + 0.2 * rnd(d).float()).to(dt)
    # one record a batch entry: n rows of q, k, v heads, then text rows of the same
    record = rnd(B, n + text, h + 2 * hk, d)
    cut = lambda t, a, b, rows: t[:, rows, a:b].permute(0, 2, 1, 3)  # noqa: E731
    image, words = slice(0, n), slice(n, None)
    heads = ((0, h), (h, h + hk), (h + hk, h + 2 * hk))

    def parts(x, y):
        p = []
        for (a, b), rot in zip(heads, (True, True, False)):
            weight = w if rot else None
            p += [RopePart(cut(x, a, b, image), cut(y, a, b, image), weight, 0, rot),
                  RopePart(cut(x, a, b, words), cut(y, a, b, words), weight, n, rot)]
        return p

    want = torch.empty_like(record)  # token-major again: every part's rows between the others'
    rope.forward(parts(record, want))
    alone = [RopePart(p.x.clone(), torch.empty_like(p.x.contiguous()), *p[2:]) for p in parts(record, want)]
    for p, q in zip(parts(record, want), alone):
        rope.forward([q])
        assert torch.equal(p.y, q.y)
    # in place, every slice on itself
    same = record.clone()
    rope.forward(parts(same, same))
    assert torch.equal(same, want)
    # gradients: written over the output gradients, and the same by themselves
    dy = rnd(*record.shape)
    into = dy.clone()
    grads = [p.y for p in parts(record, into)]
    dw = rope.backward(parts(record, want), grads, grads)
    for i, (p, q) in enumerate(zip(parts(record, dy), alone)):
        dx = torch.empty_like(q.y)
        one = rope.backward([q], [p.y.clone()], [dx])
        assert torch.equal(dx, grads[i])
        assert (one[0] is None) == (dw[i] is None)
        if one[0] is not None:
            assert (one[0].float() - dw[i].float()).abs().max() <= torch.finfo(dt).eps * dw[i].float().abs().max()
