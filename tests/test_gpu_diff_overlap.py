"""Differential attention into an output that shares memory with an input: refused, as other
rows' keys and queries are read while it is written."""
import pytest
import torch

from tests.test_gpu_diff import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_output_over_an_input_is_refused(dtype):
    c = Case("overlap", dtype, 1, 2, 128, (1, 16, 16), (1, 8, 8), (0, 4, 4))
    q, k, v, lam, w, _, _ = c.inputs()
    layer = c.layer()
    ref = layer.attention(q, k, v, lam, c.shift, w)
    n = ref.numel()
    for out in (v, q.view(-1)[n:].view_as(ref), k.view(-1)[n // 2 : n // 2 + n].view_as(ref)):
        with pytest.raises(ValueError):
            layer.attention(q, k, v, lam, c.shift, w, out=out)
    # next to the inputs in one buffer is no overlap
    room = torch.cat([v.flatten(), torch.zeros(n, dtype=v.dtype, device="cuda"), k.flatten()])
    v1, out, k1 = room[:n].view_as(v), room[n : 2 * n].view_as(ref), room[2 * n :].view_as(k)
    assert torch.equal(layer.attention(q, k1, v1, lam, c.shift, w, out=out), ref) and out.data_ptr() == room[n:].data_ptr()
