"""Layer norm with its vectors between the rows of its matrices: one wide buffer holds all of them."""
import pytest
import torch

from tests import synthetic as syn

pytestmark = pytest.mark.gpu

F32 = torch.float32


def test_vectors_between_the_rows(cuda):
    import invariant_moe_gb300 as bm
    M, H, LD = 5, 37, 80
    x, w, b, dy = (syn.normal(s, 1.0, i, F32).to(cuda) for i, s in enumerate(((M, H), (H,), (H,), (M, H))))
    y, mean, rstd = bm.bi_layer_norm_train(x, w, b)
    dx, dw, db = bm.bi_layer_norm_backward(dy, x, w, mean, rstd)
    wide = torch.full((M, LD), 9.0, device=cuda)
    rows, gap = wide[:, :H], [wide[i, H:2 * H] for i in range(M)]
    gap[0].copy_(w)
    gap[1].copy_(b)
    m, r = gap[2][:M], gap[3][:M]
    bm.bi_layer_norm_train(x, gap[0], gap[1], out=rows, mean=m, rstd=r)
    assert all(torch.equal(u, v) for u, v in ((rows, y), (m, mean), (r, rstd), (gap[0], w), (gap[1], b)))
    bm.bi_layer_norm_backward(dy, x, gap[0], m, r, dx=rows, dweight=gap[1], dbias=gap[4])
    assert all(torch.equal(u, v) for u, v in ((rows, dx), (gap[1], dw), (gap[4], db), (gap[0], w), (m, mean)))
    assert bool((wide[:, 2 * H:] == 9).all())
