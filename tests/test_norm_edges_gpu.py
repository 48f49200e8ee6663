"""Forms of the norms that the other tests do not reach, against their definitions in 64 bits."""
import pytest
import torch

from rl_post_loss_gb300 import capi

import norm_helpers as nh

pytestmark = pytest.mark.gpu

EPS = 1e-5
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("rows,cols,kind,residual", [(20000, 620, "layer", False), (20000, 620, "rms", True), (20000, 916, "rms", False),
                                                     (20000, 916, "rms", True), (5000, 513, "layer", True), (700, 1100, "layer", False),
                                                     (300, 5121, "layer", True), (9000, 516, "rms", False)])
def test_fp32_rows_that_end_inside_a_vector(rows, cols, kind, residual):
    """The last vector of an fp32 row is read whole, past the 16-byte pieces that the row was copied in: a warp per row, a
    block per row, every stage of the ring."""
    g = torch.Generator().manual_seed(cols + rows)
    layout = "pad" if cols % 4 else "tight"  # on 16-byte boundaries either way
    x, x_gpu = nh.matrix(g, rows, cols, F32, layout, 1.5, 0.5)
    res, res_gpu = nh.matrix(g, rows, cols, F32, layout, 0.5) if residual else (None, lambda: None)
    dy, dy_gpu = nh.matrix(g, rows, cols, F32, layout, 0.1)
    w, b = 1 + 0.3 * torch.randn(cols, generator=g), 0.2 * torch.randn(cols, generator=g) if kind == "layer" else None
    wg, bg = w.cuda(), None if b is None else b.cuda()
    got = capi.layer_norm(x_gpu(), wg, bg, kind=kind, eps=EPS, residual=res_gpu(), want_stats=True)
    y, h, mean, rstd, e_y, e_mean, e_rstd = nh.forward64(x, w, b, kind, EPS, res)
    nh.assert_within("y", got["y"], y, e_y, F32)
    nh.assert_within("rstd", got["rstd"], rstd, e_rstd, F32)
    del y, e_y
    back = capi.layer_norm_backward(dy_gpu(), wg, got["mean"], got["rstd"], x=nh.on_gpu(h, layout), kind=kind, dsummed=res_gpu(),
                                    want_dbias=b is not None)
    dx, dw, db, e_dx, e_dw, e_db = nh.backward64(h, dy, w, None if b is None else got["mean"].cpu(), got["rstd"].cpu(), kind, res)
    nh.assert_within("dx", back["dx"], dx, e_dx, F32)
    nh.assert_within("dweight", back["dweight"], dw, e_dw)
    if b is not None:
        nh.assert_within("dbias", back["dbias"], db, e_db)
