"""Layer norm and RMS norm on the GPU against their definitions in 64 bits (norm_helpers has the error bounds)."""
import pytest
import torch

from rl_post_loss_gb300 import capi

import norm_helpers as nh

pytestmark = pytest.mark.gpu

EPS = 1e-5
F32, BF16 = torch.float32, torch.bfloat16
NAME = {F32: "f32", BF16: "bf16"}

# both sides of every border between kernels and thread layouts, ragged last vectors and blocks, and the longest rows
COLS = [1, 2, 7, 8, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 384, 512, 513, 520, 768, 776, 1000, 1024, 1030, 1032, 1537, 2048,
        2056, 4096, 4097, 5120, 6144, 6150, 8192, 12288, 12296, 16000, 16384]


def cases():
    """Every width with some rows, types, layout and options; which ones goes by a fixed draw."""
    import random
    r = random.Random(11)
    out = []
    for cols in COLS:
        for _ in range(3 if cols < 8192 else 2):
            xt = r.choice([F32, BF16])
            out.append((cols, r.choice([1, 2, 3, 17, 64, 301, 700] if cols <= 1030 else [1, 3, 5, 40, 170] if cols <= 6150 else [1, 3, 40]),
                        r.choice(["layer", "rms"]), xt, r.choice([xt, xt, F32, BF16]), r.choice([F32, BF16]),
                        r.choice(["tight", "pad", "pad16", "offset"]), r.random() < 0.5, r.random() < 0.4, r.choice([None, "int8", "e4m3"])))
    # rows for all warps of the card, whose layouts differ from those of few rows
    for cols, rows in ((64, 30000), (128, 25000), (512, 9000), (640, 5000), (776, 5000), (1024, 5000), (2056, 2000), (4096, 1300), (6144, 1000)):
        out.append((cols, rows, "layer", BF16, BF16, F32, "pad", True, False, None))
        out.append((cols, rows, "rms", F32, F32, F32, "pad", False, True, "int8"))

    # fp32 rows of which a warp's part of shared memory holds one or two, from the rows themselves
    for cols, res in ((1024, False), (1024, True), (776, True), (640, True), (512, True), (256, True)):
        out.append((cols, 6000, "rms", F32, F32, F32, "pad", res, res, None))
        out.append((cols, 6000, "layer", F32, F32, F32, "pad16", res, False, None))
    return out


def case_id(c):
    return "%d-%d-%s-%s-%s-%s-%s%s%s%s" % (c[0], c[1], c[2], NAME[c[3]], NAME[c[4]], NAME[c[5]], c[6], "-res" if c[7] else "", "-mask" if c[8] else "",
                                           "-" + c[9] if c[9] else "")


@pytest.mark.parametrize("case", cases(), ids=case_id)
def test_forward_and_backward(case):
    cols, rows, kind, xt, yt, pt, layout, residual, masked, fmt = case
    g = torch.Generator().manual_seed(cols * 7 + rows)
    x, x_gpu = nh.matrix(g, rows, cols, xt, layout, 1.5, 0.7)
    res, res_gpu = nh.matrix(g, rows, cols, xt, layout, 0.5) if residual else (None, lambda: None)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(pt)
    b = (0.2 * torch.randn(cols, generator=g)).to(pt) if kind == "layer" else None
    mask = (torch.rand(rows, generator=g) < 0.7).to(torch.uint8) if masked else None
    dev_mask = None if mask is None else mask.cuda()
    wg, bg = w.cuda(), None if b is None else b.cuda()
    if masked:  # what masked rows hold does not matter
        xg = x_gpu()
        xg[mask.cuda() == 0] = float("nan")
    else:
        xg = x_gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    got = capi.layer_norm(xg, wg, bg, kind=kind, eps=EPS, residual=res_gpu(), mask=dev_mask, dtype=yt, want_stats=True, checkpoint=fmt,
                          device_status=status)
    y, h, mean, rstd, e_y, e_mean, e_rstd = nh.forward64(x, w, b, kind, EPS, res, mask)
    nh.assert_within("y", got["y"], y, e_y, yt)
    nh.assert_within("rstd", got["rstd"], rstd, e_rstd, F32)
    if kind == "layer":
        nh.assert_within("mean", got["mean"], mean, e_mean, F32)
    else:
        assert got["mean"] is None
    if residual:
        assert nh.same(got["summed"].cpu(), h)
    else:
        assert got["summed"] is None
    h64 = h
    if fmt:
        codes, scales = got["checkpoint"].codes.cpu(), got["checkpoint"].scales.cpu()
        if rows * cols < 300000:
            want = nh.pack64(h, fmt)
            assert nh.same(codes, want[0]) and nh.same(scales, want[1])
        h64 = nh.values64(codes, scales, fmt, F32)
    assert int(status) == 0

    # the backward pass, with the statistics and the input that the forward pass left
    dy, dy_gpu = nh.matrix(g, rows, cols, yt, layout, 0.1)
    ds, ds_gpu = nh.matrix(g, rows, cols, xt, layout, 0.1) if residual else (None, lambda: None)
    dyg, dsg = dy_gpu(), ds_gpu()
    if masked:
        dyg[mask.cuda() == 0] = float("inf")
        if residual:
            dsg[mask.cuda() == 0] = float("nan")
    again = torch.empty((rows, cols), dtype=yt, device="cuda")
    source = dict(checkpoint=got["checkpoint"], dtype=xt) if fmt else dict(x=got["summed"] if residual else xg)
    back = capi.layer_norm_backward(dyg, wg, got["mean"], got["rstd"], kind=kind, mask=dev_mask, dsummed=dsg, want_dbias=b is not None, bias=bg,
                                    y=again, device_status=status, **source)
    mean32 = got["mean"].cpu() if kind == "layer" else None
    dx, dw, db, e_dx, e_dw, e_db = nh.backward64(h64, dy, w, mean32, got["rstd"].cpu(), kind, ds, mask)
    nh.assert_within("dx", back["dx"], dx, e_dx, xt)
    nh.assert_within("dweight", back["dweight"], dw, e_dw)
    if b is not None:
        nh.assert_within("dbias", back["dbias"], db, e_db)
    else:
        assert back["dbias"] is None
    # y made again from h64 and the statistics: a difference, two products and a sum
    on = torch.ones(rows, 1, dtype=torch.float64) if mask is None else (mask != 0).double()[:, None]
    xh = (torch.where(on != 0, h64.double(), torch.zeros((), dtype=torch.float64)) - (0 if mean32 is None else mean32.double()[:, None])) * got["rstd"].cpu().double()[:, None]
    y2 = (xh * w.double() + (0 if b is None else b.double())) * on
    nh.assert_within("y again", again, y2, 6 * nh.U * ((xh * w.double()).abs() + y2.abs()), yt)
    assert int(status) == 0


def one(rows=37, cols=200, dtype=F32, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    return t(rows, cols), t(rows, cols), t(rows, cols), t(cols), t(cols)


@pytest.mark.parametrize("cols", [100, 520, 1000, 6144, 6145])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_without_parameters_and_parts_of_the_gradients(cols, kind):
    x, dy, _, w, b = one(30, cols)
    f = capi.layer_norm(x, kind=kind, want_stats=True)
    ones, zeros = torch.ones_like(w), torch.zeros_like(w)
    f1 = capi.layer_norm(x, ones, zeros, kind=kind)
    assert nh.same(f["y"], f1["y"])
    only_bias = capi.layer_norm(x, None, b, kind=kind)["y"]
    y, *_, = nh.forward64(x.cpu(), None, b.cpu(), kind, EPS)
    nh.assert_within("bias alone", only_bias, y, nh.forward64(x.cpu(), None, b.cpu(), kind, EPS)[4], F32)
    full = capi.layer_norm_backward(dy, None, f["mean"], f["rstd"], x=x, kind=kind, want_dbias=True)
    none = capi.layer_norm_backward(dy, None, f["mean"], f["rstd"], x=x, kind=kind, want_dweight=False)
    assert none["dweight"] is None and none["dbias"] is None
    bias = capi.layer_norm_backward(dy, None, f["mean"], f["rstd"], x=x, kind=kind, want_dweight=False, want_dbias=True)
    assert nh.same(bias["dbias"], full["dbias"]) and nh.same(bias["dx"], full["dx"])
    dx, dw, db, e_dx, e_dw, e_db = nh.backward64(x.cpu(), dy.cpu(), None, None if kind == "rms" else f["mean"].cpu(), f["rstd"].cpu(), kind)
    for name, got, want, e in (("dx", none["dx"], dx, e_dx), ("dw", full["dweight"], dw, e_dw), ("db", full["dbias"], db, e_db)):
        nh.assert_within(name, got, want, e, F32)


@pytest.mark.parametrize("cols", [128, 640, 6144, 4097])
def test_accumulate_adds(cols):
    x, dy, _, w, _ = one(50, cols)
    f = capi.layer_norm(x, w, want_stats=True)
    a = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], x=x, want_dbias=True)
    dw, db = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -1.0, device="cuda")
    capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], x=x, dweight=dw, dbias=db, accumulate=True)
    assert nh.same(dw, 2.0 + a["dweight"]) and nh.same(db, -1.0 + a["dbias"])
    with pytest.raises(ValueError, match="added to"):
        capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], x=x, accumulate=True)


@pytest.mark.parametrize("cols", [64, 100, 640, 2048, 6144, 6150])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(cols, dtype):
    x, dy, r, w, b = one(500, cols, dtype)
    f = capi.layer_norm(x, w, b, residual=r, want_stats=True)
    x1, r1 = x.clone(), r.clone()
    got = capi.layer_norm(x1, w, b, residual=r1, y=x1, summed=r1)
    assert got["y"] is x1 and nh.same(x1, f["y"]) and nh.same(r1, f["summed"])
    x2, r2 = x.clone(), r.clone()
    capi.layer_norm(x2, w, b, residual=r2, y=r2, summed=x2)
    assert nh.same(r2, f["y"]) and nh.same(x2, f["summed"])
    want = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], x=f["summed"], dsummed=r)
    for which in range(3):
        t = [dy.clone(), f["summed"].clone(), r.clone()]
        got = capi.layer_norm_backward(t[0], w, f["mean"], f["rstd"], x=t[1], dsummed=t[2], dx=t[which])
        assert nh.same(t[which], want["dx"]) and nh.same(got["dweight"], want["dweight"])
    t = [dy.clone(), f["summed"].clone()]  # y made again over dy, dx over x
    capi.layer_norm_backward(t[0], w, f["mean"], f["rstd"], x=t[1], dsummed=r, dx=t[1], y=t[0], bias=b)
    assert nh.same(t[1], want["dx"])
    # the same products and sums, but the difference from the rounded mean: near the forward's
    assert torch.allclose(t[0].float(), f["y"].float(), rtol=2 * nh.half_step(dtype), atol=1e-4)


@pytest.mark.parametrize("cols,rows", [(64, 20000), (200, 3000), (640, 5000), (6144, 700), (4097, 300)])
def test_results_repeat_bit_for_bit(cols, rows):
    x, dy, r, w, b = one(rows, cols, BF16)
    first = None
    for k in range(4):
        f = capi.layer_norm(x, w, b, residual=r, want_stats=True, checkpoint="int8")
        g = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], want_dbias=True, dsummed=r)
        now = [f["y"], f["summed"], f["mean"], f["rstd"], f["checkpoint"].codes, f["checkpoint"].scales, g["dx"], g["dweight"], g["dbias"]]
        if first is None:
            first = [t.clone() for t in now]
        assert all(nh.same(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("cols", [1, 64, 100, 640, 1000, 6144, 6145])
def test_nothing_beside_the_rows_is_written(cols):
    rows, guard = 21, 7
    x, dy, r, w, b = one(rows, cols, BF16)

    def room(t):
        big = torch.full((rows + 2, cols + guard), 9.0, dtype=t.dtype, device="cuda")
        return big, big[1:-1, :cols]

    by, y = room(x)
    bs, s = room(x)
    bdx, dx = room(x)
    ba = torch.full((rows + 2, cols + guard), 77, dtype=torch.uint8, device="cuda")
    bsc = torch.full((rows + 2, (cols + 31) // 32 + guard), 77, dtype=torch.uint8, device="cuda")
    a = capi.Act8(ba[1:-1, :cols], bsc[1:-1, :(cols + 31) // 32], "e4m3")
    f = capi.layer_norm(x, w, b, residual=r, y=y, summed=s, checkpoint=a, want_stats=True)
    dw = torch.full((cols + guard,), 5.0, device="cuda")
    capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=a, dx=dx, dweight=dw[:cols], dtype=BF16)
    plain = capi.layer_norm(x, w, b, residual=r, checkpoint="e4m3")
    assert nh.same(y, plain["y"]) and nh.same(s, plain["summed"])
    assert nh.same(a.codes, plain["checkpoint"].codes) and nh.same(a.scales, plain["checkpoint"].scales)
    for big in (by, bs, bdx):
        assert (big[0] == 9).all() and (big[-1] == 9).all() and (big[:, cols:] == 9).all()
    for big, n in ((ba, cols), (bsc, (cols + 31) // 32)):
        assert (big[0] == 77).all() and (big[-1] == 77).all() and (big[:, n:] == 77).all()
    assert (dw[cols:] == 5).all()


@pytest.mark.parametrize("cols", [128, 640, 6144, 6145])
def test_rows_that_are_not_finite_are_reported_and_stay_alone(cols):
    bit = 1 << capi.CODES["RL_ERR_NONFINITE"]
    x, dy, _, w, b = one(40, cols)
    good = capi.layer_norm(x, w, b, want_stats=True)
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        bad = x.clone()
        bad[7, cols // 2] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = capi.layer_norm(bad, w, b, want_stats=True, device_status=status)
        assert int(status) == bit
        keep = torch.arange(40) != 7
        assert nh.same(got["y"][keep], good["y"][keep])
        mask = torch.ones(40, dtype=torch.uint8, device="cuda")
        mask[7] = 0
        status.zero_()
        got = capi.layer_norm(bad, w, b, mask=mask, want_stats=True, device_status=status)
        assert int(status) == 0 and (got["y"][7] == 0).all() and float(got["rstd"][7]) == 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dy2 = dy.clone()
    dy2[3, 0] = float("nan")
    capi.layer_norm_backward(dy2, w, good["mean"], good["rstd"], x=x, device_status=status)
    assert int(status) == bit


@pytest.mark.parametrize("cols", [128, 640, 6144, 6145])
def test_every_row_masked(cols):
    x, dy, r, w, b = one(25, cols, BF16)
    mask = torch.zeros(25, dtype=torch.uint8, device="cuda")
    nan = torch.full_like(x, float("nan"))
    f = capi.layer_norm(nan, w, b, residual=nan, mask=mask, want_stats=True, checkpoint="int8")
    assert all((f[k] == 0).all() for k in ("y", "summed", "mean", "rstd")) and (capi.act8_unpack(f["checkpoint"]) == 0).all()
    g = capi.layer_norm_backward(nan, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], mask=mask, dsummed=nan, want_dbias=True)
    assert all((g[k] == 0).all() for k in ("dx", "dweight", "dbias"))


def test_broadcast_rows_are_refused_and_single_rows_take_any_stride():
    x, dy, _, w, b = one(4, 200)
    f = capi.layer_norm(x, w, b, want_stats=True)
    row = x[:1]
    for bad in (lambda: capi.layer_norm(row.expand(4, 200), w, b), lambda: capi.layer_norm(x, w, b, residual=row.expand(4, 200)),
                lambda: capi.layer_norm_backward(row.expand(4, 200), w, f["mean"], f["rstd"], x=x),
                lambda: capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], x=x, dsummed=row.expand(4, 200)),
                lambda: capi.act8_pack(row.expand(4, 200)), lambda: capi.layer_norm(x.as_strided((3, 200), (100, 1)), w, b)):
        with pytest.raises(ValueError, match="overlap"):
            bad()
    alone = x.as_strided((1, 200), (7, 1))
    assert nh.same(capi.layer_norm(alone, w, b)["y"], f["y"][:1])
    column = torch.randn((30, 9), device="cuda")[:, 4:5]
    assert nh.same(capi.layer_norm(column, kind="rms")["y"], capi.layer_norm(column.clone(), kind="rms")["y"])


def test_summed_without_a_residual():
    x, _, _, w, b = one(20, 640, BF16)
    s = torch.empty_like(x)
    got = capi.layer_norm(x, w, b, summed=s)
    assert got["summed"] is s and nh.same(s, x) and nh.same(got["y"], capi.layer_norm(x, w, b)["y"])


def test_no_rows():
    x = torch.empty((0, 640), device="cuda")
    w = torch.ones(640, device="cuda")
    f = capi.layer_norm(x, w, want_stats=True, checkpoint="int8")
    assert f["y"].shape == (0, 640) and f["checkpoint"].shape == (0, 640)
    g = capi.layer_norm_backward(x, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], want_dbias=True)
    assert g["dx"].shape == (0, 640) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    dw = torch.full((640,), 3.0, device="cuda")
    capi.layer_norm_backward(x, w, f["mean"], f["rstd"], x=x, dweight=dw, accumulate=True)
    assert (dw == 3).all()


@pytest.mark.parametrize("mean", [100.0, 3000.0])
@pytest.mark.parametrize("cols", [128, 6144])
def test_rows_far_from_zero(mean, cols):
    """The bounds hold where the mean is thousands of times the spread: a plain sum of squares would lose all digits."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((30, cols), generator=g) + mean
    w, b, dy = torch.ones(cols), torch.zeros(cols), torch.randn((30, cols), generator=g)
    got = capi.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, want_stats=True)
    y, _, m, rstd, e_y, e_mean, e_rstd = nh.forward64(x, w, b, "layer", EPS)
    nh.assert_within("y", got["y"], y, e_y, F32)
    nh.assert_within("mean", got["mean"], m, e_mean, F32)
    nh.assert_within("rstd", got["rstd"], rstd, e_rstd, F32)
    back = capi.layer_norm_backward(dy.cuda(), w.cuda(), got["mean"], got["rstd"], x=x.cuda())
    dx, dw, _, e_dx, e_dw, _ = nh.backward64(x, dy, w, got["mean"].cpu(), got["rstd"].cpu(), "layer")
    nh.assert_within("dx", back["dx"], dx, e_dx, F32)
    nh.assert_within("dweight", back["dweight"], dw, e_dw)


def test_rows_of_one_value():
    """Variance 0: rstd is eps^-1/2 and y the bias."""
    for cols in (128, 640, 6144, 6145):
        x = torch.full((5, cols), 3.25, device="cuda")
        b = torch.randn(cols, device="cuda")
        f = capi.layer_norm(x, None, b, eps=EPS, want_stats=True)
        assert nh.same(f["y"], b.expand(5, cols)) and torch.allclose(f["rstd"], torch.tensor(EPS ** -0.5, device="cuda"))


@pytest.mark.parametrize("layout", ["pad", "tight"])
def test_offsets_beyond_32_bits(layout):
    """Rows 2^30 elements apart: the third starts beyond 2^31."""
    cols, step = 6144, (1 << 30) + (8 if layout == "pad" else 3)
    buf = torch.empty(2 * step + cols + 64, dtype=BF16, device="cuda")
    x = buf.as_strided((3, cols), (step, 1))
    small, dy, r, w, b = one(3, cols, BF16)
    x.copy_(small)
    want = capi.layer_norm(small, w, b, want_stats=True, checkpoint="int8")
    got = capi.layer_norm(x, w, b, want_stats=True, checkpoint="int8")
    assert nh.same(got["y"], want["y"]) or layout == "tight"
    assert torch.allclose(got["y"].float(), want["y"].float(), rtol=2.0 ** -7, atol=1e-3)
    assert nh.same(got["checkpoint"].codes, want["checkpoint"].codes)
    capi.layer_norm(small, w, b, y=x)
    assert nh.same(x, want["y"])
    x.copy_(small)
    g1 = capi.layer_norm_backward(dy, w, want["mean"], want["rstd"], x=small)
    g2 = capi.layer_norm_backward(dy, w, want["mean"], want["rstd"], x=x, dx=x)
    assert g2["dx"] is x
    assert torch.allclose(x.float(), g1["dx"].float(), rtol=2.0 ** -7, atol=1e-5)
    del buf, x, g2


@pytest.mark.parametrize("cols", [128, 640, 6144, 6145])
def test_streams_and_graphs(cols):
    """On another stream than the current one; captured, and replayed on other contents, two graphs with a workspace each."""
    rows = 300
    x, dy, r, w, b = one(rows, cols, BF16)
    want = capi.layer_norm(x, w, b, residual=r, want_stats=True, checkpoint="int8")
    wg = capi.layer_norm_backward(dy, w, want["mean"], want["rstd"], checkpoint=want["checkpoint"], dsummed=r, want_dbias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = capi.layer_norm(x, w, b, residual=r, want_stats=True, checkpoint="int8", stream=side.cuda_stream)
    gr = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], dsummed=r, want_dbias=True, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert nh.same(f["y"], want["y"]) and nh.same(gr["dx"], wg["dx"]) and nh.same(gr["dweight"], wg["dweight"])

    graphs = []
    for k in range(2):
        st = dict(x=torch.zeros_like(x), dy=torch.zeros_like(dy), y=torch.empty_like(x), s=torch.empty_like(x), dx=torch.empty_like(x),
                  mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"), a=capi.act8_empty(rows, cols, "int8", x.device),
                  dw=torch.empty(cols, device="cuda"), db=torch.empty(cols, device="cuda"),
                  ws=torch.empty(capi.rl_loss_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            capi.layer_norm(st["x"], w, b, residual=r, y=st["y"], summed=st["s"], mean=st["mean"], rstd=st["rstd"], checkpoint=st["a"])
            capi.layer_norm_backward(st["dy"], w, st["mean"], st["rstd"], checkpoint=st["a"], dsummed=r, dx=st["dx"], dweight=st["dw"], dbias=st["db"],
                                     workspace=st["ws"])
            if k == 0:
                with pytest.raises(ValueError, match="workspace"):
                    capi.layer_norm_backward(st["dy"], w, st["mean"], st["rstd"], checkpoint=st["a"], dx=st["dx"], dweight=st["dw"])
        graphs.append((graph, st))
    for graph, st in graphs:
        st["x"].copy_(x)
        st["dy"].copy_(dy)
    for graph, st in graphs + graphs:
        st["dw"].zero_()
        graph.replay()
    torch.cuda.synchronize()
    for graph, st in graphs:
        assert nh.same(st["y"], want["y"]) and nh.same(st["s"], want["summed"]) and nh.same(st["a"].codes, want["checkpoint"].codes)
        assert nh.same(st["dx"], wg["dx"]) and nh.same(st["dw"], wg["dweight"]) and nh.same(st["db"], wg["dbias"])


def test_arguments_are_checked():
    x, dy, r, w, b = one(10, 200)
    st = capi.layer_norm(x, w, b, want_stats=True)
    for bad in (dict(residual=r.bfloat16()), dict(residual=r[:5]), dict(y=torch.empty((10, 199), device="cuda")), dict(mask=torch.ones(9, dtype=torch.uint8, device="cuda")),
                dict(mask=torch.ones(10, device="cuda")), dict(checkpoint=capi.act8_empty(10, 199)), dict(checkpoint="fp4"), dict(mean=torch.empty(10, dtype=torch.float64, device="cuda")),
                dict(y=torch.empty((10, 200), device="cuda"), dtype=BF16), dict(dtype=torch.float16), dict(residual=r.t()), dict(residual=r.cpu())):
        with pytest.raises(ValueError):
            capi.layer_norm(x, w, b, **bad)
    with pytest.raises(ValueError):
        capi.layer_norm(x, w.bfloat16(), b)
    with pytest.raises(ValueError):
        capi.layer_norm(x, w[:100])
    with pytest.raises(capi.RlLossError, match="UNSUPPORTED"):
        capi.layer_norm(torch.zeros((1, 16400), device="cuda"))
    with pytest.raises(capi.RlLossError, match="INVALID"):
        capi.layer_norm(x, eps=0.0)
    for bad in (dict(x=x[:9]), dict(x=x, dx=torch.empty((10, 200), dtype=BF16, device="cuda")), dict(x=x, dtype=BF16), dict(x=x, checkpoint=capi.act8_pack(x)),
                dict(checkpoint=capi.act8_pack(x[:9])), dict(x=x, dsummed=r[:, :100]), dict(x=x, dweight=torch.empty(100, device="cuda")),
                dict(x=x, y=torch.empty((10, 200), dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            capi.layer_norm_backward(dy, w, st["mean"], st["rstd"], **bad)
    with pytest.raises(ValueError):
        capi.layer_norm_backward(dy, w, None, st["rstd"], x=x)
    with pytest.raises(capi.RlLossError, match="CAPACITY"):
        capi.layer_norm_backward(dy, w, st["mean"], st["rstd"], x=x, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def at_offset(t, off, gap):
    """t's rows `gap` elements apart, the first one `off` elements into its memory, and that memory (7 elsewhere)."""
    rows, cols = t.shape
    flat = torch.full((rows * (cols + gap) + 64,), 7.0, dtype=torch.float32, device="cuda").to(t.dtype)
    at = flat[off:off + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]
    at.copy_(t)
    return at, flat


@pytest.mark.parametrize("cols", [1, 3, 8, 13, 100, 249, 255, 256, 257, 511, 520, 1030, 4097, 4104, 4600])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_rows_at_every_offset(cols, xt, yt):
    """Inputs and outputs that start at every offset in 32 bytes, each at another one, with and without a checkpoint whose own rows
    start anywhere; nothing beside an output's rows is written."""
    g = torch.Generator().manual_seed(cols)
    rows = 5
    x, r, ds = (torch.randn((rows, cols), generator=g).to(xt) for _ in range(3))
    dy = torch.randn((rows, cols), generator=g).to(yt)
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    mask = torch.tensor([1, 1, 0, 1, 1], dtype=torch.uint8)
    wg, bg, mg = w.cuda(), b.cuda(), mask.cuda()
    y, h, mean, rstd, e_y, e_mean, e_rstd = nh.forward64(x, w, b, "layer", EPS, r, mask)
    blocks = (cols + 31) // 32
    for k in range(16):
        gap = k % 3
        xg, rg, dyg, dsg = (at_offset(t, (k * m + 1) % 16, gap)[0] for t, m in ((x, 1), (r, 3), (dy, 5), (ds, 7)))
        out = {n: at_offset(torch.zeros((rows, cols), dtype=t), (k * m + o) % 16, gap)
               for n, t, m, o in (("y", yt, 1, 1), ("summed", xt, 9, 0), ("dx", xt, 1, 2), ("again", yt, 3, 3))}
        fmt = (None, "int8", "e4m3", "int8")[k % 4]
        ck = None
        if fmt:
            codes = torch.full((rows, cols + k), 9, dtype=torch.uint8, device="cuda")
            ck = capi.Act8(codes[:, k // 2:k // 2 + cols], torch.empty((rows, blocks + 1), dtype=torch.uint8, device="cuda")[:, :blocks], fmt)
        got = capi.layer_norm(xg, wg, bg, residual=rg, mask=mg, eps=EPS, y=out["y"][0], summed=out["summed"][0], want_stats=True, checkpoint=ck)
        nh.assert_within("y", got["y"], y, e_y, yt)
        assert nh.same(got["summed"], h)
        h64 = h
        if fmt:
            assert all(nh.same(p, q) for p, q in zip((ck.codes, ck.scales), nh.pack64(h, fmt)))
            h64 = nh.values64(ck.codes.cpu(), ck.scales.cpu(), fmt, F32)
            assert (codes[:, :k // 2] == 9).all() and (codes[:, k // 2 + cols:] == 9).all()
        source = dict(checkpoint=ck) if fmt else dict(x=got["summed"])
        back = capi.layer_norm_backward(dyg, wg, got["mean"], got["rstd"], mask=mg, dsummed=dsg, dx=out["dx"][0], want_dbias=True, bias=bg,
                                        y=out["again"][0], **source)
        dx, dw, db, e_dx, e_dw, e_db = nh.backward64(h64, dy, w, got["mean"].cpu(), got["rstd"].cpu(), "layer", ds, mask)
        nh.assert_within("dx", back["dx"], dx, e_dx, xt)
        nh.assert_within("dweight", back["dweight"], dw, e_dw)
        nh.assert_within("dbias", back["dbias"], db, e_db)
        for name, (view, flat) in out.items():
            view.fill_(7)
            assert (flat == 7).all(), name


@pytest.mark.parametrize("rows,cols,kind,dtype,fmt", [(30011, 1032, "rms", BF16, "int8"), (30011, 1032, "layer", BF16, None), (7400, 6144, "rms", F32, None),
                                                      (60003, 520, "rms", BF16, "e4m3"), (30003, 1024, "rms", F32, None), (30011, 1032, "layer", BF16, "e4m3")])
def test_rows_do_not_depend_on_the_blocks(rows, cols, kind, dtype, fmt):
    """Many rows with a residual go to more blocks than run at once, with a mask to no more: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r = (torch.randn((rows, cols), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.randn(cols, generator=g, device="cuda")
    b = torch.randn(cols, generator=g, device="cuda") if kind == "layer" else None
    few, many = (capi.layer_norm(x, w, b, kind=kind, residual=r, want_stats=True, checkpoint=fmt, mask=m)
                 for m in (torch.ones(rows, dtype=torch.uint8, device="cuda"), None))
    for name in ("y", "summed", "rstd") + (("mean",) if b is not None else ()):
        assert torch.equal(few[name], many[name]), name
    if fmt:
        assert torch.equal(few["checkpoint"].codes, many["checkpoint"].codes) and torch.equal(few["checkpoint"].scales, many["checkpoint"].scales)
    some = torch.arange(0, rows, 97)
    y, h, mean, rstd, e_y, _, _ = nh.forward64(x[some].cpu(), w.cpu(), None if b is None else b.cpu(), kind, EPS, r[some].cpu())
    nh.assert_within("y", many["y"][some], y, e_y, dtype)
