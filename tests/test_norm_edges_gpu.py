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


def any_scale(rows, cols, fmt, at=0):
    """A checkpoint with every scale byte and every code, as a caller may make one; rows of codes `at` bytes off 16-byte boundaries."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    blocks = (cols + 31) // 32
    ld = (cols + at + 15) // 16 * 16
    codes = torch.randint(0, 256, (rows, ld), generator=g, device="cuda", dtype=torch.uint8)[:, at:at + cols]
    scales = (torch.arange(rows * blocks, device="cuda") % 256).to(torch.uint8).view(rows, blocks)
    return capi.Act8(codes, scales, fmt)


@pytest.mark.parametrize("rows,cols,at", [(300, 64, 0), (300, 128, 0), (300, 500, 0), (5000, 640, 0), (5000, 1000, 0), (60, 6144, 0), (60, 16384, 0), (60, 4097, 3),
                                          (60, 6145, 1)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_backward_pass_reads_what_unpacking_gives(rows, cols, at, kind, fmt):
    """With mean 0, rstd 1 and no weight the output made again is the norm's input itself: the same bits as act8_unpack's for
    every scale byte, those that act8_pack does not make among them (but what is past fp32's range stays infinite)."""
    a = any_scale(rows, cols, fmt, at)
    dy = torch.zeros((rows, cols), device="cuda")
    y = torch.empty_like(dy)
    mean = torch.zeros(rows, device="cuda") if kind == "layer" else None
    capi.layer_norm_backward(dy, None, mean, torch.ones(rows, device="cuda"), checkpoint=a, kind=kind, want_dweight=False, y=y)
    want = capi.act8_unpack(a, dtype=F32)
    assert nh.same(y.clamp(-torch.finfo(F32).max, torch.finfo(F32).max), want)
    known = torch.ones_like(want, dtype=torch.bool) if fmt == "int8" else (a.codes & 127) != 127
    exact = nh.values64(a.codes.cpu(), a.scales.cpu(), fmt, F32)
    assert nh.same(torch.where(known, want, torch.zeros_like(want)), torch.where(known.cpu(), exact, torch.zeros_like(exact)))


@pytest.mark.parametrize("rows,cols", [(40, 64), (40, 128), (3000, 1024), (40, 2048), (40, 8192)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [20, 84, 112])
def test_rows_of_one_large_value_from_a_checkpoint(rows, cols, fmt, power):
    """Their variance is 0 and everything is finite (the mean of 2^n equal powers of two is exact), so the gradient from
    the checkpoint, which holds them exactly, is the one from the rows."""
    x = torch.full((rows, cols), 2.0 ** power, device="cuda")
    dy = torch.randn((rows, cols), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = capi.layer_norm(x, want_stats=True, checkpoint=fmt, eps=EPS, device_status=status)
    assert nh.same(f["mean"], torch.full((rows,), 2.0 ** power)) and (f["y"] == 0).all()
    got = capi.layer_norm_backward(dy, None, f["mean"], f["rstd"], checkpoint=f["checkpoint"], want_dbias=True, device_status=status)
    assert int(status) == 0 and (got["dweight"] == 0).all()
    dx, _, db, e_dx, _, e_db = nh.backward64(x.cpu(), dy.cpu(), None, f["mean"].cpu(), f["rstd"].cpu(), "layer")
    nh.assert_within("dx", got["dx"], dx, e_dx, F32)
    nh.assert_within("dbias", got["dbias"], db, e_db)


@pytest.mark.parametrize("rows,cols", [(40, 128), (3000, 640), (40, 6144), (40, 6145)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_that_are_not_finite_through_a_checkpoint(rows, cols, kind, fmt):
    """A row that holds NaN or infinity: its gradient is not a number, it is reported, and the other rows have theirs; with
    the row masked nothing of it is seen."""
    bit = 1 << capi.CODES["RL_ERR_NONFINITE"]
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, dy = (torch.randn((rows, cols), generator=g, device="cuda") for _ in range(2))
    w = torch.randn(cols, generator=g, device="cuda")

    def both(x, mask=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = capi.layer_norm(x, w, kind=kind, want_stats=True, checkpoint=fmt, mask=mask, device_status=status)
        first = int(status)
        status.zero_()
        b = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], kind=kind, mask=mask, device_status=status)
        return b, first, int(status)

    keep = torch.ones(rows, dtype=torch.uint8, device="cuda")
    keep[7] = 0
    good, first, second = both(x, keep)
    assert first == 0 and second == 0
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = x.clone()
        bad[7, cols // 2] = value
        got, first, second = both(bad)
        assert first == bit and second == bit
        assert got["dx"][7].isnan().all() and nh.same(got["dx"][keep != 0], good["dx"][keep != 0])
        got, first, second = both(bad, keep)
        assert first == 0 and second == 0
        assert nh.same(got["dx"], good["dx"]) and nh.same(got["dweight"], good["dweight"])


@pytest.mark.parametrize("rows,cols", [(5000, 513), (5000, 600), (20000, 640), (5000, 776), (5000, 1000), (5000, 1024), (1300, 4096), (1000, 6144), (700, 8200),
                                       (9000, 128), (9000, 200), (2500, 512), (1000, 1031)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes_that_the_norm_writes_for_many_rows(rows, cols, fmt, dtype):
    """Bit for bit those of act8_pack for the same rows, in the kernels that calls of many rows take, with and without a
    mask, and (RMS, layer norm) in their two forms."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    layout = "tight" if cols % 8 == 0 or cols == 1031 else "pad"
    spread = torch.exp2(torch.randint(-20, 20, (1, (cols + 31) // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)[:, :cols]
    x, res = ((torch.randn((rows, cols), generator=g, device="cuda") * spread).to(dtype) for _ in range(2))
    h = (x.float() + res.float()).to(dtype)
    mask = (torch.rand(rows, generator=g, device="cuda") < 0.7).to(torch.uint8)
    mask[0], mask[-1] = 0, 1
    w = torch.ones(cols, device="cuda")
    for kind in ("layer", "rms"):
        for m in (None, mask):
            for r in (None, res):
                if r is None and m is None:
                    continue  # as with a mask
                got = capi.layer_norm(nh.on_gpu(x, layout), w, kind=kind, residual=None if r is None else nh.on_gpu(r, layout), mask=m, checkpoint=fmt)
                want = x if r is None else h
                if m is not None:
                    want = torch.where(m[:, None] != 0, want, torch.zeros((), dtype=dtype, device="cuda"))
                packed = capi.act8_pack(want, format=fmt)
                assert torch.equal(got["checkpoint"].codes, packed.codes) and torch.equal(got["checkpoint"].scales, packed.scales), (kind, m is None, r is None)


@pytest.mark.parametrize("cols", [4, 12, 20, 36, 60, 68, 132, 260, 388, 508])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_short_fp32_rows_that_end_inside_a_vector(cols, kind):
    """Rows of 16-byte pieces without gaps, whose last vector is read into the row behind it."""
    rows = 3001
    g = torch.Generator().manual_seed(cols)
    x, res, dy = (torch.randn((rows, cols), generator=g) for _ in range(3))
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g) if kind == "layer" else None
    wg, bg = w.cuda(), None if b is None else b.cuda()
    got = capi.layer_norm(x.cuda(), wg, bg, kind=kind, eps=EPS, residual=res.cuda(), want_stats=True)
    y, h, mean, rstd, e_y, e_mean, e_rstd = nh.forward64(x, w, b, kind, EPS, res)
    nh.assert_within("y", got["y"], y, e_y, F32)
    nh.assert_within("rstd", got["rstd"], rstd, e_rstd, F32)
    back = capi.layer_norm_backward(dy.cuda(), wg, got["mean"], got["rstd"], x=got["summed"], kind=kind, dsummed=res.cuda(), want_dbias=b is not None)
    dx, dw, db, e_dx, e_dw, e_db = nh.backward64(h, dy, w, None if b is None else got["mean"].cpu(), got["rstd"].cpu(), kind, res)
    nh.assert_within("dx", back["dx"], dx, e_dx, F32)
    nh.assert_within("dweight", back["dweight"], dw, e_dw)
    if b is not None:
        nh.assert_within("dbias", back["dbias"], db, e_db)


@pytest.mark.parametrize("own_stream", [True, False])
def test_two_threads_at_once(own_stream):
    """Calls of two threads, on a stream each and on one stream, with the workspaces that the binding keeps."""
    import threading
    rows, widths = 700, (640, 6144)
    g = torch.Generator(device="cuda").manual_seed(3)
    data = [[torch.randn((rows, c), generator=g, device="cuda").to(BF16) for _ in range(2)] + [torch.randn(c, generator=g, device="cuda")] for c in widths]

    def step(x, dy, w, stream=None):
        f = capi.layer_norm(x, w, want_stats=True, checkpoint="int8", stream=stream)
        b = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"], want_dbias=True, stream=stream)
        return [f["y"], b["dx"], b["dweight"], b["dbias"]]

    want = [[t.clone() for t in step(*d)] for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in widths]
    got, errors = [None, None], []

    def work(k):
        try:
            with torch.cuda.stream(streams[k if own_stream else 0]):
                got[k] = [step(*data[k]) for _ in range(30)]
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for k in range(2):
        assert all(nh.same(a, b) for run in got[k] for a, b in zip(run, want[k]))


def test_the_first_call_of_a_process_captured(tmp_path):
    """Kernels that no call has loaded yet, in a graph."""
    import subprocess
    import sys
    code = """
import torch
from rl_post_loss_gb300 import capi
x, dy = (torch.randn((300, 640), device="cuda") for _ in range(2))
w = torch.ones(640, device="cuda")
y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
mean, rstd = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
ws = torch.empty(capi.rl_loss_layer_norm_workspace_bytes(300, 640), dtype=torch.uint8, device="cuda")
a = capi.act8_empty(300, 640, "int8", x.device)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    capi.layer_norm(x, w, y=y, mean=mean, rstd=rstd, checkpoint=a)
    capi.layer_norm_backward(dy, w, mean, rstd, checkpoint=a, dx=dx, dweight=dw, workspace=ws)
graph.replay()
torch.cuda.synchronize()
f = capi.layer_norm(x, w, want_stats=True, checkpoint="int8")
b = capi.layer_norm_backward(dy, w, f["mean"], f["rstd"], checkpoint=f["checkpoint"])
assert torch.equal(y, f["y"]) and torch.equal(dx, b["dx"]) and torch.equal(dw, b["dweight"])
print("same")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    assert done.returncode == 0 and b"same" in done.stdout, done.stdout.decode()[-2000:]
