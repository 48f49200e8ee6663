"""8-bit activation checkpoints on the GPU: codes, scales and what they stand for, bit for bit from the definition."""
import math

import pytest
import torch

from rl_post_loss_gb300 import capi

import norm_helpers as nh

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(1, 1), (3, 31), (5, 32), (7, 33), (4, 100), (64, 64), (37, 257), (9, 2050), (2, 4097), (5, 6144), (300, 128), (1, 16400)]


def hard_rows(cols, dtype):
    """Rows at the ends of the formats' ranges."""
    big = torch.finfo(dtype).max
    rows = [torch.zeros(cols), -torch.zeros(cols), torch.full((cols,), 127.0), torch.full((cols,), 448.0), torch.full((cols,), -127.0),
            torch.linspace(-1, 1, cols) * 2.0 ** -130, torch.full((cols,), 2.0 ** -126), torch.linspace(0, 1, cols) * big, torch.full((cols,), big),
            torch.full((cols,), -big), torch.full((cols,), math.inf), torch.full((cols,), math.nan), torch.arange(cols) * 0.5 - 40,
            torch.arange(cols) * 2.0 ** -9 + 1, torch.full((cols,), 2.0 ** 100), torch.linspace(-448.5, 448.5, cols), torch.linspace(-127.4, 127.4, cols)]
    one = torch.randn(cols, generator=torch.Generator().manual_seed(2))
    for value in (math.nan, -math.inf, 1e30):
        r = one.clone()
        r[cols // 2] = value
        rows.append(r)
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("layout", ["tight", "pad", "pad16", "offset"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_codes_and_values(shape, dtype, fmt, layout):
    rows, cols = shape
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn((rows, cols), generator=g) * torch.exp(2 * torch.randn((rows, cols), generator=g))).to(dtype)
    if cols <= 2050:
        x = torch.cat([x, hard_rows(cols, dtype)])
    a = capi.act8_pack(nh.on_gpu(x, layout), format=fmt)
    assert a.shape == x.shape and a.nbytes == x.shape[0] * (cols + (cols + 31) // 32)
    codes, scales = nh.pack64(x, fmt)
    # a code of a block without a number is not told by the definition: its scale is
    free = (scales == 255).repeat_interleave(32, 1)[:, :cols]
    assert nh.same(a.scales.cpu(), scales)
    assert nh.same(torch.where(free, torch.zeros((), dtype=torch.uint8), a.codes.cpu()), torch.where(free, torch.zeros((), dtype=torch.uint8), codes))
    for out in (F32, BF16):
        got = capi.act8_unpack(a, dtype=out)
        want = nh.values64(codes, scales, fmt, out)
        assert nh.same(got.double(), want)
        buf = nh.on_gpu(torch.zeros(x.shape, dtype=out), layout)
        capi.act8_unpack(a, out=buf)
        assert nh.same(buf, got)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("cols", [33, 64, 2050, 6144])
def test_codes_in_a_callers_tensors(cols, fmt):
    """Codes and scales with rows at odd places, and nothing beside them written."""
    x = torch.randn((11, cols), device="cuda")
    blocks = (cols + 31) // 32
    big = torch.full((13, cols + 9), 200, dtype=torch.uint8, device="cuda")
    sc = torch.full((13, blocks + 3), 200, dtype=torch.uint8, device="cuda")
    a = capi.Act8(big[1:-1, 1:1 + cols], sc[1:-1, 2:2 + blocks], fmt)
    capi.act8_pack(x, out=a)
    want = capi.act8_pack(x, format=fmt)
    assert nh.same(a.codes, want.codes) and nh.same(a.scales, want.scales)
    assert nh.same(capi.act8_unpack(a, dtype=F32), capi.act8_unpack(want, dtype=F32))
    assert (big[0] == 200).all() and (big[-1] == 200).all() and (big[:, 0] == 200).all() and (big[:, 1 + cols:] == 200).all()
    assert (sc[0] == 200).all() and (sc[-1] == 200).all() and (sc[:, :2] == 200).all() and (sc[:, 2 + blocks:] == 200).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 2, 5, 7, 8, 9, 31, 33, 63, 100, 257])
def test_rows_at_every_offset(cols, dtype):
    """Rows that start at every offset in 32 bytes, read and written, with nothing beside them read as theirs or written."""
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn((9, cols), generator=g) * torch.exp2(torch.randint(-30, 30, (9, (cols + 31) // 32), generator=g).float()).repeat_interleave(32, 1)[:, :cols]).to(dtype)
    for fmt in ("int8", "e4m3"):
        codes, scales = nh.pack64(x, fmt)
        want = nh.values64(codes, scales, fmt, dtype)
        for off in range(16):
            for gap in (0, 1, 5):
                ld = cols + gap
                flat = torch.full((9 * ld + 32,), math.nan, dtype=dtype, device="cuda")
                at = flat[off:off + 9 * ld].view(9, ld)[:, :cols]
                at.copy_(x)
                a = capi.act8_pack(at, format=fmt)
                assert nh.same(a.codes.cpu(), codes) and nh.same(a.scales.cpu(), scales)
                flat.fill_(7)
                capi.act8_unpack(a, out=at)
                assert nh.same(at.double().cpu(), want)
                at.fill_(7)
                assert (flat == 7).all()


def test_packing_what_was_read_back_changes_nothing():
    x = torch.randn((50, 1000), device="cuda", dtype=BF16) * 30
    for fmt in ("int8", "e4m3"):
        once = capi.act8_unpack(capi.act8_pack(x, format=fmt))
        assert nh.same(capi.act8_unpack(capi.act8_pack(once, format=fmt)), once)


def test_offsets_beyond_32_bits():
    cols, step = 4096, (1 << 31) + 64
    buf = torch.empty(step + cols, dtype=torch.uint8, device="cuda")
    x = torch.randn((2, cols), device="cuda")
    want = capi.act8_pack(x)
    a = capi.Act8(buf.as_strided((2, cols), (step, 1)), torch.empty((2, cols // 32), dtype=torch.uint8, device="cuda"), "int8")
    capi.act8_pack(x, out=a)
    assert nh.same(a.codes, want.codes) and nh.same(a.scales, want.scales)
    assert nh.same(capi.act8_unpack(a), capi.act8_unpack(want))


def test_graphs_streams_and_no_rows():
    x = torch.randn((40, 1000), device="cuda", dtype=BF16)
    a, out = capi.act8_empty(40, 1000, "e4m3", x.device), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        capi.act8_pack(x, out=a)
        capi.act8_unpack(a, out=out)
    for k in range(2):
        x.normal_()
        graph.replay()
        assert nh.same(out, capi.act8_unpack(capi.act8_pack(x, format="e4m3")))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = capi.act8_unpack(capi.act8_pack(x, format="e4m3", stream=side.cuda_stream), stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert nh.same(got, out)
    empty = capi.act8_pack(x[:0])
    assert empty.shape == (0, 1000) and empty.codes.shape == (0, 1000) and capi.act8_unpack(empty).shape == (0, 1000)


def test_arguments_are_checked():
    x = torch.randn((4, 100), device="cuda")
    a = capi.act8_pack(x)
    for call in (lambda: capi.act8_pack(x, out=capi.act8_empty(4, 99)), lambda: capi.act8_pack(x.half()), lambda: capi.act8_pack(x.t()),
                 lambda: capi.act8_pack(x, format="int4"), lambda: capi.act8_unpack(a, dtype=torch.float16), lambda: capi.act8_unpack(a, out=x[:3]),
                 lambda: capi.act8_unpack(a, out=x, dtype=BF16), lambda: capi.Act8(a.codes, a.scales[:, :3], "int8"),
                 lambda: capi.Act8(a.codes.int(), a.scales, "int8"), lambda: capi.Act8(a.codes, a.scales, "int4")):
        with pytest.raises(ValueError):
            call()
