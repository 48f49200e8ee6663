"""The norms' and the 8-bit format's reference forms against differences and torch's own arithmetic, and the refusals of
the entry points (no GPU needed: an argument error returns before anything is launched)."""
import ctypes
import math

import pytest
import torch

from rl_post_loss_gb300 import capi

import norm_helpers as nh

F64 = torch.float64


# ---------------------------------------------------------------------------- the reference itself

@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_reference_gradient_is_that_of_differences(kind):
    g = torch.Generator().manual_seed(3)
    R, C, eps = 3, 7, 1e-3
    x, dy, ds = (torch.randn((R, C), generator=g, dtype=F64) for _ in range(3))
    w, b = torch.randn(C, generator=g, dtype=F64), torch.randn(C, generator=g, dtype=F64)

    def loss(x, w, b):
        mean = x.mean(1, keepdim=True) if kind == "layer" else 0.0
        d = x - mean
        y = d * ((d * d).mean(1, keepdim=True) + eps) ** -0.5 * w + b
        return float((y * dy).sum() + (x * ds).sum())

    mean = x.mean(1) if kind == "layer" else torch.zeros(R, dtype=F64)
    rstd = ((x - mean[:, None]).square().mean(1) + eps) ** -0.5
    dx, dw, db, *_ = nh.backward64(x, dy, w, mean, rstd, kind, ds)
    for t, grad in ((x, dx), (w, dw), (b, db)):
        for i in range(t.numel()):
            old = t.view(-1)[i].item()
            at = []
            for h in (1e-5, -1e-5):
                t.view(-1)[i] = old + h
                at.append(loss(x, w, b))
            t.view(-1)[i] = old
            assert abs((at[0] - at[1]) / 2e-5 - grad.view(-1)[i].item()) < 1e-8


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_reference_equals_torch(kind):
    g = torch.Generator().manual_seed(4)
    x, w, b = torch.randn((5, 33), generator=g, dtype=F64), torch.randn(33, generator=g, dtype=F64), torch.randn(33, generator=g, dtype=F64)
    y = nh.forward64(x, w, b, kind, 1e-5)[0]
    want = torch.nn.functional.layer_norm(x, (33,), w, b, 1e-5) if kind == "layer" else x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * w + b
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)


def test_e4m3_table_is_the_types():
    codes = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(nh.e4m3_values(), codes.view(torch.float8_e4m3fn).to(F64))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_reference_codes_are_the_nearest(fmt):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((20, 70), generator=g) * torch.exp(3 * torch.randn((20, 70), generator=g))
    codes, scales = nh.pack64(x, fmt)
    v = nh.values64(codes, scales, fmt, torch.float32)
    step = 2.0 ** (scales.to(F64) - 127).repeat_interleave(32, 1)[:, :70]
    # int8: half a step; e4m3: half a step of 3 bits, 2^-4 of the value, or of the smallest, 2^-10
    bound = step / 2 if fmt == "int8" else torch.maximum(x.to(F64).abs() / 16, step * 2.0 ** -10)
    assert ((v - x.to(F64)).abs() <= bound).all()
    assert (v.abs().amax(1) >= x.to(F64).abs().amax(1) * (1 - 1 / 16)).all()


# ---------------------------------------------------------------------------- refusals at the C entries

FAKE = 1 << 20  # an address that is never followed


def norm_config(**kw):
    base = dict(kind=0, cols=64, x_dtype=1, y_dtype=1, param_dtype=1, eps=1e-5)
    base.update(kw)
    return capi.rl_ln_config(*base.values())


def act8(**kw):
    base = dict(codes=FAKE, scales=FAKE, ld_codes=64, ld_scales=2, format=0)
    base.update(kw)
    return capi.rl_act8(*base.values())


def forward(cfg=None, rows=4, **kw):
    a = dict(x=FAKE, ld_x=64, residual=None, ld_residual=0, weight=FAKE, bias=None, mask=None, y=FAKE + 4096, ld_y=64, summed=None,
             ld_summed=0, checkpoint=None, mean=None, rstd=None, status=None, stream=None)
    a.update(kw)
    return capi.STATUS_NAMES[capi.load().rl_loss_layer_norm(norm_config() if cfg is None else cfg, rows, *a.values())]


def backward(cfg=None, rows=4, **kw):
    a = dict(dy=FAKE, ld_dy=64, x=FAKE + 4096, ld_x=64, checkpoint=None, weight=FAKE, bias=None, mask=None, mean=FAKE, rstd=FAKE,
             dsummed=None, ld_dsummed=0, dx=FAKE + 8192, ld_dx=64, dweight=FAKE, dbias=FAKE + 1024, accumulate=0, y=None, ld_y=0,
             workspace=FAKE, workspace_bytes=1 << 30, status=None, stream=None)
    a.update(kw)
    return capi.STATUS_NAMES[capi.load().rl_loss_layer_norm_backward(norm_config() if cfg is None else cfg, rows, *a.values())]


@pytest.mark.parametrize("kw,error", [
    (dict(cfg=norm_config(x_dtype=2)), "RL_ERR_DTYPE"), (dict(cfg=norm_config(y_dtype=-1)), "RL_ERR_DTYPE"),
    (dict(cfg=norm_config(param_dtype=7)), "RL_ERR_DTYPE"), (dict(rows=-1), "RL_ERR_SHAPE"),
    (dict(cfg=norm_config(cols=0)), "RL_ERR_SHAPE"), (dict(cfg=norm_config(cols=16385)), "RL_ERR_UNSUPPORTED"),
    (dict(cfg=norm_config(kind=2)), "RL_ERR_INVALID_ARG"), (dict(cfg=norm_config(eps=0.0)), "RL_ERR_INVALID_ARG"),
    (dict(cfg=norm_config(eps=math.nan)), "RL_ERR_INVALID_ARG"), (dict(cfg=norm_config(eps=math.inf)), "RL_ERR_INVALID_ARG"),
    (dict(x=None), "RL_ERR_INVALID_ARG"), (dict(y=None), "RL_ERR_INVALID_ARG"), (dict(ld_x=63), "RL_ERR_SHAPE"),
    (dict(ld_y=63), "RL_ERR_SHAPE"), (dict(residual=FAKE, ld_residual=63), "RL_ERR_SHAPE"),
    (dict(summed=FAKE, ld_summed=1), "RL_ERR_SHAPE"), (dict(x=FAKE + 1), "RL_ERR_ALIGNMENT"),
    (dict(weight=FAKE + 1), "RL_ERR_ALIGNMENT"), (dict(mean=FAKE + 2), "RL_ERR_ALIGNMENT"), (dict(status=FAKE + 2), "RL_ERR_ALIGNMENT"),
    (dict(checkpoint=act8(codes=None)), "RL_ERR_INVALID_ARG"), (dict(checkpoint=act8(format=2)), "RL_ERR_INVALID_ARG"),
    (dict(checkpoint=act8(ld_codes=63)), "RL_ERR_SHAPE"), (dict(checkpoint=act8(ld_scales=1)), "RL_ERR_SHAPE"),
    (dict(y=FAKE, ld_y=72), "RL_ERR_INVALID_ARG"), (dict(cfg=norm_config(y_dtype=0), y=FAKE), "RL_ERR_INVALID_ARG"),
    (dict(summed=FAKE + 4096, ld_summed=64), "RL_ERR_INVALID_ARG"), (dict(rows=0, x=None, y=None), "RL_OK"),
])
def test_forward_refusals(kw, error):
    assert forward(**kw) == error


@pytest.mark.parametrize("kw,error", [
    (dict(cfg=norm_config(x_dtype=2)), "RL_ERR_DTYPE"), (dict(rows=-1), "RL_ERR_SHAPE"),
    (dict(cfg=norm_config(cols=20000)), "RL_ERR_UNSUPPORTED"), (dict(cfg=norm_config(kind=-1)), "RL_ERR_INVALID_ARG"),
    (dict(accumulate=2), "RL_ERR_INVALID_ARG"), (dict(dweight=FAKE + 2), "RL_ERR_ALIGNMENT"),
    (dict(dbias=FAKE), "RL_ERR_INVALID_ARG"), (dict(dy=None), "RL_ERR_INVALID_ARG"), (dict(dx=None), "RL_ERR_INVALID_ARG"),
    (dict(rstd=None), "RL_ERR_INVALID_ARG"), (dict(mean=None), "RL_ERR_INVALID_ARG"), (dict(x=None), "RL_ERR_INVALID_ARG"),
    (dict(checkpoint=act8()), "RL_ERR_INVALID_ARG"), (dict(x=None, checkpoint=act8(scales=None)), "RL_ERR_INVALID_ARG"),
    (dict(x=None, checkpoint=act8(ld_codes=8)), "RL_ERR_SHAPE"), (dict(ld_dy=63), "RL_ERR_SHAPE"), (dict(ld_dx=0), "RL_ERR_SHAPE"),
    (dict(ld_x=-64), "RL_ERR_SHAPE"), (dict(dsummed=FAKE, ld_dsummed=2), "RL_ERR_SHAPE"), (dict(y=FAKE + 512, ld_y=3), "RL_ERR_SHAPE"),
    (dict(dx=FAKE, ld_dx=72), "RL_ERR_INVALID_ARG"), (dict(y=FAKE + 8192, ld_y=64), "RL_ERR_INVALID_ARG"),
    (dict(dsummed=FAKE + 512, ld_dsummed=64, y=FAKE + 512, ld_y=64), "RL_ERR_INVALID_ARG"), (dict(rstd=FAKE + 1), "RL_ERR_ALIGNMENT"),
    (dict(workspace=None), "RL_ERR_INVALID_ARG"), (dict(workspace=FAKE + 16), "RL_ERR_ALIGNMENT"),
    (dict(workspace_bytes=255), "RL_ERR_CAPACITY"), (dict(rows=0, accumulate=1, dy=None), "RL_OK"),
])
def test_backward_refusals(kw, error):
    assert backward(**kw) == error


@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("kw,error", [
    (dict(dtype=3), "RL_ERR_DTYPE"), (dict(rows=-1), "RL_ERR_SHAPE"), (dict(cols=0), "RL_ERR_SHAPE"),
    (dict(cols=(1 << 30) + 1), "RL_ERR_SHAPE"), (dict(x=None), "RL_ERR_INVALID_ARG"), (dict(a=None), "RL_ERR_INVALID_ARG"),
    (dict(a=act8(codes=None)), "RL_ERR_INVALID_ARG"), (dict(a=act8(format=-1)), "RL_ERR_INVALID_ARG"),
    (dict(a=act8(ld_codes=63)), "RL_ERR_SHAPE"), (dict(a=act8(ld_scales=1)), "RL_ERR_SHAPE"), (dict(ld=63), "RL_ERR_SHAPE"),
    (dict(x=FAKE + 1), "RL_ERR_ALIGNMENT"), (dict(rows=0, x=None), "RL_OK"),
])
def test_act8_refusals(pack, kw, error):
    a = dict(dtype=1, rows=4, cols=64, x=FAKE, ld=64, a=act8())
    a.update(kw)
    lib = capi.load()
    if pack:
        code = lib.rl_loss_act8_pack(a["dtype"], a["rows"], a["cols"], a["x"], a["ld"], a["a"], None)
    else:
        code = lib.rl_loss_act8_unpack(a["dtype"], a["rows"], a["cols"], a["a"], a["x"], a["ld"], None)
    assert capi.STATUS_NAMES[code] == error


def test_workspace_sizes():
    most = capi.rl_loss_layer_norm_max_cols()
    assert most == 16384
    for rows in (0, 1, 37, 100000, 2 ** 31 - 1):
        for cols in (1, 64, 513, 6144, most):
            n = capi.rl_loss_layer_norm_workspace_bytes(rows, cols)
            assert n >= 256 and n % 256 == 0 and n <= 64 << 20
    assert capi.rl_loss_layer_norm_workspace_bytes(5, most + 1) == 256


def test_python_refusals():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        capi.layer_norm(x)
    with pytest.raises(ValueError, match="kind"):
        capi.layer_norm(x, kind="batch")
    with pytest.raises(ValueError, match="kind"):
        capi.layer_norm_backward(x, None, None, None, x=x, kind="batch")
    with pytest.raises(ValueError, match="as x or as a checkpoint"):
        capi.layer_norm_backward(x, None, None, None)
    with pytest.raises(ValueError, match="int8"):
        capi.act8_empty(4, 64, "e5m2", "cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        capi.act8_pack(x)
    with pytest.raises(ValueError, match="column"):
        capi.act8_empty(4, 0, "int8", "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        capi.Act8(x, x, "int8")


def test_normed_projection_refuses_without_a_handle():
    lib = capi.load()
    assert lib.rl_loss_normed_projection_workspace_bytes(None) == 0
    code = lib.rl_loss_normed_projection_forward_backward(None, norm_config(), capi.rl_loss_final_norm(), None, 0, capi.rl_loss_inputs(),
                                                          None, 0, capi.rl_loss_outputs(), None, 0, None)
    assert capi.STATUS_NAMES[code] == "RL_ERR_INVALID_ARG"


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(capi.rl_ln_config) == 24 and ctypes.sizeof(capi.rl_act8) == 40 and ctypes.sizeof(capi.rl_loss_final_norm) == 64


class Tall:
    """A CUDA matrix of this shape as far as the binding's checks look (no memory: an address that is never followed)."""
    is_cuda, dtype, device = True, torch.float32, torch.device("cuda", 0)

    def __init__(self, rows, cols, dtype=torch.float32):
        self.shape, self.dtype = (rows, cols), dtype

    def dim(self):
        return 2

    def stride(self, k=None):
        return (self.shape[1], 1) if k is None else (self.shape[1], 1)[k]

    def data_ptr(self):
        return FAKE

    def get_device(self):
        return 0


@pytest.mark.parametrize("rows,cols", [(2 ** 31, 1), (2 ** 32 + 3, 64), (1, 2 ** 32 + 64)])
def test_sizes_past_32_bits_are_refused(rows, cols):
    """The C entries take 32-bit sizes; ctypes would pass the low 32 bits of a longer one without a word."""
    with pytest.raises(ValueError, match="2\\^31"):
        capi._matrix("x", Tall(rows, cols))
    with pytest.raises(ValueError, match="2\\^31"):
        capi.act8_empty(rows, cols, "int8", "meta")
    with pytest.raises(ValueError, match="2\\^31"):
        capi.Act8(Tall(rows, cols, torch.uint8), Tall(rows, (cols + 31) // 32, torch.uint8), "int8")
    assert capi._matrix("x", Tall(2 ** 31 - 1, 2))[0] == 2 ** 31 - 1
