"""Workloads of the norm before the output projection, its gradient and 8-bit activation checkpoints, with their plain forms.

Four passes over rows of activations (packed tokens by hidden size):

  norm    layer norm or RMS norm, forward (with the residual sum and the statistics that its gradient needs)
  grad    its backward pass from the 16- or 32-bit input: gradients of the input, the weight and the bias
  act8    activations kept in 8 bits and read back
  kept    a training step of the norm whose input is kept in 8 bits: the forward pass writes the checkpoint, the
          backward pass works from it

An 8-bit checkpoint holds blocks of 32 columns under one power of two, the smallest 2^e with
max |x| <= 127 * 2^e (int8) or 448 * 2^e (e4m3), e >= -126, and x / 2^e rounded to the nearest code, ties to even.

``listed()`` names fixed workloads and ``draw()`` draws others of the same ranges; ``prepare()`` makes a
workload's tensors from a seed, ``run()`` makes one pass, ``exact()`` gives the same outputs in 64 bits from
the definitions, ``work()`` the bytes and operations a pass cannot do without. With ``own`` false ``run()``
is elementary torch arithmetic in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

EPS = 1e-5
QMAX = {"int8": 127.0, "e4m3": 448.0}
EMAX = {"int8": 7, "e4m3": 9}  # 2^EMAX is the power of two above QMAX
BLOCK = 32


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # the last norm of one decoded token: latency
        dict(name="norm-1x6144-rms-bf16", op="norm", rows=1, cols=6144, kind="rms", dtype="bf16", wdtype="bf16",
             bias=False, residual=False, stats=False, masked=0.0, tight=False),
        # the indexer's key norm over a whole long context: many short rows, fp32 weights
        dict(name="norm-202752x128-layer-bf16", op="norm", rows=202752, cols=128, kind="layer", dtype="bf16",
             wdtype="f32", bias=True, residual=False, stats=True, masked=0.0, tight=False),
        # one chunk of the fused projection: the residual sum and its norm
        dict(name="norm-4096x6144-rms-res-bf16", op="norm", rows=4096, cols=6144, kind="rms", dtype="bf16",
             wdtype="bf16", bias=False, residual=True, stats=True, masked=0.0, tight=False),
        # a small fp32 step on an odd width whose rows start anywhere
        dict(name="grad-577x4097-layer-f32", op="grad", rows=577, cols=4097, kind="layer", dtype="f32", wdtype="f32",
             bias=True, residual=False, masked=0.0, tight=True),
        # the backward pass of one chunk of the fused projection
        dict(name="grad-4096x6144-rms-bf16", op="grad", rows=4096, cols=6144, kind="rms", dtype="bf16", wdtype="bf16",
             bias=False, residual=True, masked=0.0, tight=False),
        # a whole batch of response tokens, a quarter of them masked
        dict(name="grad-65536x6144-layer-bf16", op="grad", rows=65536, cols=6144, kind="layer", dtype="bf16",
             wdtype="f32", bias=True, residual=True, masked=0.25, tight=False),
        # the activations of a handful of tokens
        dict(name="act8-37x6144-int8-bf16", op="act8", rows=37, cols=6144, format="int8", dtype="bf16", tight=False),
        # fp32 activations of a ragged batch, the last block of a row cut off
        dict(name="act8-8191x2050-e4m3-f32", op="act8", rows=8191, cols=2050, format="e4m3", dtype="f32", tight=True),
        # the residual stream of a whole batch
        dict(name="act8-65536x6144-int8-bf16", op="act8", rows=65536, cols=6144, format="int8", dtype="bf16",
             tight=False),
        # a small step: a few short responses, the smallest model of the framework's workloads
        dict(name="kept-578x4096-layer-e4m3-f32", op="kept", rows=578, cols=4096, kind="layer", dtype="f32",
             wdtype="f32", bias=True, residual=False, format="e4m3", masked=0.0, tight=False),
        # a micro-batch of long responses, prompt tokens masked
        dict(name="kept-16384x6144-rms-int8-bf16", op="kept", rows=16384, cols=6144, kind="rms", dtype="bf16",
             wdtype="bf16", bias=False, residual=True, format="int8", masked=0.3, tight=False),
        # a whole batch of response tokens
        dict(name="kept-65536x6144-rms-int8-bf16", op="kept", rows=65536, cols=6144, kind="rms", dtype="bf16",
             wdtype="bf16", bias=False, residual=True, format="int8", masked=0.0, tight=False),
    ]


def draw(rng):
    op = rng.choice(["norm", "grad", "act8", "kept"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    cols = int(round(math.exp(rng.uniform(math.log(48), math.log(16384)))))
    if rng.random() < 0.5:
        cols = rng.choice([64, 128, 512, 1024, 1536, 2048, 4096, 5120, 6144, 7168, 8192, 12288, 16384])
    most = 3e8 if dtype == "bf16" else 1.5e8
    rows = int(round(math.exp(rng.uniform(0.0, math.log(min(250000.0, most / cols))))))
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, tight=rng.random() < 0.3)
    if op in ("act8", "kept"):
        case.update(format=rng.choice(["int8", "e4m3"]))
    if op != "act8":
        kind = rng.choice(["layer", "rms"])
        case.update(kind=kind, wdtype=rng.choice([dtype, "f32"]), bias=kind == "layer", residual=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.0, 0.1, 0.3]))
    if op == "norm":
        case.update(stats=rng.random() < 0.7)
    return case


# ---------------------------------------------------------------------------- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    R, C, dt, op = case["rows"], case["cols"], _dtype(case["dtype"]), case["op"]
    per16 = 8 if case["dtype"] == "bf16" else 4
    # rows start on 16-byte boundaries, as a framework's own buffers do, or follow one another without a gap
    ld = C if case["tight"] else (C + per16 - 1) // per16 * per16
    # hidden states: normal values whose channels differ in scale, a few of them by much
    loud = torch.exp(0.5 * torch.randn(C, generator=g, device=dev))
    loud[torch.rand(C, generator=g, device=dev) < 0.003] *= 20.0

    def rows(scale, shift=0.0):
        t = torch.empty((R, ld), dtype=dt, device=dev)
        step = max(1, (1 << 27) // ld)
        for r in range(0, R, step):
            n = min(R, r + step) - r
            part = torch.randn((n, C), generator=g, device=dev)
            t[r:r + n, :C] = part.mul_(scale).add_(shift)
        return t[:, :C]

    st = dict(case=dict(case), x=rows(loud, 0.1))
    if op == "act8":
        return st
    wt = _dtype(case["wdtype"])
    st["weight"] = (1.0 + 0.2 * torch.randn(C, generator=g, device=dev)).to(wt)
    st["bias"] = (0.1 * torch.randn(C, generator=g, device=dev)).to(wt) if case["bias"] else None
    st["mask"] = (torch.rand(R, generator=g, device=dev) >= case["masked"]).to(torch.uint8) if case["masked"] else None
    residual = case["residual"]
    st["residual"] = rows(0.5) if residual and op != "grad" else None  # what the sublayer before the norm adds
    if op != "norm":
        st["dy"] = rows(1e-3)
        st["dsummed"] = rows(1e-3) if residual else None  # the gradient that comes along the residual stream
    if op == "grad":  # the statistics that the forward pass kept
        mean, rstd = torch.empty(R, device=dev), torch.empty(R, device=dev)
        step = max(1, (1 << 26) // C)
        for r in range(0, R, step):
            h = st["x"][r:r + step].double()
            m = h.mean(1) if case["kind"] == "layer" else torch.zeros(len(h), dtype=torch.float64, device=dev)
            mean[r:r + step] = m
            rstd[r:r + step] = ((h - m[:, None]).square().mean(1) + EPS).rsqrt()
        st.update(mean=mean if case["kind"] == "layer" else None, rstd=rstd)
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    return (_library if own else _plain)[st["case"]["op"]](st)


def _off(st, *rows):
    """Zero rows where the mask is 0."""
    if st["mask"] is None:
        return rows
    on = st["mask"] != 0
    return [None if r is None else torch.where(on if r.dim() == 1 else on[:, None], r, 0) for r in rows]


def _plain_forward(st):
    """(y, h, mean, rstd) with y and the statistics in 32 bits, h in the type of x."""
    h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(st["x"].dtype)
    v = h.float()
    mean = None
    if st["case"]["kind"] == "layer":
        mean = v.mean(1)
        v = v - mean[:, None]
    rstd = torch.rsqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None] * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y, h, mean, rstd


def _plain_backward(st, h, mean, rstd):
    """h in 32 bits: the input of the norm or what its checkpoint stands for."""
    xhat = (h if mean is None else h - mean[:, None]) * rstd[:, None]
    dy = st["dy"].float()
    if st["mask"] is not None:
        xhat, dy = _off(st, xhat, dy)
    g = dy * st["weight"].float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd[:, None]
    if st["dsummed"] is not None:
        dx = dx + st["dsummed"].float()
    out = {"dx": _off(st, dx)[0].to(st["x"].dtype), "dweight": (dy * xhat).sum(0)}
    if st["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _plain_norm(st):
    y, h, mean, rstd = _plain_forward(st)
    y, mean, rstd, h = _off(st, y, mean, rstd, h)
    out = {"y": y.to(st["x"].dtype)}
    if st["residual"] is not None:
        out["summed"] = h
    if st["case"]["stats"]:
        out["rstd"] = rstd
        if mean is not None:
            out["mean"] = mean
    return out


def _plain_grad(st):
    return _plain_backward(st, st["x"].float(), st["mean"], st["rstd"])


def _power32(e):
    """2^e, -126 <= e <= 127, from its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_8bit(x, fmt):
    """What an 8-bit checkpoint of x stands for, in 32 bits."""
    R, C = x.shape
    pad = -C % BLOCK
    v = x.float()
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    v = v.view(R, -1, BLOCK)
    m, k = torch.frexp(v.abs().amax(2, keepdim=True))  # amax = m 2^k, m in [1/2, 1)
    e = k - EMAX[fmt] + (m > QMAX[fmt] / 2.0 ** EMAX[fmt]).int()
    e = torch.where(m == 0, -126, e.clamp_min(-126)).int()
    v = v * _power32(-e)
    v = torch.round(v) if fmt == "int8" else v.to(torch.float8_e4m3fn).float()
    return (v * _power32(e)).view(R, C + pad)[:, :C]


def _plain_act8(st):
    return {"x": _plain_8bit(st["x"], st["case"]["format"]).to(st["x"].dtype)}


def _plain_kept(st):
    y, h, mean, rstd = _plain_forward(st)
    out = {"y": _off(st, y)[0].to(st["x"].dtype)}
    del y
    if st["residual"] is not None:
        out["summed"] = _off(st, h)[0]
    out.update(_plain_backward(st, _plain_8bit(h, st["case"]["format"]), mean, rstd))
    return out


_plain = {"norm": _plain_norm, "grad": _plain_grad, "act8": _plain_act8, "kept": _plain_kept}


# ---------------------------------------------------------------------------- the same through the library

def _library_norm(st):
    from rl_post_loss_gb300 import capi
    case = st["case"]
    got = capi.layer_norm(st["x"], st["weight"], st["bias"], kind=case["kind"], eps=EPS, residual=st["residual"],
                          mask=st["mask"], want_stats=case["stats"])
    return {k: v for k, v in got.items() if v is not None}


def _library_backward(st, mean, rstd, **saved):
    from rl_post_loss_gb300 import capi
    got = capi.layer_norm_backward(st["dy"], st["weight"], mean, rstd, kind=st["case"]["kind"], mask=st["mask"],
                                   dsummed=st["dsummed"], want_dbias=st["bias"] is not None, **saved)
    return {k: v for k, v in got.items() if v is not None}


def _library_grad(st):
    return _library_backward(st, st["mean"], st["rstd"], x=st["x"])


def _library_act8(st):
    from rl_post_loss_gb300 import capi
    return {"x": capi.act8_unpack(capi.act8_pack(st["x"], format=st["case"]["format"]), dtype=st["x"].dtype)}


def _library_kept(st):
    from rl_post_loss_gb300 import capi
    case = st["case"]
    got = capi.layer_norm(st["x"], st["weight"], st["bias"], kind=case["kind"], eps=EPS, residual=st["residual"],
                          mask=st["mask"], want_stats=True, checkpoint=case["format"])
    out = {"y": got["y"]} if st["residual"] is None else {"y": got["y"], "summed": got["summed"]}
    out.update(_library_backward(st, got["mean"], got["rstd"], checkpoint=got["checkpoint"], dtype=st["x"].dtype))
    return out


_library = {"norm": _library_norm, "grad": _library_grad, "act8": _library_act8, "kept": _library_kept}


# ---------------------------------------------------------------------------- 64 bits, from the definitions

def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _log2_floor(x):
    """The whole part of log2 x, from the bits of a positive x."""
    return (x.view(torch.int64) >> 52) - 1023


def _exact_8bit(x, fmt):
    """The code nearest to x / 2^e, block by block, as the value it stands for; x in 64 bits."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        b = x[:, c:c + BLOCK]
        ratio = b.abs().amax(1, keepdim=True) / QMAX[fmt]
        e = _log2_floor(ratio.clamp_min(2.0 ** -200))
        e = (e + (ratio > _power64(e))).clamp_min(-126)
        q = b * _power64(-e)
        if fmt == "int8":
            q = q.round()
        else:  # 3 bits after the leading one, steps of 2^-9 below 2^-6
            grid = _power64(_log2_floor(q.abs().clamp_min(2.0 ** -6)) - 3)
            q = (q / grid).round() * grid
        out[:, c:c + BLOCK] = q * _power64(e)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    R, C, op, dt = case["rows"], case["cols"], case["op"], st["x"].dtype
    f64 = dict(dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // C)
    blocks = [slice(r, min(R, r + step)) for r in range(0, R, step)]
    if op == "act8":
        out = torch.empty((R, C), **f64)
        for b in blocks:
            out[b] = _exact_8bit(st["x"][b].double(), case["format"])
        return {"x": out}

    layer = case["kind"] == "layer"
    w = st["weight"].double()
    out = {}
    if op != "grad":
        out["y"] = torch.empty((R, C), **f64)
        if st["residual"] is not None:
            out["summed"] = torch.empty((R, C), **f64)
    if op == "norm" and case["stats"]:
        out["rstd"] = torch.empty(R, **f64)
        if layer:
            out["mean"] = torch.empty(R, **f64)
    if op != "norm":
        out.update(dx=torch.empty((R, C), **f64), dweight=torch.zeros(C, **f64))
        if st["bias"] is not None:
            out["dbias"] = torch.zeros(C, **f64)
    for b in blocks:
        on = st["mask"][b].double()[:, None] if st["mask"] is not None else torch.ones((b.stop - b.start, 1), **f64)
        h = st["x"][b].double()
        if st["residual"] is not None:
            h = (h + st["residual"][b].double()).to(dt).double()
            out["summed"][b] = h * on
        if op == "grad":
            rstd = st["rstd"][b].double()[:, None]
            mean = st["mean"][b].double()[:, None] if layer else 0.0
        else:
            mean = h.sum(1, keepdim=True) / C if layer else 0.0
            rstd = ((h - mean).pow(2).sum(1, keepdim=True) / C + EPS).pow(-0.5)
            y = (h - mean) * rstd * w
            out["y"][b] = (y if st["bias"] is None else y + st["bias"].double()) * on
            if "rstd" in out:
                out["rstd"][b] = (rstd * on)[:, 0]
                if layer:
                    out["mean"][b] = (mean * on)[:, 0]
        if op == "norm":
            continue
        if op == "kept":
            h = _exact_8bit(h, case["format"])
        xhat, dy = (h - mean) * rstd, st["dy"][b].double() * on
        out["dweight"] += torch.einsum("rc,rc->c", dy, xhat)
        if st["bias"] is not None:
            out["dbias"] += dy.sum(0)
        g = dy * w
        a = torch.einsum("rc,rc->r", g, xhat)[:, None] / C
        dx = rstd * (g - (g.sum(1, keepdim=True) / C if layer else 0.0) - xhat * a)
        out["dx"][b] = (dx if st["dsummed"] is None else dx + st["dsummed"][b].double()) * on
    return out


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    R, C, op = case["rows"], case["cols"], case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    kept = C + (C + BLOCK - 1) // BLOCK  # bytes of a row's 8-bit checkpoint
    if op == "act8":  # read, kept, read back, written
        return {"bytes": R * (2 * C * es + 2 * kept), "flops": R * C * 5}
    ws = 2 if case["wdtype"] == "bf16" else 4
    on = R * (1 - case["masked"])  # rows that are read; every row is written
    bias, res = int(case["bias"]), int(case["residual"])
    stats = 8 if case["kind"] == "layer" else 4
    forward = on * C * es * (1 + res) + R * C * es * (1 + res) + C * ws * (1 + bias) + R * (case["masked"] > 0)
    backward = on * C * es * (1 + res) + R * C * es + on * stats + C * (ws + 4 + 4 * bias) + R * (case["masked"] > 0)
    if op == "norm":
        return {"bytes": forward + R * stats * case["stats"], "flops": on * C * 8}
    if op == "grad":
        return {"bytes": backward + on * C * es, "flops": on * C * 14}
    return {"bytes": forward + backward + (R + on) * kept + R * stats, "flops": on * C * 26}
