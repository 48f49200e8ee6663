"""The fused projection with the last norm before it, and the norms, 8-bit checkpoints and the projection run together."""
import pytest
import torch

from rl_post_loss_gb300 import capi, synthetic

import norm_helpers as nh

pytestmark = pytest.mark.gpu

EPS = 1e-5


def batch(hidden, chunk, device="cuda"):
    return synthetic.make_projection_batch(device=device, prompts=2, group=4, length=24, hidden=hidden, vocab=600, chunk=chunk)


def setup(hidden=128, chunk=80, x_dtype=torch.bfloat16, kind="rms"):
    pb = batch(hidden, chunk)
    g = torch.Generator(device="cuda").manual_seed(5)
    T = pb.batch.num_tokens
    x = (torch.randn((T, hidden), generator=g, device="cuda") * 2 + 0.3).to(x_dtype)
    w = 1 + 0.2 * torch.randn(hidden, generator=g, device="cuda")
    b = 0.1 * torch.randn(hidden, generator=g, device="cuda") if kind == "layer" else None
    return pb, x, w, b


def by_parts(rl, pb, x, w, b, kind):
    """The same step as three calls."""
    f = capi.layer_norm(x, w, b, kind=kind, eps=EPS, dtype=torch.bfloat16, want_stats=True)
    out = capi.alloc_projection_outputs(pb)
    bt = pb.batch
    rl.fused_projection_forward_backward(f["y"], pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv, **out)
    g = capi.layer_norm_backward(out["dhidden"], w, f["mean"], f["rstd"], x=x, kind=kind, want_dbias=b is not None)
    return out, g


@pytest.fixture(scope="module", autouse=True)
def _lib():
    capi.load()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chunk", [80, 4096])
def test_equals_its_parts(chunk, x_dtype, kind):
    pb, x, w, b = setup(chunk=chunk, x_dtype=x_dtype, kind=kind)
    rl = capi.projection_handle(pb)
    want, g = by_parts(rl, pb, x, w, b, kind)
    out = {k: v for k, v in capi.alloc_projection_outputs(pb).items() if k != "dhidden"}
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    db = None if b is None else torch.empty_like(b)
    bt = pb.batch
    launches = rl.launch_count()

    def step(dx):
        rl.normed_projection_forward_backward(x, w, pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens,
                                              bt.rewards_or_adv, dx=dx, dnorm_weight=dw, norm_bias=b, dnorm_bias=db, kind=kind, eps=EPS, **out)
    step(dx)
    assert rl.launch_count() > launches
    for k in ("loss", "loss_f64", "logp", "entropy", "flags", "dw_lm"):
        assert nh.same(out[k], want[k]), k
    assert nh.same(dx, g["dx"])
    # the sums over rows are the chunks' here: the same terms in another order
    f = capi.layer_norm(x, w, b, kind=kind, eps=EPS, dtype=torch.bfloat16, want_stats=True)
    _, dw64, db64, _, e_dw, e_db = nh.backward64(x.cpu(), want["dhidden"].cpu(), w.cpu(), None if b is None else f["mean"].cpu(), f["rstd"].cpu(), kind)
    nh.assert_within("dnorm_weight", dw, dw64, e_dw)
    if b is not None:
        nh.assert_within("dnorm_bias", db, db64, e_db)
    assert rl.device_status() == 0
    # over x itself
    x2 = x
    keep = x.clone()
    step(x2)
    assert nh.same(x2, dx)
    x.copy_(keep)


def test_no_tokens_and_refusals():
    pb, x, w, b = setup()
    rl = capi.projection_handle(pb)
    bt = pb.batch
    out = {k: v for k, v in capi.alloc_projection_outputs(pb).items() if k != "dhidden"}
    dw = torch.full_like(w, 3.0)
    args = (bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv)
    kw = dict(dx=torch.empty_like(x), dnorm_weight=dw, **out)
    none = {k: v for k, v in out.items() if k in ("loss", "dw_lm")}
    rl.normed_projection_forward_backward(x[:0], w, pb.w, bt.targets[:0], bt.logp_old[:0], bt.logp_infer[:0], bt.mask[:0],
                                          torch.zeros_like(bt.cu_seqlens), bt.rewards_or_adv, dx=kw["dx"][:0], dnorm_weight=dw, **none)
    assert (dw == 0).all() and (out["dw_lm"] == 0).all()
    rl.device_status()
    with pytest.raises(ValueError):
        rl.normed_projection_forward_backward(x[:, :64], w, pb.w, *args, **kw)
    with pytest.raises(ValueError):
        rl.normed_projection_forward_backward(x, w.double(), pb.w, *args, **kw)
    with pytest.raises(capi.RlLossError, match="CAPACITY"):
        rl.normed_projection_forward_backward(x, w, pb.w, *args, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"), **kw)
    with pytest.raises(capi.RlLossError, match="INVALID"):
        rl.normed_projection_forward_backward(x, w, pb.w, *args, eps=-1.0, **kw)
    plain = capi.handle_for_batch(bt)
    with pytest.raises(capi.RlLossError, match="INVALID"):  # no projection_setup
        plain.normed_projection_forward_backward(x, w, pb.w, *args, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), **kw)


def test_captured_step():
    pb, x, w, b = setup(kind="layer")
    rl = capi.projection_handle(pb)
    bt = pb.batch
    out = {k: v for k, v in capi.alloc_projection_outputs(pb).items() if k != "dhidden"}
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(capi.load().rl_loss_normed_projection_workspace_bytes(rl.handle), dtype=torch.uint8, device="cuda")

    def step():
        rl.normed_projection_forward_backward(x, w, pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv, dx=dx,
                                              dnorm_weight=dw, norm_bias=b, dnorm_bias=db, kind="layer", workspace=ws, **out)
    step()
    want = [t.clone() for t in (out["loss"], out["dw_lm"], dx, dw, db)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t in (out["loss"], out["dw_lm"], dx, dw, db):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(nh.same(a, b) for a, b in zip(want, (out["loss"], out["dw_lm"], dx, dw, db)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_training_step_with_checkpoints(fmt):
    """Two norms with residual sums before the projection, their inputs kept in 8 bits; the gradients against automatic
    differentiation in 64 bits in which each norm's backward pass takes the kept input."""
    pb = batch(128, 4096)
    bt, T, H = pb.batch, pb.batch.num_tokens, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    emb = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    mix = (torch.randn((H, H), generator=g, device="cuda") / H ** 0.5).bfloat16()
    w1, w2 = (1 + 0.2 * torch.randn(H, generator=g, device="cuda") for _ in range(2))
    rl = capi.projection_handle(pb)

    # forward: h1 = emb, a = norm1(h1) mix, h2 = h1 + a, hidden = norm2(h2)
    f1 = capi.layer_norm(emb, w1, kind="rms", eps=EPS, want_stats=True, checkpoint=fmt)
    a = f1["y"] @ mix
    f2 = capi.layer_norm(a, w2, kind="rms", eps=EPS, residual=emb, want_stats=True, checkpoint=fmt)
    out = capi.alloc_projection_outputs(pb)
    rl.fused_projection_forward_backward(f2["y"], pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv, **out)
    b2 = capi.layer_norm_backward(out["dhidden"], w2, None, f2["rstd"], checkpoint=f2["checkpoint"], kind="rms", dtype=torch.bfloat16)
    y1 = torch.empty_like(emb)
    dy1 = b2["dx"] @ mix.t()
    b1 = capi.layer_norm_backward(dy1, w1, None, f1["rstd"], checkpoint=f1["checkpoint"], kind="rms", dsummed=b2["dx"], y=y1, dtype=torch.bfloat16)
    dmix = y1.float().t() @ b2["dx"].float()

    def back(kept, dy, w, rstd, ds=None):
        h = capi.act8_unpack(kept, dtype=torch.float32).cpu()
        return nh.backward64(h, dy.cpu(), w.cpu(), None, rstd.cpu(), "rms", None if ds is None else ds.cpu())

    dx2, dw2, _, e2, ew2, _ = back(f2["checkpoint"], out["dhidden"], w2, f2["rstd"])
    nh.assert_within("dx of the second norm", b2["dx"], dx2, e2, torch.bfloat16)
    nh.assert_within("dweight of the second norm", b2["dweight"], dw2, ew2)
    dx1, dw1, _, e1, ew1, _ = back(f1["checkpoint"], dy1, w1, f1["rstd"], b2["dx"])
    nh.assert_within("dx of the first norm", b1["dx"], dx1, e1, torch.bfloat16)
    nh.assert_within("dweight of the first norm", b1["dweight"], dw1, ew1)

    # what 8 bits cost: the whole step's gradients against those from the inputs themselves. A kept value is within 1 / 127 of
    # its block's largest (int8: half a step; 63.5 steps are less than the largest) or 2^-4 of itself (e4m3), so each gradient, a sum of products with
    # kept values and other factors that do not change, is off by no more than that times its terms' sizes.
    full2 = capi.layer_norm_backward(out["dhidden"], w2, None, f2["rstd"], x=f2["summed"], kind="rms")
    full1 = capi.layer_norm_backward(dy1, w1, None, f1["rstd"], x=emb, kind="rms", dsummed=b2["dx"])
    for kept, full, h, rstd, dy in ((b2, full2, f2["summed"], f2["rstd"], out["dhidden"]), (b1, full1, emb, f1["rstd"], dy1)):
        hf = h.float()
        top = hf.view(T, -1, 32).abs().amax(2).repeat_interleave(32, 1)
        off = top / 127 if fmt == "int8" else torch.maximum(hf.abs() * 2.0 ** -4, top * 2.0 ** -17)
        bound = ((dy.float() * rstd[:, None]).abs() * off).sum(0) * 1.001 + 1e-6 * full["dweight"].abs() + 1e-9
        assert ((kept["dweight"] - full["dweight"]).abs() <= bound).all()
    assert torch.isfinite(dmix).all()
