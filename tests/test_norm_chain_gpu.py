"""Norms with 8-bit checkpoints and the projection as one step, against automatic differentiation of the whole chain in 64 bits."""
import pytest
import torch

from rl_post_loss_gb300 import capi, synthetic

import norm_helpers as nh

pytestmark = pytest.mark.gpu

EPS = 1e-5
F64 = torch.float64
BF16 = torch.bfloat16


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_gradients_of_a_step_are_those_of_the_chain(fmt):
    """h1 = emb, y1 = norm1(h1), h2 = emb + y1 mix, hidden = norm2(h2): the gradients of emb, mix and both weights for the
    projection's dhidden. In the chain each norm's input is what its checkpoint holds, with the forward pass's rstd, and
    that of rstd follows rstd' = -rstd^3 h / C there; nothing else is rounded."""
    H = 128
    pb = synthetic.make_projection_batch(device="cuda", prompts=2, group=4, length=24, hidden=H, vocab=600, chunk=4096)
    bt, T = pb.batch, pb.batch.num_tokens
    g = torch.Generator(device="cuda").manual_seed(9)
    emb = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    mix = (torch.randn((H, H), generator=g, device="cuda") / H ** 0.5).to(BF16)
    w1, w2 = (1 + 0.2 * torch.randn(H, generator=g, device="cuda") for _ in range(2))
    rl = capi.projection_handle(pb)

    f1 = capi.layer_norm(emb, w1, kind="rms", eps=EPS, want_stats=True, checkpoint=fmt)
    a = (f1["y"].float() @ mix.float()).to(BF16)
    f2 = capi.layer_norm(a, w2, kind="rms", eps=EPS, residual=emb, want_stats=True, checkpoint=fmt)
    out = capi.alloc_projection_outputs(pb)
    rl.fused_projection_forward_backward(f2["y"], pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv, **out)
    dhidden = out["dhidden"]
    b2 = capi.layer_norm_backward(dhidden, w2, None, f2["rstd"], checkpoint=f2["checkpoint"], kind="rms", dtype=BF16)
    dy1 = (b2["dx"].float() @ mix.float().t()).to(BF16)
    y1 = torch.empty_like(emb)
    b1 = capi.layer_norm_backward(dy1, w1, None, f1["rstd"], checkpoint=f1["checkpoint"], kind="rms", dsummed=b2["dx"], y=y1, dtype=BF16)
    dmix = y1.float().t() @ b2["dx"].float()

    # the chain
    kept1, kept2 = (capi.act8_unpack(f["checkpoint"], dtype=torch.float32).cpu().to(F64) for f in (f1, f2))
    r1, r2 = (f["rstd"].cpu().to(F64)[:, None] for f in (f1, f2))
    leaf = [t.cpu().to(F64).requires_grad_() for t in (emb, mix, w1, w2)]
    e, m, v1, v2 = leaf

    def norm(h, kept, r, w):
        h = h + (kept - h).detach()
        return h * (r - r ** 3 * (kept * (h - kept)).mean(1, keepdim=True)) * w

    n1 = norm(e, kept1, r1, v1)
    h2 = e + n1 @ m
    (norm(h2, kept2, r2, v2) * dhidden.cpu().to(F64)).sum().backward()
    d_emb, d_mix, d_w1, d_w2 = (t.grad for t in leaf)

    # Error bounds. Of the second norm's own results: norm_helpers, and the rounding of dx to bf16.
    u = nh.half_step(BF16)
    dx2, _, _, e2, e_w2, _ = nh.backward64(kept2, dhidden.cpu(), w2.cpu(), None, f2["rstd"].cpu(), "rms")
    e2 = e2 + u * (dx2.abs() + e2)
    # dy1: H products in fp32, rounded to bf16
    am, adx2 = mix.cpu().to(F64).abs(), dx2.abs() + e2
    dy1_64 = dx2 @ mix.cpu().to(F64).t()
    e_dy1 = e2 @ am.t() + (H + 2) * nh.U * (adx2 @ am.t())
    e_dy1 = e_dy1 + u * (dy1_64.abs() + e_dy1)
    # The first norm is linear in dy1 and dsummed; beside what comes with these, its own error and rounding.
    xh1, aw1 = (kept1 * r1).abs(), w1.cpu().to(F64).abs()
    _, _, _, e1, e_w1, _ = nh.backward64(kept1, dy1.cpu(), w1.cpu(), None, f1["rstd"].cpu(), "rms", b2["dx"].cpu())
    e1 = e1 + r1 * (aw1 * e_dy1 + xh1 * (xh1 * aw1 * e_dy1).mean(1, keepdim=True)) + e2
    e1 = e1 + u * (d_emb.abs() + e1)
    e_w1 = e_w1 + (e_dy1 * xh1).sum(0)
    # y1: a product with rstd and one with the weight, rounded to bf16; dmix: T products in fp32
    y64 = n1.detach()
    e_y1 = (6 * nh.U + u) * y64.abs() * (1 + u)
    e_mix = e_y1.t() @ adx2 + y64.abs().t() @ e2 + (T + 2) * nh.U * ((y64.abs() + e_y1).t() @ adx2)

    tiny = 1e-30
    nh.assert_within("y1", y1, y64, e_y1 + tiny)
    nh.assert_within("dweight of the second norm", b2["dweight"], d_w2, e_w2 + tiny)
    nh.assert_within("dmix", dmix, d_mix, e_mix + tiny)
    nh.assert_within("dweight of the first norm", b1["dweight"], d_w1, e_w1 + tiny)
    nh.assert_within("demb", b1["dx"], d_emb, e1 + tiny)
    assert d_emb.abs().max() > 0 and d_w1.abs().max() > 0 and d_mix.abs().max() > 0


@pytest.mark.parametrize("hidden", [8, 200, 1096, 4104])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_normed_projection_equals_its_parts_at_other_hidden_sizes(hidden, kind):
    """The parts chunk by chunk: how a norm lays rows over threads, and so the order of a row's sums, goes by a call's rows."""
    chunk = 80
    pb = synthetic.make_projection_batch(device="cuda", prompts=2, group=4, length=24, hidden=hidden, vocab=600, chunk=chunk)
    bt, T = pb.batch, pb.batch.num_tokens
    g = torch.Generator(device="cuda").manual_seed(hidden)
    x = (torch.randn((T, hidden), generator=g, device="cuda") * 2 + 0.3).to(BF16)
    w = 1 + 0.2 * torch.randn(hidden, generator=g, device="cuda")
    b = 0.1 * torch.randn(hidden, generator=g, device="cuda") if kind == "layer" else None
    rl = capi.projection_handle(pb)
    parts = [slice(r, min(T, r + chunk)) for r in range(0, T, chunk)]
    f = [capi.layer_norm(x[p], w, b, kind=kind, eps=EPS, want_stats=True) for p in parts]
    hidden_states = torch.cat([q["y"] for q in f])
    want = capi.alloc_projection_outputs(pb)
    rl.fused_projection_forward_backward(hidden_states, pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv, **want)
    dx_parts = torch.cat([capi.layer_norm_backward(want["dhidden"][p].contiguous(), w, q["mean"], q["rstd"], x=x[p], kind=kind)["dx"] for p, q in zip(parts, f)])
    mean, rstd = None if b is None else torch.cat([q["mean"] for q in f]).cpu(), torch.cat([q["rstd"] for q in f]).cpu()
    out = {k: v for k, v in capi.alloc_projection_outputs(pb).items() if k != "dhidden"}
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    rl.normed_projection_forward_backward(x, w, pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv,
                                          dx=dx, dnorm_weight=dw, norm_bias=b, kind=kind, eps=EPS, **out)
    for k in ("loss", "loss_f64", "logp", "entropy", "flags", "dw_lm"):
        assert nh.same(out[k], want[k]), k
    assert nh.same(dx, dx_parts)
    _, dw64, _, _, e_dw, _ = nh.backward64(x.cpu(), want["dhidden"].cpu(), w.cpu(), mean, rstd, kind)
    nh.assert_within("dnorm_weight", dw, dw64, e_dw)
    assert rl.device_status() == 0
