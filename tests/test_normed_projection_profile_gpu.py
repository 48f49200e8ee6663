"""The event pairs around the kernels of the fused projection with the last norm before it."""
import pytest
import torch

from rl_post_loss_gb300 import capi, synthetic

import norm_helpers as nh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk", [80, 6])
@pytest.mark.parametrize("with_dweight", [True, False])
def test_every_kernel_is_between_events(chunk, with_dweight):
    """Also the norm's, and in a call of 32 chunks, the most that a call's events are kept for."""
    pb = synthetic.make_projection_batch(device="cuda", prompts=2, group=4, length=24, hidden=128, vocab=600, chunk=chunk)
    bt, T = pb.batch, pb.batch.num_tokens
    x = torch.randn((T, 128), device="cuda").bfloat16()
    w = torch.ones(128, device="cuda")
    rl = capi.projection_handle(pb)
    out = {k: v for k, v in capi.alloc_projection_outputs(pb).items() if k != "dhidden"}
    dx, dw = torch.empty_like(x), torch.empty_like(w) if with_dweight else None

    def step():
        rl.normed_projection_forward_backward(x, w, pb.w, bt.targets, bt.logp_old, bt.logp_infer, bt.mask, bt.cu_seqlens, bt.rewards_or_adv,
                                              dx=dx, dnorm_weight=dw, **out)

    step()
    want = [t.clone() for t in (out["loss"], out["dw_lm"], dx)]
    rl.profile_start(2)
    step()
    step()
    prof = rl.profile_read()
    chunks = (T + chunk - 1) // chunk
    assert chunks == {80: 3, 6: 32}[chunk]
    each = {"seg_prep": 1, "seg_reduce": 1, "final_reduce": 1}
    each.update({k: chunks for k in ("token_prep", "proj_gemm", "proj_rows", "proj_bwd", "norm_forward", "norm_backward")})
    assert {k: n for k, (n, _) in prof.items() if n} == {k: 2 * n for k, n in each.items()}
    assert all(ms > 0 for n, ms in prof.values() if n)
    assert all(nh.same(a, b) for a, b in zip(want, (out["loss"], out["dw_lm"], dx)))
