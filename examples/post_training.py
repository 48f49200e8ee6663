"""Post-training a small policy with the losses over its whole vocabulary, one after the other:

1. the frozen reference policy scores the responses (log-probs and entropies, no gradient);
2. a few steps of the policy loss with a KL term to that reference;
3. distillation from the reference's highest logits, which pulls the policy back towards it;
4. a preference loss over pairs of responses, again against the reference's log-probs.

The policy is one linear layer over random features, so the example shows the calls and not a model: its
logits are a plain product, each loss hands back dL/dlogits, and the layer's gradient is another product.

    python examples/post_training.py            # prints a line per stage
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rl_post_loss_gb300 import capi  # noqa: E402


def make_batch(vocab: int, hidden: int, seed: int = 0) -> dict:
    """Two prompts of four responses each: features, sampled tokens, rewards, and a mask over tool tokens."""
    rng = torch.Generator().manual_seed(seed)
    lengths = [23, 40, 31, 7, 64, 18, 1, 36]
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    T = int(cu[-1])
    return {"features": torch.randn(T, hidden, generator=rng).bfloat16().cuda(),
            "targets": torch.randint(0, vocab, (T,), generator=rng, dtype=torch.int32).cuda(),
            "mask": (torch.rand(T, generator=rng) > 0.1).to(torch.uint8).cuda(),
            "cu_seqlens": cu.cuda(),
            "rewards": torch.rand(len(lengths), generator=rng).cuda()}


def main(vocab: int = 5003, hidden: int = 64, steps: int = 12, k: int = 32) -> dict:
    batch = make_batch(vocab, hidden)
    x, y, mask, cu = batch["features"], batch["targets"], batch["mask"], batch["cu_seqlens"]
    T, S = x.shape[0], cu.shape[0] - 1
    ld = (vocab + 7) // 8 * 8  # rows on 16-byte boundaries
    torch.manual_seed(1)
    reference = 0.4 * torch.randn(ld, hidden, device="cuda")
    weight = reference.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def logits_of(w):
        return x @ w.bfloat16().t()

    def step(dlogits, rate):
        dlogits[:, vocab:] = 0
        weight.sub_(rate * (dlogits.t().float() @ x.float()))

    report = {}

    # 1. the reference's pass, without a gradient
    logits = logits_of(reference)
    logp_ref, entropy = capi.token_logp(logits, y, mask, vocab=vocab, want_entropy=True, device_status=status)
    ids = logits[:, :vocab].float().topk(k, dim=1).indices
    vals = logits[:, :vocab].float().log_softmax(1)
    teacher_ids, teacher_vals = ids.to(torch.int32).contiguous(), vals.gather(1, ids).contiguous()
    report["reference entropy"] = [float(entropy.sum() / mask.sum())]

    # 2. the policy loss with a KL term; the policy that sampled is the reference
    rl = capi.RlLoss(vocab_size=vocab, group_size=4, max_tokens=T, max_seqs=S, logits_dtype=capi.RL_BF16)
    loss, mean_kl = (torch.empty(1, device="cuda") for _ in range(2))
    report["policy loss"], report["KL to the reference"] = [], []
    for _ in range(steps):
        logits = logits_of(weight)
        rl.forward_backward_kl(logits, y, logp_ref, logp_ref, mask, cu, batch["rewards"], logp_ref, kl_coef=0.05,
                               kl_estimator="k3", loss=loss, dlogits=logits, mean_kl=mean_kl)
        step(logits, 0.1)
        report["policy loss"].append(float(loss))
        report["KL to the reference"].append(float(mean_kl))
    rl.close()

    # 3. back towards the reference, from its k highest logits and the mass that these leave
    report["distillation loss"] = []
    for _ in range(steps):
        logits = logits_of(weight)
        out = capi.distill_loss(logits, teacher_ids, teacher_vals, mask, cu, vocab=vocab, mode="tail",
                                direction="forward", loss_norm=capi.RL_NORM_PER_TOKEN, dlogits=logits,
                                device_status=status)
        step(logits, 2.0)
        report["distillation loss"].append(float(out["loss"]))

    # 4. responses 0, 2, ... preferred to 1, 3, ...
    report["preference loss"] = []
    for _ in range(steps):
        logits = logits_of(weight)
        out = capi.preference_loss(logits, y, logp_ref, mask, cu, vocab=vocab, beta=0.1, dlogits=logits,
                                   device_status=status)
        step(logits, 0.2)
        report["preference loss"].append(float(out["loss"]))

    report["status"] = [int(status)]
    return report


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--steps", type=int, default=12)
    args = ap.parse_args()
    for name, values in main(vocab=args.vocab, steps=args.steps).items():
        print("%-22s %s" % (name, " ".join("%.6g" % v for v in values)))
