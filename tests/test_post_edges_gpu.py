"""The post-training losses on the GPU where single values decide: log-probs whose rounding is large beside the
differences taken from them. Rows that a warp takes by itself, rows over rings and rows too long for them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import post_helpers as ph  # noqa: E402
from rl_post_loss_gb300 import build as nvbuild  # noqa: E402
from rl_post_loss_gb300 import capi  # noqa: E402

pytestmark = pytest.mark.gpu

BIT = {k: 1 << v for k, v in capi.CODES.items()}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    nvbuild.build()
    capi.load()


def dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda().contiguous()


def rows_of(T, V, dtype, value=0.0):
    """[T, ld] logits of one value on the GPU, NaN past the vocabulary."""
    es = 8 if dtype == "bf16" else 4
    z = torch.full((T, (V + es - 1) // es * es), float("nan"), dtype=DT[dtype], device="cuda")
    z[:, :V] = value
    return z


def policy(z, V, y, cu, adv, ref, old, *, coef, estimator="k3", mask=None, **config):
    """One call of the loss with a KL term, its outputs, and the device status bits."""
    T, S = z.shape[0], len(cu) - 1
    rl = capi.RlLoss(V, 1, T, S, capi.RL_BF16 if z.dtype == torch.bfloat16 else capi.RL_F32, **config)
    f32 = torch.float32
    out = dict(loss=torch.empty(1, device="cuda"), loss_f64=torch.empty(1, dtype=torch.float64, device="cuda"),
               dlogits=torch.empty_like(z), logp=torch.empty(T, device="cuda"), kl=torch.empty(T, device="cuda"),
               mean_kl=torch.empty(1, device="cuda"))
    old = dev(old, f32)
    rl.forward_backward_kl(z, dev(y, torch.int32), old, old, dev(np.ones(T) if mask is None else mask, torch.uint8),
                           dev(cu, torch.int32), dev(adv, f32), dev(ref, f32), kl_coef=coef, kl_estimator=estimator, **out)
    torch.cuda.synchronize()
    bits = rl.device_status()
    rl.close()
    return out, bits


# ---------------------------------------------------------------- differences of log-probs

@pytest.mark.parametrize("low", [False, True])
@pytest.mark.parametrize("V,dtype", [(4092, "bf16"), (4092, "f32"), (20050, "bf16"), (20050, "f32"), (600003, "f32")])
def test_differences_are_taken_before_the_log_prob_is_rounded(V, dtype, low):
    """Equal logits, or the sampled token's one lower: logp = -ln V or -1 - ln(V - 1 + 1/e), and V is one whose
    log-prob is 4.2e-7 or more from its fp32 value. Every sum of ones is exact, so what is left of an error in
    logp is the two-part logarithm's, 2e-8 (twice the 1e-8 of its exponential), and in d = logp - logp_ref and
    in ln r that and half a step of the difference. A ratio's exponential adds two steps, its products and the
    weight one."""
    T = 7
    z = rows_of(T, V, dtype)
    y = (np.arange(T) * 577 + 3) % V
    if low:
        z[torch.arange(T), torch.from_numpy(y)] = -1.0
    logp = -1 - math.log(V - 1 + math.exp(-1)) if low else -math.log(V)
    assert abs(float(np.float32(logp)) - logp) > 4.2e-7
    ref, old = np.float32(logp + 1 / 64), np.float32(logp - 1 / 16)
    d, ln_r = logp - float(ref), logp - float(old)
    d_tol, r_tol = 2e-8 + ph.U * abs(d), 2e-8 + ph.U * abs(ln_r)
    full = lambda x: np.full(T, x, np.float32)
    # the KL term alone
    out, bits = policy(z, V, y, [0, T], [0.0], full(ref), full(old), coef=1.0, estimator="k1")
    assert bits == 0
    assert np.abs(out["kl"].double().cpu().numpy() - d).max() <= d_tol
    assert abs(out["mean_kl"].item() - d) <= d_tol + 2 * ph.U * abs(d)
    assert abs(out["loss_f64"].item() - d) <= d_tol + 2 * ph.U * abs(d)
    # the policy term alone: every advantage 1, no clip
    out, bits = policy(z, V, y, [0, T], [1.0], full(ref), full(old), coef=0.0, adv_mode=capi.RL_ADV_PER_SEQ)
    assert bits == 0
    r = math.exp(ln_r)
    assert abs(-out["loss_f64"].item() - r) <= r * (r_tol + 6 * ph.U)
    # both, with an advantage of -1: a loss that is a small difference of the two terms
    out, bits = policy(z, V, y, [0, T], [-1.0], full(ref), full(old), coef=64.0, estimator="k1", adv_mode=capi.RL_ADV_PER_SEQ)
    assert bits == 0 and abs(64 * d + r) < 0.1
    assert abs(out["loss_f64"].item() - (64 * d + r)) <= 64 * d_tol + r * (r_tol + 6 * ph.U)


# ---------------------------------------------------------------- threads

@pytest.mark.parametrize("V", [4099, 40001])
def test_two_threads_on_one_stream(V):
    """Each thread's calls, without a workspace of their own, give what they give alone, bit for bit."""
    import threading

    def job(seed, T, K):
        g = torch.Generator().manual_seed(seed)
        z = rows_of(T, V, "bf16")
        z[:, :V] = (torch.randn(T, V, generator=g) * 2).bfloat16().cuda()
        ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)])
        vals = torch.log_softmax(torch.randn(T, K, generator=g), 1) - 0.2
        ids, vals, y = dev(ids, torch.int32), dev(vals), dev(torch.randint(0, V, (T,), generator=g), torch.int32)
        mask, cu = dev(np.ones(T), torch.uint8), dev([0, T // 3, T], torch.int32)

        def run():
            a = capi.distill_loss(z, ids, vals, mask, cu, vocab=V, mode="tail", tail_floor=1e-6)
            b = capi.preference_loss(z, y, None, mask, cu, vocab=V)
            return [a["loss"], a["kl"], a["dlogits"][:, :V], b["loss"], b["seq_logratio"], b["dlogits"][:, :V]]
        return run

    jobs = [job(1, 60, 9), job(2, 201, 24)]
    want = [[t.clone() for t in run()] for run in jobs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2, timeout=60)

    def work(run, expected):
        start.wait()
        for i in range(40):
            if not all(torch.equal(a, b) for a, b in zip(run(), expected)):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not wrong and not any(t.is_alive() for t in threads)
