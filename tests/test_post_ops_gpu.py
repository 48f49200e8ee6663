"""The vocabulary-wide post-training operators on the GPU against their 64-bit definitions (post_helpers.py
derives the tolerances), over types, vocabularies from 1 to 151552, single rows, strides, masked rows that hold
NaN, -inf logits, bad ids and targets, empty responses; in place, on another stream, in a graph, run to run."""
import numpy as np
import pytest
import torch

import oracle
import post_helpers as ph
from parity_helpers import OracleRun, params_for
from rl_post_loss_gb300 import build as nvbuild
from rl_post_loss_gb300 import capi, synthetic

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BIT = {k: 1 << v for k, v in capi.CODES.items()}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    nvbuild.build()
    capi.load()


def logits_of(T, V, dtype, seed, pad=0, spread=3.0):
    """[T, ld] on the GPU, the columns past V and every masked row later filled with NaN by the caller."""
    g = torch.Generator().manual_seed(seed)
    ld = synthetic.padded_ld(V, dtype) + pad * (8 if dtype == "bf16" else 4)
    z = torch.full((T, ld), float("nan"), dtype=DT[dtype])
    z[:, :V] = (torch.randn(T, V, generator=g) * spread - 1.1 * torch.log(torch.arange(1.0, V + 1))).to(DT[dtype])
    return z


def f64(z, V):
    return z[:, :V].double().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def close(got, want, tol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    want, tol = np.asarray(want, np.float64), np.broadcast_to(np.asarray(tol, np.float64), np.shape(want))
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN places differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    over = err > tol[ok]
    assert not over.any(), f"{what}: {over.sum()} of {err.size} off, worst {np.max(err / np.maximum(tol[ok], 1e-300)):.3g} x tol"


# ---------------------------------------------------------------- token log-probs

LOGP = [(1, 1, 0), (3, 7, 1), (5, 8, 0), (4, 9, 0), (2, 1000, 3), (70, 4097, 0), (700, 1003, 0), (1, 32768, 0), (9, 32003, 0),
        (1, 151552, 0), (5, 151553, 1), (40, 50257, 0), (460, 5003, 0), (2, 1000003, 0), (1500, 64, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,pad", LOGP)
def test_token_logp(T, V, pad, dtype):
    z = logits_of(T, V, dtype, T + V, pad)
    rng = np.random.default_rng(V)
    y = rng.integers(0, V, T).astype(np.int32)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[0] = 1
    zf = f64(z, V)
    z[torch.from_numpy(mask == 0)] = float("nan")  # what masked rows hold does not matter
    _, lp, ent, lp_tol, ent_tol = ph.token_logp(zf, y, mask)
    zc, yc, mc, st = z.cuda(), torch.from_numpy(y).cuda(), torch.from_numpy(mask).cuda(), status()
    logp, entropy = capi.token_logp(zc, yc, mc, vocab=V, want_entropy=True, device_status=st)
    only, none = capi.token_logp(zc, yc, mc, vocab=V)
    torch.cuda.synchronize()
    assert none is None and st.item() == 0
    close(logp, lp, lp_tol, "logp")
    close(only, lp, lp_tol, "logp without the entropy")
    close(entropy, ent, ent_tol, "entropy")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [9, 1003, 40000])
def test_token_logp_infinities_and_bad_rows(V, dtype):
    z = logits_of(7, V, dtype, 5)
    low = torch.finfo(DT[dtype]).min
    z[0, :V - 1] = -float("inf")         # one finite entry: probability 1
    z[1, 0] = -float("inf")              # a target of probability 0
    z[2, 1:V] = low                      # the type's lowest value
    z[3, :V] = -float("inf")             # nothing left: not finite
    z[4, V // 2] = float("nan")
    z[5, V // 2] = float("inf")
    y = torch.tensor([V - 1, 0, 0, 0, 0, 0, V], dtype=torch.int32)
    for rows, bits in (([0, 1, 2], 0), ([3], BIT["RL_ERR_NONFINITE"]), ([4], BIT["RL_ERR_NONFINITE"]),
                       ([5], BIT["RL_ERR_NONFINITE"]), ([6], BIT["RL_ERR_TARGET_RANGE"])):
        st = status()
        logp, ent = capi.token_logp(z[rows].cuda(), y[rows].cuda(), vocab=V, want_entropy=True, device_status=st)
        assert st.item() == bits, (rows, st.item())
        if rows == [0, 1, 2]:
            want = ph.Rows(f64(z[rows], V))
            lp = want.lp[np.arange(3), y[rows].numpy()]
            tol = 1e-6 + want.logp_tol(lp)
            close(logp, lp, tol, "logp")
            close(ent, want.entropy, want.eps * (1 + 2 * want.mean_d) + 1e-6, "entropy")
            assert logp[0].item() == 0.0 and ent[0].item() == 0.0 and logp[1].item() == -float("inf")
        elif rows == [6]:
            assert torch.isnan(logp).all() and torch.isfinite(ent).all()
        else:
            assert not torch.isfinite(logp).any()


def test_token_logp_keeps_digits_near_zero():
    """A confident row: log p_y = -log1p((V - 1) e^-20) is about -1e-5; its relative error stays small."""
    V = 5003
    z = torch.zeros(1, 5004)
    z[0, 17] = 20.0
    logp, _ = capi.token_logp(z.cuda(), torch.tensor([17], dtype=torch.int32).cuda(), vocab=V)
    want = -np.log1p((V - 1) * np.exp(-20.0))
    assert abs(logp.item() - want) <= 2 * ph.U + 1e-4 * abs(want)  # S = 1 + 1e-5 is held to u


# ---------------------------------------------------------------- the loss with a KL term

KLC = [(0, [5, 17, 1, 64, 33, 0, 16, 128], 4096, {}), (1, [40, 3, 0, 90, 11, 25, 64, 1], 1001, {}),
       (2, [7, 1, 30, 12, 44, 2, 9, 21], 32003, dict(mask_frac=0.3)),
       (0, [9, 12, 1, 3, 8, 0, 6, 7], 151552, dict(loss_norm=1)),
       (0, [20, 31, 7, 9, 8, 11, 6, 7], 517, dict(objective=1, loss_norm=1)),
       (1, [20, 31, 7, 9, 8, 11, 6, 7], 2048, dict(token_adv="normal")),
       (1, [20, 31, 7, 9, 8, 11, 6, 7], 2048, dict(token_adv="teacher")),
       (0, [1, 0, 1, 0, 1, 0, 0, 1], 1000001, {}), (1, [1, 0, 0, 1, 1, 0, 0, 1], 2000003, {})]


@pytest.mark.parametrize("estimator", ["k1", "k2", "k3"])
@pytest.mark.parametrize("n", range(len(KLC)))
def test_loss_with_kl(n, estimator):
    case_id, lengths, V, over = KLC[n]
    b = synthetic.make_batch(case_id, "cuda", lengths=lengths, vocab=V, case_overrides=over)
    T, coef = b.num_tokens, 0.07
    mask = b.mask.cpu().numpy()
    y = b.targets.cpu().numpy()
    run = OracleRun(b, params_for(b))
    ref = (run.tok["logp"] + 0.3 * np.random.default_rng(n).normal(size=T)).astype(np.float32)
    out = capi.alloc_outputs(b)
    kl, mean_kl = torch.full((T,), 9.0, device="cuda"), torch.empty(1, device="cuda")
    rl = capi.handle_for_batch(b)
    adv = capi.batch_inputs(b)["rewards_or_adv"]
    rl.forward_backward_kl(b.logits, b.targets, b.logp_old, b.logp_infer, b.mask, b.cu_seqlens, adv,
                           torch.from_numpy(ref).cuda(), kl_coef=coef, kl_estimator=estimator, kl=kl, mean_kl=mean_kl, **out)
    torch.cuda.synchronize()
    assert rl.device_status() & ~BIT["RL_ERR_EMPTY_SEQ"] == 0
    # the policy part's own coefficient and objective from the oracle, the KL part from its formula
    r, lp, ent, lp_tol, ent_tol = ph.token_logp(f64(b.logits, V), y, np.ones(T, np.uint8))
    w = np.repeat(run.w, np.diff(run.np["cu_seqlens"])) * (mask != 0)
    extra, k, gk = ph.kl_loss_part(lp, ref, mask, w, estimator, coef)
    close(out["logp"], lp, lp_tol, "logp")
    close(out["entropy"], ent, ent_tol, "entropy")
    _, dk = ph.kl_terms(estimator, lp - ref)
    k_tol = np.abs(dk) * (lp_tol + 2 * ph.U * np.abs(ref)) + 8 * ph.U * (np.abs(k) + np.abs(lp - ref)) + lp_tol ** 2
    close(kl, k, np.where(mask != 0, k_tol, 0), "kl")
    on = mask != 0
    close(mean_kl, [k[on].mean()], [k_tol[on].mean() + ph.U * abs(k[on].mean())], "mean_kl")
    # tokens whose log-prob is within its tolerance of a clip or gate threshold may go either way
    ref_lp = run.np["logp_infer"] if b.objective == 1 else run.np["logp_old"]
    e = lp - ref_lp.astype(np.float64)
    hi, lo = oracle.thresholds_f32(b.beta, b.eps_low, b.eps_high)[1:]
    edge = np.minimum(np.abs(e - hi), np.abs(e - lo)) <= lp_tol + 4 * ph.U * (np.abs(lp) + 1)
    if b.adv_mode == 3:  # the advantage's own sign, and its error
        edge |= np.abs(run.token_adv - lp) <= lp_tol + 2 * ph.U * np.abs(lp)
    flags = out["flags"].cpu().numpy()
    assert np.array_equal(flags[~edge], run.tok["flags"][~edge])
    ratio = np.exp(e)
    rel = lp_tol + 4 * ph.U * np.abs(lp) + 12 * ph.U
    obj, g = run.tok["tok_obj"], run.tok["g"]
    slack = w * 2 * ratio * rel * (1 + np.abs(lp)) * (b.adv_mode == 3 or b.objective == 1)  # terms with logp as a factor
    dg = np.abs(g) * rel + slack + coef * w * (lp_tol * (1 + np.abs(dk)) * (estimator != "k1") + 8 * ph.U * (np.abs(dk) + 1))
    loss = -(w * obj).sum() + extra
    loss_tol = (w * (np.abs(obj) * rel + coef * k_tol)).sum() + slack.sum() + 2 * ph.U * abs(loss)
    assert not edge.any() or n >= 5
    if not edge.any():
        close(out["loss_f64"], [loss], [loss_tol], "loss")
        close(out["loss"], [loss], [loss_tol + ph.U * abs(loss)], "loss")
    d, tol = ph.onehot_grad(r, g + gk, y, dg, lp_tol, b.dtype)
    close(out["dlogits"][:, :V][torch.from_numpy(~edge).cuda()], d[~edge], tol[~edge], "dlogits")
    want = capi.run_batch(rl, b, capi.alloc_outputs(b))
    torch.cuda.synchronize()
    assert torch.equal(out["counts"][2:], want["counts"][2:]) and torch.equal(out["seq_adv"], want["seq_adv"])
    if not edge.any():
        assert torch.equal(out["counts"], want["counts"])


def test_loss_with_kl_skips_masked_rows_unless_their_outputs_are_wanted():
    b = synthetic.make_batch(2, "cuda", lengths=[64] * 8, vocab=3001, case_overrides=dict(mask_frac=0.4))
    off = b.mask == 0
    assert off.any()
    rl = capi.handle_for_batch(b)
    full, some = capi.alloc_outputs(b), capi.alloc_outputs(b)
    for out in (full, some):
        out["dlogits"].zero_()  # the columns past the vocabulary are not written
    args = lambda z: (z, b.targets, b.logp_old, b.logp_infer, b.mask, b.cu_seqlens, b.rewards_or_adv, b.logp_old)
    rl.forward_backward_kl(*args(b.logits), kl_coef=0.1, **full)
    z = b.logits.clone()
    z[off] = float("nan")
    for name in ("logp", "entropy"):
        some[name] = None
    rl.forward_backward_kl(*args(z), kl_coef=0.1, **some)
    torch.cuda.synchronize()
    assert rl.device_status() == 0
    for name in ("loss_f64", "dlogits", "counts", "mean_entropy"):
        assert torch.equal(full[name], some[name]), name
    assert torch.equal(full["flags"][~off], some["flags"][~off])
    rl.forward_backward_kl(*args(z), kl_coef=0.1, **full)  # now they are read
    torch.cuda.synchronize()
    assert rl.device_status() == BIT["RL_ERR_NONFINITE"]
    assert torch.equal(full["dlogits"], some["dlogits"])  # and still leave no trace in the gradient


def test_loss_with_kl_and_no_tokens():
    rl = capi.RlLoss(100, 2, 8, 2, capi.RL_F32)
    e = torch.empty(0, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 5.0, device="cuda")
    rl.forward_backward_kl(e.view(0, 100), i, e, e, e.to(torch.uint8), torch.zeros(3, dtype=torch.int32, device="cuda"),
                           torch.ones(2, device="cuda"), e, kl_coef=0.1, loss=loss, dlogits=e.view(0, 100))
    torch.cuda.synchronize()
    assert loss.item() == 0.0 and rl.device_status() == BIT["RL_ERR_EMPTY_SEQ"]


# ---------------------------------------------------------------- distillation

def distill_case(T, V, K, dtype, seed, mode, tau, pad=0, lengths=None):
    z = logits_of(T, V, dtype, seed, pad)
    rng = np.random.default_rng(seed)
    zt = f64(z, V) / tau + 0.6 * rng.normal(size=(T, V))
    lt = zt - zt.max(1, keepdims=True)
    lt -= np.log(np.exp(lt).sum(1, keepdims=True))
    k = min(K, V)
    ids = np.full((T, K), -1, np.int32)
    ids[:, :k] = np.argsort(-lt, 1, kind="stable")[:, :k]
    vals = np.full((T, K), -np.inf, np.float32)
    vals[:, :k] = np.take_along_axis(lt, ids[:, :k].astype(np.int64), 1) + (3.0 if mode == "renorm" else 0.0)
    for t in range(0, T, 3):  # padded rows
        n = rng.integers(1, k + 1)
        ids[t, n:], vals[t, n:] = -1, -np.inf
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[-1] = 1
    lengths = lengths or ([T] if T < 4 else [1, 0, T - 3, 2])
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    assert cu[-1] == T
    return z, ids, vals, mask, cu


DISTILL = [(1, 1, 1), (1, 9, 4), (4, 7, 16), (5, 64, 64), (9, 1000, 1), (30, 4097, 64), (6, 32003, 33), (3, 151552, 128),
           (4, 5000, 1024), (70, 1001, 8), (300, 517, 5), (2, 2000003, 16), (3, 600001, 7),
           (500, 2048, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode,reverse,tau", [("renorm", 0, 1.0), ("tail", 0, 2.0), ("tail", 1, 1.0), ("renorm", 0, 0.5)])
@pytest.mark.parametrize("T,V,K", DISTILL)
def test_distill(T, V, K, mode, reverse, tau, dtype):
    per_token, floor, scale = bool(T % 2), 1e-6, tau * tau
    z, ids, vals, mask, cu = distill_case(T, V, K, dtype, T * 7 + V + K, mode, tau, pad=T % 3)
    zf = f64(z, V)
    if reverse and V > 3:
        zf[0, -1] = -np.inf
        z[0, V - 1] = -float("inf")
    z[torch.from_numpy(mask == 0)] = float("nan")
    args = (ids, vals, mask, cu, mode, reverse, tau, scale, floor, per_token)
    with np.errstate(all="ignore"):
        loss, kl, d = ph.distill(zf, *args)
        loss_tol, kl_tol, d_tol = ph.distill_tol(zf, *args, dtype, kl, d)
    st = status()
    f = lambda x: torch.from_numpy(x).cuda()
    zc = z.cuda()
    before = zc.clone()
    loss64 = torch.empty(1, dtype=torch.float64, device="cuda")
    dz = torch.full_like(zc, 7.0)
    out = capi.distill_loss(zc, f(ids), f(vals), f(mask), f(cu), vocab=V, mode=mode,
                            direction="reverse" if reverse else "forward", temperature=tau, scale=scale, tail_floor=floor,
                            loss_norm=int(per_token), loss_f64=loss64, dlogits=dz, device_status=st)
    torch.cuda.synchronize()
    n = [int(mask[a:b].sum()) for a, b in zip(cu, cu[1:])]
    assert st.item() == (BIT["RL_ERR_EMPTY_SEQ"] if 0 in n else 0)
    close(out["kl"], kl, kl_tol, "kl")
    close(loss64, [loss], [loss_tol], "loss")
    close(out["loss"], [loss], [loss_tol + ph.U * abs(loss)], "loss")
    close(dz[:, :V], d, d_tol, "dlogits")
    assert bool((dz[:, V:] == 7.0).all()), "columns past the vocabulary were written"
    assert torch.equal(before.view(torch.uint8), zc.view(torch.uint8)), "the logits changed"
    # in place: the same bits
    capi.distill_loss(zc, f(ids), f(vals), f(mask), f(cu), vocab=V, mode=mode,
                      direction="reverse" if reverse else "forward", temperature=tau, scale=scale, tail_floor=floor,
                      loss_norm=int(per_token), dlogits=zc)
    torch.cuda.synchronize()
    assert torch.equal(zc[:, :V], dz[:, :V])


@pytest.mark.parametrize("V", [50, 40000])
def test_distill_bad_rows(V):
    T, K = 6, 4
    z, ids, vals, mask, cu = distill_case(T, V, K, "f32", 11, "tail", 1.0, lengths=[T])
    mask[:] = 1
    ids[0], ids[1] = [3, 9, 3, 4], [1, 2, V, 5]           # a position listed twice; one outside
    ids[2], ids[3] = [-2, 1, 2, 3], [-1, -1, -1, -1]      # a negative one that is not padding; nothing
    ids[4], vals[4] = [7, 8, 9, 10], -np.inf              # entries without mass
    ids[5] = [V - 1, 0, 1, 2]
    vals[[0, 1, 2, 3, 5]] = np.log(0.2)
    f = lambda x: torch.from_numpy(x).cuda()
    st = status()
    out = capi.distill_loss(z.cuda(), f(ids), f(vals), f(mask), f(cu), vocab=V, mode="tail", tail_floor=1e-6,
                            loss_norm=1, device_status=st)
    torch.cuda.synchronize()
    assert st.item() == BIT["RL_ERR_TARGET_RANGE"]
    kl, dz = out["kl"].cpu(), out["dlogits"][:, :V].cpu()
    assert torch.isnan(kl[:3]).all() and torch.isfinite(kl[3:]).all()
    assert bool((dz[:3] == 0).all())
    assert kl[3] == 0 and bool((dz[3] == 0).all())  # nothing known of the row: it contributes nothing
    want = {t: ph.distill_row(f64(z, V)[t], ids[t], vals[t], "tail", 0, 1.0, 1e-6) for t in (4, 5)}
    for t in (4, 5):
        assert abs(kl[t].item() - want[t][0]) <= 2e-5 * max(1.0, abs(want[t][0]))
        assert np.abs(dz[t].numpy() - want[t][1] / T).max() <= 2e-5 / T
    loss = out["loss"].item()
    assert abs(loss - (want[4][0] + want[5][0]) / T) <= 1e-5


def test_distill_no_tokens_and_all_masked():
    f32, dev = torch.float32, "cuda"
    e = torch.empty(0, 64, device=dev)
    out = capi.distill_loss(e, torch.empty(0, 4, dtype=torch.int32, device=dev), torch.empty(0, 4, device=dev),
                            torch.empty(0, dtype=torch.uint8, device=dev), torch.zeros(2, dtype=torch.int32, device=dev))
    assert out["loss"].item() == 0.0
    z, ids, vals, mask, cu = distill_case(5, 100, 4, "bf16", 3, "renorm", 1.0)
    z[:] = float("nan")
    f = lambda x: torch.from_numpy(x).cuda()
    st = status()
    out = capi.distill_loss(z.cuda(), f(ids), f(vals), torch.zeros(5, dtype=torch.uint8, device=dev), f(cu), vocab=100,
                            device_status=st)
    assert out["loss"].item() == 0.0 and bool((out["dlogits"][:, :100] == 0).all()) and bool((out["kl"] == 0).all())
    assert st.item() == BIT["RL_ERR_EMPTY_SEQ"]


@pytest.mark.parametrize("mode,reverse", [("renorm", 0), ("tail", 0), ("tail", 1)])
def test_distill_gradient_against_differences_of_the_loss(mode, reverse):
    """Directional derivative of the kernel's own fp64 loss. Central step h: truncation h^2 / 6 times a third
    derivative of at most 8 max|u|^3 per row of weight, and rounding of two losses each within loss_tol."""
    T, V, K, h = 12, 700, 16, 2.0 ** -5
    z, ids, vals, mask, cu = distill_case(T, V, K, "f32", 21, mode, 1.0, lengths=[T])
    u = np.random.default_rng(2).choice([-1.0, 1.0], size=(T, V)).astype(np.float32)
    f = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    kw = dict(vocab=V, mode=mode, direction="reverse" if reverse else "forward", tail_floor=1e-6, loss_norm=1)
    base = z[:, :V].numpy()

    def loss(x):
        out = torch.empty(1, dtype=torch.float64, device="cuda")
        g = capi.distill_loss(f(x), f(ids), f(vals), f(mask), f(cu), loss_f64=out, **kw)["dlogits"]
        return out.item(), g
    lo, hi = base - h * u, base + h * u
    g = loss(base)[1].double().cpu().numpy()
    slope = (loss(hi)[0] - loss(lo)[0]) / (2 * h)
    args = (ids, vals, mask, cu, mode, reverse, 1.0, 1.0, 1e-6, True)
    l64, kl64, d64 = ph.distill(base, *args)
    tol = ph.distill_tol(base, *args, "f32", kl64, d64)[0] / h + 8 * h * h / 6
    assert abs(slope - (g * u).sum()) <= tol
    assert abs((g * u).sum()) > 3 * tol or mode != "renorm"  # the test sees a gradient


# ---------------------------------------------------------------- preference

PREF = [([1, 1], 1), ([3, 0], 9), ([5, 2, 1, 7], 1000), ([40, 33, 0, 0, 12, 1], 4097), ([9, 30], 32003), ([3, 2], 151552),
        ([200, 340, 90, 7], 517), ([1, 2], 1000003)]


def check_pref(lengths, V, dtype, kind, mean, use_ref, seed=0, nll=0.2, smoothing=0.1):
    T = sum(lengths)
    z = logits_of(T, V, dtype, seed + V, pad=len(lengths) % 2, spread=1.0)
    rng = np.random.default_rng(seed + T)
    y = rng.integers(0, V, T).astype(np.int32)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    zf = f64(z, V)
    z[torch.from_numpy(mask == 0)] = float("nan")
    lp = ph.Rows(zf).lp[np.arange(T), y]
    ref = (lp + 0.2 * rng.normal(size=T)).astype(np.float32) if use_ref else None
    beta, margin = (0.3, 0.1) if use_ref else (0.02, 0.1)
    args = (y, ref, mask, cu, kind, mean, beta, margin, smoothing if kind == "sigmoid" else 0.0, nll)
    want = ph.preference(zf, *args)
    f = lambda x: None if x is None else torch.from_numpy(x).cuda()
    st, zc = status(), z.cuda()
    dz = torch.full_like(zc, 7.0)
    loss64 = torch.empty(1, dtype=torch.float64, device="cuda")
    kw = dict(vocab=V, loss_type=kind, length_norm=bool(mean), beta=beta, margin=margin, label_smoothing=args[8], nll_coef=nll)
    out = capi.preference_loss(zc, f(y), f(ref), f(mask), f(cu), loss_f64=loss64, dlogits=dz, device_status=st, **kw)
    torch.cuda.synchronize()
    assert st.item() == (BIT["RL_ERR_EMPTY_SEQ"] if 0 in want["n"] else 0)
    r = want["rows"]
    lp_tol = np.where(mask != 0, r.logp_tol(lp) + ph.U * np.abs(lp), 0.0)
    close(out["logp"], want["logp"], lp_tol, "logp")
    S = len(lengths)
    s_tol = np.array([(lp_tol[a:b].sum() / (max(1, want["n"][i]) if mean else 1)) for i, (a, b) in enumerate(zip(cu, cu[1:]))])
    s_tol = s_tol + 2 * ph.U * np.abs(want["s"])
    close(out["seq_logratio"], want["s"], s_tol, "seq_logratio")
    D_tol = s_tol[0::2] + s_tol[1::2]
    curve = {"sigmoid": beta * beta / 4, "hinge": 0.0, "ipo": 2.0}[kind]  # bound of the second derivative in D
    near_kink = (np.abs(beta * (want["s"][0::2] - want["s"][1::2]) - margin - 1) <= beta * D_tol) if kind == "hinge" else np.zeros(S // 2, bool)
    assert not near_kink.any()
    like_tol = nll * np.array([lp_tol[a:b].sum() / max(1, want["n"][2 * j]) for j, (a, b) in enumerate(zip(cu[0::2], cu[1::2]))])
    pair_tol = np.abs(want["slope"]) * D_tol + curve * D_tol ** 2 + like_tol + 2 * ph.U * np.abs(want["pair"])
    close(out["pair_loss"], want["pair"], pair_tol, "pair_loss")
    close(loss64, [want["loss"]], [pair_tol.mean()], "loss")
    close(out["loss"], [want["loss"]], [pair_tol.mean() + ph.U * abs(want["loss"])], "loss")
    dg = np.zeros(T)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        per = max(1, want["n"][i]) if mean else 1
        dg[a:b] = (curve * D_tol[i // 2] / per) / (S // 2)
    dg += 2 * ph.U * np.abs(want["g"])
    d, tol = ph.onehot_grad(r, want["g"], y, dg, lp_tol, dtype)
    close(dz[:, :V], d, tol, "dlogits")
    assert bool((dz[:, V:] == 7.0).all())
    capi.preference_loss(zc, f(y), f(ref), f(mask), f(cu), dlogits=zc, **kw)
    torch.cuda.synchronize()
    assert torch.equal(zc[:, :V], dz[:, :V]), "in place"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,mean,use_ref", [("sigmoid", 0, True), ("sigmoid", 1, False), ("hinge", 0, True), ("ipo", 1, True)])
@pytest.mark.parametrize("lengths,V", PREF)
def test_preference(lengths, V, dtype, kind, mean, use_ref):
    check_pref(lengths, V, dtype, kind, mean, use_ref)


def test_preference_bad_targets_and_no_tokens():
    z = logits_of(6, 100, "f32", 1)
    y = torch.tensor([3, 100, 5, 7, -1, 8], dtype=torch.int32)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32)
    mask = torch.ones(6, dtype=torch.uint8)
    st = status()
    out = capi.preference_loss(z.cuda(), y.cuda(), None, mask.cuda(), cu.cuda(), vocab=100, beta=0.1, device_status=st)
    torch.cuda.synchronize()
    assert st.item() == BIT["RL_ERR_TARGET_RANGE"]
    want = ph.preference(f64(z, 100), y.numpy(), None, mask.numpy(), cu.numpy(), "sigmoid", 0, 0.1, 0.0, 0.0, 0.0)
    close(out["logp"], want["logp"], 1e-5, "logp")
    close(out["loss"], [want["loss"]], [1e-5], "loss")
    assert bool((out["dlogits"][[1, 4]] == 0).all()) and bool((out["dlogits"][[0, 2, 3, 5], :100] != 0).any(1).all())
    e = torch.empty(0, 64, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    out = capi.preference_loss(e, i, None, i.to(torch.uint8), torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out["loss"].item() == pytest.approx(np.log(2), rel=1e-6)
    # a non-finite row shows
    z[2, 4] = float("nan")
    st.zero_()
    out = capi.preference_loss(z.cuda(), y.clamp(0, 99).cuda(), None, mask.cuda(), cu.cuda(), vocab=100, device_status=st)
    assert st.item() == BIT["RL_ERR_NONFINITE"] and torch.isnan(out["loss"]).all()


# ---------------------------------------------------------------- all of them: repeats, streams, graphs, guards

def _everything(seed, T=60, V=5003, dtype="bf16"):
    """One call of each operator as (name, function) over shared inputs; every function returns its outputs."""
    z, ids, vals, mask, cu = distill_case(T, V, 24, dtype, seed, "tail", 1.0, lengths=[T // 4] * 4)
    rng = np.random.default_rng(seed)
    f = lambda x: torch.from_numpy(x).cuda()
    zc, y, m, c = z.cuda(), f(rng.integers(0, V, T).astype(np.int32)), f(mask), f(cu)
    ref = f((-6 + rng.normal(size=T)).astype(np.float32))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
          (capi.rl_loss_distill_workspace_bytes(T, 4), capi.rl_loss_preference_workspace_bytes(T, 4))]
    rl = capi.RlLoss(V, 2, T, 4, capi.RL_BF16 if dtype == "bf16" else capi.RL_F32)
    rew = torch.tensor([1.0, 0.0, 0.0, 1.0], device="cuda")

    def policy():
        out = dict(loss=torch.empty(1, device="cuda"), dlogits=torch.zeros_like(zc), logp=torch.empty(T, device="cuda"),
                   counts=torch.empty(4, dtype=torch.int32, device="cuda"), kl=torch.empty(T, device="cuda"),
                   mean_kl=torch.empty(1, device="cuda"))
        rl.forward_backward_kl(zc, y, ref, ref, m, c, rew, ref, kl_coef=0.1, **out)
        return out

    def logp():
        a, b = capi.token_logp(zc, y, m, vocab=V, want_entropy=True)
        return {"logp": a, "entropy": b}

    f_ids, f_vals = f(ids), f(vals)
    zeros = lambda: torch.zeros_like(zc)
    return [("logp", logp), ("policy", policy),
            ("distill", lambda: capi.distill_loss(zc, f_ids, f_vals, m, c, vocab=V, mode="tail", tail_floor=1e-6,
                                                  dlogits=zeros(), workspace=ws[0])),
            ("pref", lambda: capi.preference_loss(zc, y, ref, m, c, vocab=V, beta=0.1, dlogits=zeros(), workspace=ws[1]))]


def _same(a, b):
    return all(torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8)) for k in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(60, 5003), (8, 151552), (1200, 260)])
def test_repeats_and_streams_give_the_same_bits(T, V, dtype):
    ops = _everything(1, T, V, dtype)
    first = {n: op() for n, op in ops}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = {n: op() for n, op in ops}
        side.synchronize()
        for n, _ in ops:
            assert _same(first[n], again[n]), n


def test_captured_in_a_graph():
    for name, op in _everything(2):
        want = op()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = op()
        for _ in range(3):
            for t in got.values():
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(want, got), name
        del graph


def test_a_capture_without_a_workspace_is_refused():
    z = torch.zeros(2, 64, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    m = torch.ones(2, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    dz = torch.empty_like(z)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(ValueError, match="workspace"):
            capi.preference_loss(z, i, None, m, cu, dlogits=dz)
        z.add_(1.0)  # the capture goes on
    graph.replay()
    torch.cuda.synchronize()


def test_malformed_cu_seqlens_are_reported():
    T, V = 6, 64
    z, y = torch.zeros(T, V, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    m = torch.ones(T, dtype=torch.uint8, device="cuda")
    for cu in ([0, 4, 2, 5, 6], [0, 2, 3, 4, 5], [1, 2, 3, 4, 6], [0, 2, 9, 9, 6], [0, -3, 2, 4, 6]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st = status()
        capi.preference_loss(z, y, None, m, c, device_status=st)
        torch.cuda.synchronize()
        assert st.item() & BIT["RL_ERR_SEQLENS"], cu
        st.zero_()
        capi.distill_loss(z, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.zeros(T, 1, device="cuda"), m, c,
                          device_status=st)
        torch.cuda.synchronize()
        assert st.item() & BIT["RL_ERR_SEQLENS"], cu


def test_wrong_tensors_are_refused():
    z = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    m = torch.ones(4, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (y.long(), y[:3], y.cpu(), torch.zeros(8, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError, match="targets"):
            capi.token_logp(z, bad)
    with pytest.raises(ValueError, match="rows"):
        capi.token_logp(z.t(), y)
    with pytest.raises(ValueError, match="float32"):
        capi.token_logp(z.half(), y)
    with pytest.raises(ValueError, match="vocab"):
        capi.token_logp(z, y, vocab=65)
    with pytest.raises(ValueError, match="mask"):
        capi.preference_loss(z, y, None, m.bool(), cu)
    with pytest.raises(ValueError, match="dlogits"):
        capi.preference_loss(z, y, None, m, cu, dlogits=z.bfloat16())
    with pytest.raises(ValueError, match="teacher_ids"):
        capi.distill_loss(z, y.view(4, 1).long(), z[:, :1], m, cu)
    with pytest.raises(ValueError, match="shape"):
        capi.distill_loss(z, y.view(4, 1), z[:, :2].contiguous(), m, cu)
