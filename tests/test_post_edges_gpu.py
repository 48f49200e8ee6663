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


# ---------------------------------------------------------------- sampled tokens of probability 0

EVERY = [(1003, "bf16"), (1003, "f32"), (20011, "bf16"), (600001, "f32")]  # a warp per row, rings, rows too long for them
NAN = float("nan")


def random_rows(T, V, dtype, seed):
    z = rows_of(T, V, dtype, NAN)
    g = torch.Generator().manual_seed(seed)
    z[:, :V] = (torch.randn(T, V, generator=g) * 2).to(DT[dtype]).cuda()
    return z


@pytest.mark.parametrize("kind,mean,eps", [("sigmoid", 0, 0.0), ("sigmoid", 1, 0.1), ("hinge", 0, 0.0), ("ipo", 1, 0.0)])
@pytest.mark.parametrize("V,dtype", EVERY)
def test_preference_of_an_impossible_token(V, dtype, kind, mean, eps):
    """One token of the rejected (or the preferred) response has a -inf logit. D is +inf (-inf), so the pair's loss
    and slope are their limits; the other pair's values are as ever. Tolerances as elsewhere, from the error model."""
    cu, beta, P = np.array([0, 3, 5, 9, 12]), 0.3, 2
    T = int(cu[-1])
    y = (np.arange(T) * 37 + 5) % V
    mask = np.ones(T, np.uint8)
    for t, D in ((4, np.inf), (1, -np.inf)):
        z = random_rows(T, V, dtype, V + t)
        z[t, int(y[t])] = -math.inf
        zf = z[:, :V].double().cpu().numpy()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = capi.preference_loss(z, dev(y, torch.int32), None, dev(mask), dev(cu, torch.int32), vocab=V, loss_type=kind,
                                   length_norm=bool(mean), beta=beta, label_smoothing=eps, device_status=st)
        torch.cuda.synchronize()
        r = ph.Rows(zf)
        lp = r.lp[np.arange(T), y]
        tol = r.logp_tol(lp)
        x = beta * D
        if kind == "sigmoid":
            loss = np.inf if x < 0 or eps > 0 else 0.0
            slope = -beta * (1 - eps) if x < 0 else beta * eps
        elif kind == "hinge":
            loss, slope = (np.inf, -beta) if x < 0 else (0.0, 0.0)
        else:
            loss, slope = np.inf, 2 * D
        got = out["logp"].double().cpu().numpy()
        assert got[t] == -np.inf
        fin = np.arange(T) != t
        assert np.abs(got[fin] - lp[fin]).max() <= (tol[fin] + ph.U * np.abs(lp[fin])).max()
        s = out["seq_logratio"].cpu().numpy()
        assert s[1 if t == 4 else 0] == -np.inf and np.isfinite(np.delete(s, 1 if t == 4 else 0)).all()
        pair = out["pair_loss"].cpu().numpy()
        assert pair[0] == loss
        rest = slice(5, 12)
        want = ph.preference(zf[rest], y[rest], None, mask[rest], cu[2:] - 5, kind, mean, beta, 0.0, eps, 0.0)
        s_tol = (tol[rest] + ph.U * np.abs(lp[rest])).sum()
        curve = {"sigmoid": beta * beta / 4, "hinge": 0.0, "ipo": 2.0}[kind]
        pair_tol = abs(want["slope"][0]) * s_tol + curve * s_tol ** 2 + 4 * ph.U * abs(want["pair"][0])
        assert abs(pair[1] - want["pair"][0]) <= pair_tol
        if np.isinf(loss):
            assert out["loss"].item() == np.inf and st.item() == BIT["RL_ERR_NONFINITE"]
        else:
            assert abs(out["loss"].item() - want["pair"][0] / P) <= pair_tol and st.item() == 0
        dz = out["dlogits"][:, :V].double().cpu().numpy()
        per = np.array([1 / 3, 1 / 2]) if mean else np.ones(2)
        g = np.concatenate([np.repeat([slope * per[0], -slope * per[1]], [3, 2]), want["g"]]) / P
        if kind == "ipo":  # an infinite coefficient
            assert not np.isfinite(dz[:5]).any(1).all()
            g[:5] = 0
        dg = np.concatenate([np.zeros(5), np.full(7, curve * s_tol / P)]) + 4 * ph.U * np.abs(g)
        d, d_tol = ph.onehot_grad(r, g, y, dg, np.where(fin, tol, 0), dtype)
        on = np.arange(T) >= (5 if kind == "ipo" else 0)
        assert (np.abs(dz - d)[on] <= d_tol[on]).all()


@pytest.mark.parametrize("estimator,limit", [("k1", -np.inf), ("k2", np.inf), ("k3", np.inf)])
@pytest.mark.parametrize("V,dtype", EVERY)
def test_loss_with_kl_of_an_impossible_token(V, dtype, estimator, limit):
    """The token's ratio is 0 and its estimate infinite: with a coefficient the loss is infinite, without one it is
    the policy term's. Other rows keep their gradients."""
    T, t = 6, 2
    z = random_rows(T, V, dtype, V)
    y = (np.arange(T) * 31 + 4) % V
    z[t, int(y[t])] = -math.inf
    zf = z[:, :V].double().cpu().numpy()
    r = ph.Rows(zf)
    lp = r.lp[np.arange(T), y]
    tol = r.logp_tol(lp)
    base = np.where(np.isfinite(lp), lp, -9.0).astype(np.float32)
    w = 1 / T
    ratio = np.exp(lp - base.astype(np.float64))
    rel = tol + 12 * ph.U * (1 + np.abs(base))
    for coef in (0.0, 0.5):
        out, bits = policy(z, V, y, [0, T], [1.0], base + np.float32(0.25), base, coef=coef, estimator=estimator,
                           adv_mode=capi.RL_ADV_PER_SEQ)
        kl = out["kl"].cpu().numpy()
        assert kl[t] == limit and np.isfinite(np.delete(kl, t)).all() and out["mean_kl"].item() == limit
        assert out["logp"][t].item() == -np.inf
        if coef:
            assert out["loss"].item() == limit and bits == BIT["RL_ERR_NONFINITE"]
        else:
            assert bits == 0 and abs(out["loss_f64"].item() + w * ratio.sum()) <= w * (ratio * rel).sum()
        _, dk = ph.kl_terms(estimator, np.where(np.isfinite(lp), lp, 0) - (base + np.float32(0.25)))
        g = w * (coef * dk - ratio)
        g[t] = 0.0
        dg = w * (ratio * rel + coef * (tol + 8 * ph.U * 9) * (1 + np.abs(dk)))
        d, d_tol = ph.onehot_grad(r, g, y, dg, np.where(np.isfinite(lp), tol, 0), dtype)
        dz = out["dlogits"][:, :V].double().cpu().numpy()
        on = np.arange(T) != t if coef else np.ones(T, bool)
        assert (np.abs(dz - d)[on] <= d_tol[on]).all()


# ---------------------------------------------------------------- masses at the end of fp32's range

DEEP = [60, 87, 89, 92, 95, 99, 102]  # -ln of a mass: the last ones are subnormal


def deep_rows(V, what):
    """Logits, teacher ids and log-probs of a row for each of DEEP, whose one mass is about e^-L."""
    z, ids, vals = np.zeros((len(DEEP), V)), [], []
    for row, L in zip(z, DEEP):
        gap = L + round(math.log(V - 1))
        if what == "po":        # the student's mass outside the teacher's entries
            row[3] = gap
            e = [(3, math.log(0.5)), (-1, -np.inf)]
        elif what == "pk":      # the student's mass at one of them
            row[5], row[7] = round(math.log(V)), round(math.log(V)) - L
            e = [(5, math.log(0.3)), (7, math.log(0.3))]
        elif what == "qk":      # the teacher's mass at one of them
            row[5], row[7] = round(math.log(V)), round(math.log(V)) + 1
            e = [(5, math.log(0.6)), (7, -float(L))]
        else:                   # the teacher's remaining mass (its floor is that of the test)
            row[5] = round(math.log(V))
            e = [(5, 0.0), (-1, -np.inf)]
        ids.append([i for i, _ in e])
        vals.append([v for _, v in e])
    return z, np.array(ids, np.int32), np.array(vals, np.float32)


@pytest.mark.parametrize("what,mode,reverse", [("po", "tail", 1), ("pk", "tail", 1), ("qk", "tail", 0), ("qk", "renorm", 0),
                                               ("qo", "tail", 0), ("po", "tail", 0), ("qk", "tail", 1)])
@pytest.mark.parametrize("V,dtype", EVERY + [(9, "f32")])
def test_distill_with_masses_at_the_end_of_the_range(V, dtype, what, mode, reverse):
    """A term h ln(h / o) - h + o with h near 0 is near o: the divergence and the gradient stay finite."""
    zn, ids, vals = deep_rows(V, what)
    for floor in ([math.exp(-float(L)) for L in DEEP] if what == "qo" else [1e-6]):
        check_distill(zn, ids, vals, dtype, mode, reverse, float(np.float32(floor)))


@pytest.mark.parametrize("V,dtype", EVERY)
def test_distill_with_a_mass_scaled_below_the_range(V, dtype):
    """Reverse, where one of 300 entries has a mass whose exponential is in range and whose share of the sum is not."""
    steps = [80, 84, 85, 86, 87]
    zn = np.zeros((len(steps), V))
    ids = np.tile(np.arange(300, dtype=np.int32), (len(steps), 1))
    vals = np.full(ids.shape, math.log(0.4 / 299), np.float32)
    vals[:, 299] = math.log(0.3)
    for row, L in zip(zn, steps):
        row[:299], row[299] = 4, 4 - L
    check_distill(zn, ids, vals, dtype, "tail", 1, 1e-6)


def check_distill(zn, ids, vals, dtype, mode, reverse, floor):
    """One call, every row on, against 64 bits and the error model's bounds, which are finite."""
    T, V = zn.shape
    z = rows_of(T, V, dtype, NAN)
    z[:, :V] = torch.from_numpy(zn).cuda().to(DT[dtype])
    zf = z[:, :V].double().cpu().numpy()
    assert np.array_equal(zf, zn)  # the steps are representable
    mask, cu = np.ones(T, np.uint8), np.array([0, T], np.int32)
    args = (ids, vals, mask, cu, mode, reverse, 1.0, 1.0, floor, True)
    loss, kl, d = ph.distill(zf, *args)
    loss_tol, kl_tol, d_tol = ph.distill_tol(zf, *args, dtype, kl, d)
    assert np.isfinite(kl).all() and np.isfinite(d).all()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = capi.distill_loss(z, dev(ids), dev(vals), dev(mask), dev(cu), vocab=V, mode=mode,
                            direction="reverse" if reverse else "forward", tail_floor=floor,
                            loss_norm=capi.RL_NORM_PER_TOKEN, device_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert (np.abs(out["kl"].double().cpu().numpy() - kl) <= kl_tol).all()
    assert abs(out["loss"].item() - loss) <= loss_tol + ph.U * abs(loss)
    assert (np.abs(out["dlogits"][:, :V].double().cpu().numpy() - d) <= d_tol).all()


@pytest.mark.parametrize("V,dtype", EVERY)
def test_reverse_distillation_of_a_certain_teacher(V, dtype):
    """Teacher rows whose entries sum to 1 or more in fp32, under the defaults: finite, and the floor's values."""
    T, K = 4, 3
    z = random_rows(T, V, dtype, V)
    ids = np.array([[5, 1, 2], [7, -1, -1], [0, 3, 4], [8, 6, 2]], np.int32)
    vals = np.array([[0.0, -30.0, -40.0], [0.0, -np.inf, -np.inf], np.log([0.5, 0.25, 0.25]), np.log([0.6, 0.2, 0.1])], np.float32)
    mask, cu = np.ones(T, np.uint8), np.array([0, T], np.int32)
    call = lambda **kw: capi.distill_loss(z, dev(ids), dev(vals), dev(mask), dev(cu), vocab=V, mode="tail",
                                          loss_norm=capi.RL_NORM_PER_TOKEN, **kw)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(direction="reverse", device_status=st)
    assert st.item() == 0 and torch.isfinite(out["loss"]).all()
    assert torch.isfinite(out["kl"]).all() and torch.isfinite(out["dlogits"][:, :V].float()).all()
    same = call(direction="reverse", tail_floor=1e-9)
    assert torch.equal(out["kl"], same["kl"]) and torch.equal(out["dlogits"][:, :V], same["dlogits"][:, :V])
    assert torch.equal(call()["kl"], call(tail_floor=0.0)["kl"])  # forward: no floor


@pytest.mark.parametrize("mode", ["renorm", "tail"])
@pytest.mark.parametrize("V,dtype", EVERY)
def test_distill_bad_ids_of_rows_without_mass(V, dtype, mode):
    """A bad id is reported whatever its row's values are: also where these leave the row no mass."""
    ids = np.array([[-2, -1, -1], [V, -1, -1], [4, 9, 4], [V - 1, -1, V - 1], [-1, -1, -1], [3, 1, V - 1], [2, 7, 1]], np.int32)
    vals = np.full(ids.shape, -np.inf, np.float32)
    vals[6] = np.log([0.5, 0.2, 0.1])
    T = len(ids)
    mask, cu = np.ones(T, np.uint8), np.array([0, T], np.int32)
    z = random_rows(T, V, dtype, V)
    for rows, bits in (([0, 5, 6], BIT["RL_ERR_TARGET_RANGE"]), ([1, 6], BIT["RL_ERR_TARGET_RANGE"]),
                       ([2, 6], BIT["RL_ERR_TARGET_RANGE"]), ([3, 6], BIT["RL_ERR_TARGET_RANGE"]), ([4, 5, 6], 0)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = len(rows)
        out = capi.distill_loss(z[rows].contiguous(), dev(ids[rows]), dev(vals[rows]), dev(mask[:n]),
                                dev([0, n], torch.int32), vocab=V, mode=mode, device_status=st)
        kl, dz = out["kl"].cpu(), out["dlogits"][:, :V]
        assert st.item() == bits, rows
        for i, t in enumerate(rows):
            if t < 4:
                assert math.isnan(kl[i].item()) and not dz[i].any()
            elif t == 4 or (t == 5 and mode == "renorm"):
                assert kl[i].item() == 0.0 and not dz[i].any()
            else:
                assert math.isfinite(kl[i].item()) and dz[i].any()
        assert torch.isfinite(out["loss"]).all()


# ---------------------------------------------------------------- what masked and popped tokens hold

@pytest.mark.parametrize("V,dtype", EVERY)
@pytest.mark.parametrize("adv_mode", [capi.RL_ADV_PER_TOKEN, capi.RL_ADV_TEACHER_LOGP])
@pytest.mark.parametrize("objective", [capi.RL_OBJ_GRPO_ICEPOP, capi.RL_OBJ_DIS])
def test_loss_with_kl_of_masked_tokens_that_hold_nan(V, dtype, adv_mode, objective):
    """Masked tokens' inputs, and advantages of tokens that are popped or have a bad target, may be NaN or infinite."""
    if objective == capi.RL_OBJ_DIS and adv_mode == capi.RL_ADV_TEACHER_LOGP:
        pytest.skip("not a configuration")
    T = 8
    z = random_rows(T, V, dtype, V)
    y = (np.arange(T) * 31 + 4) % V
    y[6] = V
    mask = np.array([1, 0, 1, 0, 1, 1, 1, 0], np.uint8)
    logp = torch.log_softmax(z[:, :V].double(), 1).cpu().numpy()[np.arange(T), np.minimum(y, V - 1)].astype(np.float32)
    old, infer, ref, adv = (x.copy() for x in (logp + 0.1, logp + 0.1, logp - 0.2, np.linspace(-1, 1, T).astype(np.float32)))
    if adv_mode == capi.RL_ADV_TEACHER_LOGP:
        adv += logp
    infer[5] = infer[5] + 3.0  # popped (outside the interval with the other objective)
    code = capi.RL_BF16 if dtype == "bf16" else capi.RL_F32
    rl = capi.RlLoss(V, 1, T, 1, code, adv_mode=adv_mode, objective=objective)

    def call(old, infer, ref, adv, z):
        out = dict(loss=torch.empty(1, device="cuda"), loss_f64=torch.empty(1, dtype=torch.float64, device="cuda"),
                   dlogits=torch.zeros_like(z), kl=torch.empty(T, device="cuda"), mean_kl=torch.empty(1, device="cuda"),
                   counts=torch.empty(4, dtype=torch.int32, device="cuda"))
        rl.forward_backward_kl(z, dev(y, torch.int32), dev(old), dev(infer), dev(mask), dev([0, T], torch.int32), dev(adv),
                               dev(ref), kl_coef=0.1, kl_estimator="k3", **out)
        torch.cuda.synchronize()
        assert rl.device_status() == BIT["RL_ERR_TARGET_RANGE"]
        return out

    want = call(old, infer, ref, adv, z)
    off = mask == 0
    for bad in (NAN, math.inf, -math.inf):
        a = [x.copy() for x in (old, infer, ref, adv)]
        for x in a:
            x[off] = bad
        a[3][[5, 6]] = bad
        zb = z.clone()
        zb[torch.from_numpy(off).cuda()] = bad
        got = call(*a, zb)
        on = torch.arange(T) != 6  # the bad target's estimate is NaN
        assert torch.isfinite(want["loss"]).all()
        for name in want:
            pick = (lambda x: x[on.cuda()]) if name == "kl" else lambda x: x
            assert torch.equal(pick(got[name]), pick(want[name])), (name, bad)
    rl.close()


# ---------------------------------------------------------------- arguments

def test_wrong_status_words_and_workspaces_are_refused():
    z = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    m = torch.ones(4, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    ids, vals = y.view(4, 1), torch.zeros(4, 1, device="cuda")
    calls = [lambda **kw: capi.token_logp(z, y, m, **kw), lambda **kw: capi.distill_loss(z, ids, vals, m, cu, **kw),
             lambda **kw: capi.preference_loss(z, y, None, m, cu, **kw)]
    for call in calls:
        for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                    torch.zeros(1, dtype=torch.int64, device="cuda")):
            with pytest.raises(ValueError, match="device_status"):
                call(device_status=bad)
        call(device_status=torch.zeros(1, dtype=torch.uint32, device="cuda"))
    for call in calls[1:]:
        big = torch.zeros(1 << 17, dtype=torch.uint8, device="cuda")
        for bad in (torch.zeros(1 << 16, dtype=torch.uint8), big[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(workspace=bad)
        call(workspace=big.view(torch.float32))
    torch.cuda.synchronize()


@pytest.mark.parametrize("adv_mode", [capi.RL_ADV_GROUP_REWARDS, capi.RL_ADV_PER_TOKEN])
def test_loss_with_kl_refuses_wrong_tensors(adv_mode):
    T, S, V = 6, 2, 64
    f = lambda n: torch.zeros(n, device="cuda")
    rl = capi.RlLoss(V, 2, T, S, capi.RL_F32, adv_mode=adv_mode)
    good = dict(logits=torch.zeros(T, V, device="cuda"), targets=torch.zeros(T, dtype=torch.int32, device="cuda"), logp_old=f(T),
                logp_infer=f(T), mask=torch.ones(T, dtype=torch.uint8, device="cuda"),
                cu_seqlens=torch.tensor([0, 2, T], dtype=torch.int32, device="cuda"),
                rewards_or_adv=f(T if adv_mode >= capi.RL_ADV_PER_TOKEN else S), logp_ref=f(T), loss=f(1),
                loss_f64=torch.zeros(1, dtype=torch.float64, device="cuda"), dlogits=torch.zeros(T, V, device="cuda"), logp=f(T),
                entropy=f(T), flags=torch.zeros(T, dtype=torch.uint8, device="cuda"), seq_adv=f(S),
                counts=torch.zeros(4, dtype=torch.int32, device="cuda"), mean_entropy=f(1), kl=f(T), mean_kl=f(1))
    call = lambda **over: rl.forward_backward_kl(**{**good, **over}, kl_coef=0.1)
    call()
    for name, t in good.items():
        flat = t.dim() == 1
        bad = [t.cpu(), t.double() if t.dtype != torch.float64 else t.float()]
        if name not in ("targets", "cu_seqlens"):  # these say how many tokens and responses there are
            bad.append(t[:-1])
        bad.append(torch.zeros(2 * len(t), dtype=t.dtype, device="cuda")[::2] if flat and len(t) > 1 else t[:0])
        if not flat:
            bad += [t[:, :V - 1], torch.zeros(V, T, device="cuda").t(), t.bfloat16()]
        if name in ("targets", "mask"):
            bad.append(t.long() if name == "targets" else t.bool())
        for b in bad:
            with pytest.raises(ValueError, match=name if name != "logits" else "logits|CUDA"):
                call(**{name: b})
    call()
    torch.cuda.synchronize()
    assert rl.device_status() == 0
    rl.close()


@pytest.mark.parametrize("V,dtype", EVERY)
def test_a_new_gradient_is_zero_past_the_vocabulary(V, dtype):
    """Where the memory it is given held NaN, also on a stream that is not the current one."""
    T = 6
    z = random_rows(T, V, dtype, V)
    assert z.shape[1] > V
    y, m = dev((np.arange(T) * 7) % V, torch.int32), dev(np.ones(T), torch.uint8)
    cu, ids, vals = dev([0, 2, T], torch.int32), dev(np.ones((T, 1)), torch.int32), dev(np.full((T, 1), -1.0), torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side.cuda_stream):
        for call in (lambda: capi.distill_loss(z, ids, vals, m, cu, vocab=V, mode="tail", stream=stream),
                     lambda: capi.preference_loss(z, y, None, m, cu, vocab=V, stream=stream)):
            with torch.cuda.stream(side if stream else torch.cuda.current_stream()):
                held = torch.full_like(z, NAN)
            at = held.data_ptr()
            del held
            out = call()
            torch.cuda.synchronize()
            assert out["dlogits"].data_ptr() == at
            assert not out["dlogits"][:, V:].any() and torch.isfinite(out["dlogits"].float()).all()


# ---------------------------------------------------------------- accuracy

@pytest.mark.parametrize("gap", [20.0, 30.0, 40.0])
@pytest.mark.parametrize("V,dtype", EVERY)
def test_confident_rows_keep_their_digits(V, dtype, gap):
    """One logit above V - 1 zeros: ln p = -log1p((V - 1) e^-gap), down to -e^-30. The others' sum is exact and the
    exponential's argument rounded twice, 2 U gap relative, and its result and the logarithm's 8 U; the gradient at
    the sampled entry is that times a coefficient of a dozen more roundings."""
    T = 2
    y = np.array([17, V - 3])
    z = rows_of(T, V, dtype)
    z[torch.arange(T), torch.from_numpy(y)] = gap
    lp = -math.log1p((V - 1) * math.exp(-gap))
    rel = (2 * gap + 8) * ph.U
    logp, _ = capi.token_logp(z, dev(y, torch.int32), vocab=V)
    assert np.abs(logp.double().cpu().numpy() / lp - 1).max() <= rel
    rest = -math.expm1(lp)  # 1 - p
    half = ph.half_step(dtype)

    def at(dz):
        return dz[torch.arange(T), torch.from_numpy(y)].double().cpu().numpy()

    out, bits = policy(z, V, y, [0, T], [1.0], np.zeros(T), np.zeros(T), coef=0.0, adv_mode=capi.RL_ADV_PER_SEQ)
    assert bits == 0
    assert np.abs(out["logp"].double().cpu().numpy() / lp - 1).max() <= rel
    assert np.abs(at(out["dlogits"]) / (-math.exp(lp) / T * rest) - 1).max() <= rel + 12 * ph.U + half
    out = capi.preference_loss(z, dev(y, torch.int32), None, dev(np.ones(T), torch.uint8), dev([0, 1, 2], torch.int32),
                               vocab=V, beta=0.3)
    assert np.abs(at(out["dlogits"]) / (0.15 * rest * np.array([-1, 1])) - 1).max() <= rel + 12 * ph.U + half


@pytest.mark.parametrize("T,V,dtype", [(64, 1003, "bf16"), (64, 6144, "f32"), (64, 12288, "bf16"), (64, 20011, "bf16"),
                                       (600, 32003, "f32"), (64, 151552, "bf16"), (700, 151552, "bf16"), (40, 600001, "f32")])
def test_token_logp_error_is_that_of_a_tree(T, V, dtype):
    """A lane folds at most 20 batches in sequence (a ring's slice is at most 20 batches of 1024 entries for each of
    eight warps), and the rest are trees: 36 additions on a term's way, up to eight moves of the reference and three
    merges of 6 U each, 4 U for an exponential and 2 U of its argument's size. So no row is off by more than
    (100 + 2 mean|d|) U and its own rounding; and where the roundings are independent (0.6 U each) the rms is below
    4 U, with the result's rounding at |logp| of 8 to 16 (4.6 U) and the exponential's bias (1 U) below 8 U: 16 U
    leaves a factor of two."""
    z = random_rows(T, V, dtype, T + V)
    z[:, :V] -= (1.1 * torch.log(torch.arange(1.0, V + 1, device="cuda"))).to(z.dtype)
    y = np.random.default_rng(V).integers(0, V, T)
    logp, ent = capi.token_logp(z, dev(y, torch.int32), vocab=V, want_entropy=True)
    r = ph.Rows(z[:, :V].double().cpu().numpy())
    lp = r.lp[np.arange(T), y]
    err = logp.double().cpu().numpy() - lp
    assert (np.abs(err) <= (100 + 2 * r.mean_d + np.abs(lp)) * ph.U).all()
    assert math.sqrt((err ** 2).mean()) <= 16 * ph.U * max(1.0, np.abs(lp).max() / 16)
    err = ent.double().cpu().numpy() - r.entropy
    assert (np.abs(err) <= (100 + 2 * r.mean_d) * (1 + r.mean_d) * ph.U).all()
    assert math.sqrt((err ** 2).mean()) <= 16 * ph.U * (1 + r.mean_d.max())


# ---------------------------------------------------------------- graphs

@pytest.mark.parametrize("T,V,dtype", [(40, 40001, "bf16"), (8, 151552, "bf16"), (1200, 32768, "bf16"), (4, 600001, "f32"),
                                       (60, 20011, "f32")])
def test_long_rows_captured_in_a_graph(T, V, dtype):
    """Rows over rings, one CTA or a cluster each, with the launches that begin while the one before ends."""
    import test_post_ops_gpu as ops
    for name, op in ops._everything(2, T, V, dtype):
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
            assert ops._same(want, got), name
        del graph
