"""Workloads of the vocabulary-wide post-training operators, with their plain forms.

Four operators over packed response tokens whose logits row covers the whole vocabulary:

  logp     log-prob (and entropy) of the sampled tokens, forward only: the reference or old policy's pass
  policy   the clipped policy loss with a KL term to a reference policy, forward and backward
  distill  distillation from a teacher's top logits, forward and backward
  pref     a preference loss over pairs of responses (paired log ratios), forward and backward

``listed()`` names fixed workloads and ``draw()`` draws others of the same ranges; ``prepare()`` makes a
workload's tensors from a seed, ``run()`` makes one pass, ``exact()`` gives the same outputs in 64 bits from
the definitions, ``work()`` the bytes and operations a pass cannot do without. With ``own`` false ``run()``
is elementary torch arithmetic in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

EPS_LOW, EPS_HIGH, BETA_POP, ADV_EPS = 0.2, 0.28, 2.0, 1e-6


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # the log-prob of a handful of tokens, as when one short response is scored by itself: latency
        dict(name="logp-8x151552-bf16", op="logp", seqs=1, lo=8, hi=8, vocab=151552, dtype="bf16", masked=0.0,
             entropy=True),
        # an fp32 evaluation batch with an odd vocabulary
        dict(name="logp-1201x32003-f32", op="logp", seqs=5, lo=120, hi=360, vocab=32003, dtype="f32", masked=0.1,
             entropy=True),
        # the reference policy's pass over a training batch; prompt and tool tokens are masked
        dict(name="logp-16kx151552-bf16", op="logp", seqs=16, lo=512, hi=1536, vocab=151552, dtype="bf16", masked=0.25,
             entropy=False),
        # two prompts of four short responses: the smallest training step
        dict(name="policy-tiny-f32", op="policy", seqs=8, group=4, lo=16, hi=128, vocab=4096, dtype="f32", masked=0.0,
             estimator="k3", coef=0.02, per_token=False),
        # eight prompts of eight responses on a mid-size vocabulary
        dict(name="policy-18kx32768-bf16", op="policy", seqs=64, group=8, lo=64, hi=512, vocab=32768, dtype="bf16",
             masked=0.0, estimator="k3", coef=0.05, per_token=False),
        # long responses on the large vocabulary with tool tokens masked, mean over tokens
        dict(name="policy-9kx151552-bf16", op="policy", seqs=8, group=8, lo=512, hi=1792, vocab=151552, dtype="bf16",
             masked=0.25, estimator="k2", coef=0.01, per_token=True),
        # one short on-policy response: a few rows, few teacher entries
        dict(name="distill-37x151552-k16-bf16", op="distill", seqs=1, lo=37, hi=37, vocab=151552, dtype="bf16",
             masked=0.0, k=16, mode="renorm", direction="forward", temperature=1.0, per_token=True),
        # softened distributions with the remaining mass as one more outcome; fp32 logits, odd vocabulary
        dict(name="distill-3kx32001-k64-f32", op="distill", seqs=12, lo=64, hi=448, vocab=32001, dtype="f32", masked=0.1,
             k=64, mode="tail", direction="forward", temperature=2.0, per_token=False),
        # on-policy distillation at scale: mode-seeking direction, many teacher entries
        dict(name="distill-8kx151552-k128-bf16", op="distill", seqs=16, lo=256, hi=768, vocab=151552, dtype="bf16",
             masked=0.2, k=128, mode="tail", direction="reverse", temperature=1.0, per_token=True),
        # two short pairs
        dict(name="pref-2pairs-32768-bf16", op="pref", seqs=4, lo=20, hi=60, vocab=32768, dtype="bf16", masked=0.0,
             kind="sigmoid", mean=False, ref=True),
        # sixteen pairs on a mid-size vocabulary, prompt tokens masked
        dict(name="pref-16pairs-32768-bf16", op="pref", seqs=32, lo=64, hi=512, vocab=32768, dtype="bf16", masked=0.3,
             kind="sigmoid", mean=False, ref=True),
        # eight long pairs on the large vocabulary, length-normalised, no reference
        dict(name="pref-8pairs-151552-bf16", op="pref", seqs=16, lo=256, hi=1024, vocab=151552, dtype="bf16", masked=0.3,
             kind="sigmoid", mean=True, ref=False),
    ]


def draw(rng):
    op = rng.choice(["logp", "policy", "distill", "pref"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    vocab = int(round(math.exp(rng.uniform(math.log(4000), math.log(155000)))))
    if rng.random() < 0.3:
        vocab = rng.choice([4096, 32768, 151552])
    most = 1.2e9 if dtype == "bf16" else 0.6e9  # logits of a batch
    tokens = math.exp(rng.uniform(math.log(2), math.log(min(20000, most / vocab))))
    group = rng.choice([2, 4, 8])
    unit = {"policy": group, "pref": 2}.get(op, 1)
    seqs = unit * max(1, int(round(tokens ** rng.uniform(0.1, 0.6) / unit)))
    mean_len = max(1.0, tokens / seqs)
    lo = max(1, int(mean_len * rng.uniform(0.3, 1.0)))
    hi = max(lo, int(2 * mean_len) - lo)
    case = dict(op=op, seqs=seqs, lo=lo, hi=hi, vocab=vocab, dtype=dtype, masked=rng.choice([0.0, 0.1, 0.3]))
    if op == "logp":
        case.update(entropy=rng.random() < 0.5)
    elif op == "policy":
        case.update(group=group, estimator=rng.choice(["k1", "k2", "k3"]), coef=rng.choice([0.005, 0.02, 0.1]),
                    per_token=rng.random() < 0.5)
    elif op == "distill":
        mode = rng.choice(["renorm", "tail"])
        case.update(k=int(round(math.exp(rng.uniform(math.log(2), math.log(160))))), mode=mode,
                    direction="forward" if mode == "renorm" else rng.choice(["forward", "reverse"]),
                    temperature=rng.choice([1.0, 1.0, 2.0]), per_token=rng.random() < 0.5)
    else:
        case.update(kind=rng.choice(["sigmoid", "sigmoid", "ipo"]), mean=rng.random() < 0.4, ref=rng.random() < 0.7)
    return case


def _lengths(case):
    """Response lengths: spread evenly over [lo, hi] in a shuffled order that depends on the case alone."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    even = [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else (lo + hi) // 2 for i in range(n)]
    step = next(s for s in (7, 5, 3, 11, 13, 1) if math.gcd(s, n) == 1)
    return [even[(i * step) % n] for i in range(n)]


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    lengths = _lengths(case)
    S, T, V, op = len(lengths), sum(lengths), case["vocab"], case["op"]
    dt, per16 = (torch.bfloat16, 8) if case["dtype"] == "bf16" else (torch.float32, 4)
    ld = (V + per16 - 1) // per16 * per16  # rows start on 16-byte boundaries; the columns past V hold anything
    cu = torch.zeros(S + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lengths), 0)
    cu = cu.to(dev)
    st = dict(case=dict(case), T=T, S=S, V=V, cu=cu)

    # logits: normal values over a falling prior of the token ids, as the framework's own workloads have
    prior = -1.1 * torch.log(torch.arange(1, ld + 1, device=dev, dtype=torch.float32))
    logits = torch.empty((T, ld), dtype=dt, device=dev)
    targets = torch.empty(T, dtype=torch.int32, device=dev)
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    K = case.get("k", 0)
    if K:
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        vals = torch.empty((T, K), dtype=torch.float32, device=dev)
    rows = max(1, (1 << 27) // ld)
    for r0 in range(0, T, rows):
        r1 = min(T, r0 + rows)
        logits[r0:r1] = randn(r1 - r0, ld).mul_(3.0).add_(prior)
        z = logits[r0:r1, :V].float()
        if K:  # a teacher near the student: the log-probs of its top entries at the temperature, largest first
            top = torch.log_softmax((z + 0.7 * randn(r1 - r0, V)) / case["temperature"], 1).topk(K, 1)
            vals[r0:r1], ids[r0:r1] = top.values, top.indices.to(torch.int32)
        else:  # targets drawn from softmax(z)
            y = (z - torch.log(-torch.log(rand(r1 - r0, V).clamp_(1e-30, 1 - 1e-7)))).argmax(1)
            targets[r0:r1] = y.to(torch.int32)
            logp[r0:r1] = torch.log_softmax(z, 1).gather(1, y[:, None])[:, 0]
        del z

    # masked tokens (prompt or tool output): the leading part of each response, at least one token stays
    n = torch.tensor(lengths, device=dev)
    seq = torch.repeat_interleave(torch.arange(S, device=dev), n)
    place = torch.arange(T, device=dev) - cu[:-1].long()[seq]
    skip = (rand(S) * 2 * case["masked"] * n).floor().long().clamp_max(n - 1)
    st.update(logits=logits, mask=(place >= skip[seq]).to(torch.uint8), targets=targets, seq=seq)
    st["dlogits"] = torch.empty_like(logits) if op != "logp" else None

    if op == "policy":
        # old and inference log-probs as in the framework's workloads. logp - logp_old within 1e-4 of a clip
        # threshold is moved off it: there the last bit of a log-prob would decide the branch
        noise = 0.15 * randn(T)
        for edge in (-math.log1p(EPS_HIGH), -math.log1p(-EPS_LOW)):
            noise = torch.where((noise - edge).abs() < 1e-4, noise + 4e-4, noise)
        old = logp + noise
        infer = old + 0.1 * randn(T) + 2.0 * (rand(T) < 0.02)
        st.update(logp_old=old, logp_infer=infer, logp_ref=logp + 0.3 * randn(T), rewards=(rand(S) < 0.5).float())
        if own:  # the handle a trainer keeps
            from rl_post_loss_gb300 import capi
            st["rl"] = capi.RlLoss(V, case["group"], T, S, capi.RL_BF16 if case["dtype"] == "bf16" else capi.RL_F32,
                                   loss_norm=capi.RL_NORM_PER_TOKEN if case["per_token"] else capi.RL_NORM_PER_RESPONSE)
    if op == "pref":
        st["logp_ref"] = logp + 0.1 * randn(T) if case["ref"] else None
    if op == "distill":
        # some rows keep fewer entries (-1 / -inf padding, as a top-k over a short row gives)
        keep = torch.where(rand(T) < 0.1, (1 + rand(T) * (K - 1)).long(), torch.full((T,), K, device=dev))
        pad = torch.arange(K, device=dev)[None, :] >= keep[:, None]
        st.update(ids=ids.masked_fill_(pad, -1), vals=vals.masked_fill_(pad, -math.inf))
    if op != "distill":
        st["logp"] = torch.empty(T, dtype=torch.float32, device=dev)
    return st


def _pref_numbers(case):
    """beta, margin, label smoothing and weight of the likelihood term."""
    return (2.0, 0.5, 0.0, 0.0) if case["mean"] else (0.1, 0.0, 0.1, 0.2)


# ---------------------------------------------------------------------------- one pass

def run(st):
    return (_library if own else _plain)[st["case"]["op"]](st)


def _rows(st):
    """Row maxima, exponentials against them and their sums, of the logits in 32 bits."""
    z = st["logits"][:, :st["V"]].float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    return z, m, e, e.sum(1, keepdim=True)


def _token_logp(st, z, m, s):
    return (z.gather(1, st["targets"].long()[:, None]) - m - torch.log(s))[:, 0]


def _seq_sum(st, x):
    """Sums over each response, in 64 bits."""
    return torch.zeros(st["S"], dtype=torch.float64, device=x.device).index_add_(0, st["seq"], x.double())


def _logits_grad(st, g, e, s):
    """g (1[v == y] - p_v), rounded once."""
    d = e * (-g[:, None] / s)
    d.scatter_add_(1, st["targets"].long()[:, None], g[:, None])
    return d.to(st["logits"].dtype)


def _weights(st, m):
    """1/(S n_i) or 1/N for every token, 0 where it is masked."""
    n = _seq_sum(st, m)
    if st["case"]["per_token"]:
        return (m.double() / n.sum()).float()
    return (m.double() / (st["S"] * n[st["seq"]])).float()


def _plain_logp(st):
    z, m, e, s = _rows(st)
    on = st["mask"] != 0
    out = {"logp": torch.where(on, _token_logp(st, z, m, s), 0.0)}
    if st["case"]["entropy"]:
        h = torch.log(s)[:, 0] - (e * (z - m)).sum(1) / s[:, 0]
        out["entropy"] = torch.where(on, h, 0.0)
    return out


def _plain_policy(st):
    case, on = st["case"], st["mask"].float()
    z, m, e, s = _rows(st)
    logp = _token_logp(st, z, m, s)
    r = st["rewards"].double().view(-1, case["group"])
    adv = ((r - r.mean(1, keepdim=True)) / (r.std(1, keepdim=True, unbiased=False) + ADV_EPS)).view(-1).float()
    A, w = adv[st["seq"]], _weights(st, on)
    d = st["logp_old"] - st["logp_infer"]
    rho = torch.where(d.abs() <= math.log(BETA_POP), torch.exp(d), 0.0)
    lr = logp - st["logp_old"]
    ratio = torch.exp(lr)
    clipped = torch.where(A > 0, lr > math.log1p(EPS_HIGH), (A < 0) & (lr < math.log1p(-EPS_LOW)))
    obj = rho * A * torch.where(clipped, ratio.clamp(1 - EPS_LOW, 1 + EPS_HIGH), ratio)
    grad = torch.where(clipped, 0.0, -rho * A * ratio)
    dk = (logp - st["logp_ref"]).double()  # a difference of near values, then one of nearer ones
    kl, dkl = {"k1": (dk, torch.ones_like(dk)), "k2": (0.5 * dk * dk, dk),
               "k3": (torch.expm1(-dk) + dk, -torch.expm1(-dk))}[case["estimator"]]
    loss = (w.double() * (case["coef"] * kl - obj)).sum()
    g = w * (grad + case["coef"] * dkl).float()
    return {"loss": loss.float(), "logp": logp, "kl": torch.where(on != 0, kl, 0.0).float(),
            "dlogits": _logits_grad(st, g, e, s)}


def _plain_distill(st):
    case, on = st["case"], st["mask"].float()
    tau = case["temperature"]
    z = st["logits"][:, :st["V"]].float() / tau
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    real = st["ids"] >= 0
    at = st["ids"].long().clamp_min(0)
    vals = st["vals"].double()
    ek = torch.where(real, e.gather(1, at), 0.0)
    rest = e.scatter(1, torch.where(real, at, at[:, :1]), 0.0).sum(1, keepdim=True)  # the entries outside the teacher's
    s = rest + ek.sum(1, keepdim=True)
    lp = torch.where(real, z.gather(1, at) - m - torch.log(s), 0.0).double()
    if case["mode"] == "renorm":
        lq = vals - torch.logsumexp(vals, 1, keepdim=True)
        q, qo = torch.exp(lq), torch.zeros_like(lq[:, :1])
    else:
        lq, q = vals, torch.exp(vals)
        qo = (1 - q.sum(1, keepdim=True)).clamp_min(1e-9)
    lq = torch.where(real, lq, 0.0)
    po = (rest / s).double()
    lo = torch.log(po) - torch.log(qo.clamp_min(1e-300))
    p = torch.exp(lp) * real
    if case["direction"] == "forward":
        kl = (q * (lq - lp)).sum(1) - (qo * lo)[:, 0] * (case["mode"] == "tail")
        total = q.sum(1, keepdim=True) + qo
        top, tail = total * p - q, total / s - qo / rest
    else:
        kl = (p * (lp - lq)).sum(1) + (po * lo)[:, 0]
        top, tail = p * (lp - lq - kl[:, None]), (lo - kl[:, None]) / s
    w = (_weights(st, on) / tau)[:, None]
    d = e * (w * tail).float()
    d.scatter_(1, torch.where(real, at, at[:, :1]), torch.where(real, w * top, (w * top)[:, :1]).float())
    loss = (_weights(st, on).double() * kl).sum()
    return {"loss": loss.float(), "kl": torch.where(on != 0, kl, 0.0).float(), "dlogits": d.to(st["logits"].dtype)}


def _plain_pref(st):
    case, on = st["case"], st["mask"].float()
    beta, margin, eps, nll = _pref_numbers(case)
    z, m, e, s = _rows(st)
    logp = _token_logp(st, z, m, s) * on
    n = _seq_sum(st, on)
    scale = 1 / n if case["mean"] else torch.ones_like(n)
    ref = st["logp_ref"] * on if st["logp_ref"] is not None else torch.zeros_like(logp)
    ratio = (_seq_sum(st, logp) - _seq_sum(st, ref)) * scale
    diff = ratio[0::2] - ratio[1::2]
    if case["kind"] == "sigmoid":
        h = beta * diff - margin
        lose, win = torch.log1p(torch.exp(-h.abs())) + (-h).clamp_min(0), torch.log1p(torch.exp(-h.abs())) + h.clamp_min(0)
        pair = (1 - eps) * lose + eps * win
        slope = beta * (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h))
    else:
        pair, slope = (diff - 1 / (2 * beta)) ** 2, 2 * (diff - 1 / (2 * beta))
    P = st["S"] // 2
    like = -_seq_sum(st, logp)[0::2] / n[0::2]
    loss = (pair + nll * like).sum() / P
    g = torch.stack([slope * scale[0::2] - nll / n[0::2], -slope * scale[1::2]], 1).view(-1) / P
    return {"loss": loss.float(), "logp": logp, "ratio": ratio.float(), "pair": (pair + nll * like).float(),
            "dlogits": _logits_grad(st, g.float()[st["seq"]] * on, e, s)}


_plain = {"logp": _plain_logp, "policy": _plain_policy, "distill": _plain_distill, "pref": _plain_pref}


# ---------------------------------------------------------------------------- the same through the library

def _library_logp(st):
    from rl_post_loss_gb300 import capi
    logp, entropy = capi.token_logp(st["logits"], st["targets"], st["mask"], vocab=st["V"], logp=st["logp"],
                                    want_entropy=st["case"]["entropy"])
    return {"logp": logp, "entropy": entropy} if st["case"]["entropy"] else {"logp": logp}


def _library_policy(st):
    case = st["case"]
    dev = st["logits"].device
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    kl = torch.empty(st["T"], dtype=torch.float32, device=dev)
    st["rl"].forward_backward_kl(st["logits"], st["targets"], st["logp_old"], st["logp_infer"], st["mask"], st["cu"],
                                 st["rewards"], st["logp_ref"], kl_coef=case["coef"], kl_estimator=case["estimator"],
                                 loss=loss, dlogits=st["dlogits"], logp=st["logp"], kl=kl)
    return {"loss": loss[0], "logp": st["logp"], "kl": kl, "dlogits": st["dlogits"][:, :st["V"]]}


def _library_distill(st):
    from rl_post_loss_gb300 import capi
    case = st["case"]
    out = capi.distill_loss(st["logits"], st["ids"], st["vals"], st["mask"], st["cu"], vocab=st["V"], mode=case["mode"],
                            direction=case["direction"], temperature=case["temperature"], tail_floor=1e-9,
                            loss_norm=capi.RL_NORM_PER_TOKEN if case["per_token"] else capi.RL_NORM_PER_RESPONSE,
                            dlogits=st["dlogits"])
    return {"loss": out["loss"][0], "kl": out["kl"], "dlogits": out["dlogits"][:, :st["V"]]}


def _library_pref(st):
    from rl_post_loss_gb300 import capi
    case = st["case"]
    beta, margin, eps, nll = _pref_numbers(case)
    out = capi.preference_loss(st["logits"], st["targets"], st["logp_ref"], st["mask"], st["cu"], vocab=st["V"],
                               loss_type=case["kind"], length_norm=case["mean"], beta=beta, margin=margin,
                               label_smoothing=eps, nll_coef=nll, dlogits=st["dlogits"], logp=st["logp"])
    return {"loss": out["loss"][0], "logp": out["logp"], "ratio": out["seq_logratio"], "pair": out["pair_loss"],
            "dlogits": out["dlogits"][:, :st["V"]]}


_library = {"logp": _library_logp, "policy": _library_policy, "distill": _library_distill, "pref": _library_pref}


# ---------------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    T, S, V, op = st["T"], st["S"], st["V"], case["op"]
    cu = st["cu"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    mask = st["mask"].double()
    n = torch.stack([mask[a:b].sum() for a, b in zip(cu, cu[1:])])
    owner = st["seq"]
    step = max(1, (1 << 27) // V)
    blocks = [slice(a, min(T, a + step)) for a in range(0, T, step)]
    z64 = lambda b: st["logits"][b, :V].double()  # noqa: E731

    if op == "distill":
        return _exact_distill(st, case, mask, n, blocks, z64, f64)

    y = st["targets"].long()
    logp, ent = torch.empty(T, **f64), torch.empty(T, **f64)
    for b in blocks:
        lsm = z64(b)
        lsm -= torch.logsumexp(lsm, 1, keepdim=True)
        logp[b] = lsm.gather(1, y[b, None])[:, 0]
        if op == "logp" and case["entropy"]:
            ent[b] = -(lsm.exp() * lsm).sum(1)
    if op == "logp":
        out = {"logp": logp * mask}
        if case["entropy"]:
            out["entropy"] = ent * mask
        return out

    if op == "policy":
        w = mask / n.sum() if case["per_token"] else mask / (S * n[owner])
        R = st["rewards"].double().view(-1, case["group"])
        sd = (R - R.mean(1, keepdim=True)).square().mean(1, keepdim=True).sqrt()
        A = ((R - R.mean(1, keepdim=True)) / (sd + ADV_EPS)).reshape(-1)[owner]
        gap = st["logp_old"] - st["logp_infer"]  # the interval is decided on the 32-bit difference
        inside = gap.abs() <= torch.tensor(math.log(BETA_POP), device="cuda")
        rho = (st["logp_old"].double() - st["logp_infer"].double()).exp() * inside
        r = (logp - st["logp_old"].double()).exp()
        cut = r.clamp(1 - EPS_LOW, 1 + EPS_HIGH)
        low = cut * A < r * A
        obj = rho * torch.where(low, cut * A, r * A)
        D = logp - st["logp_ref"].double()
        if case["estimator"] == "k1":
            kl, dkl = D, torch.ones_like(D)
        elif case["estimator"] == "k2":
            kl, dkl = D * D / 2, D
        else:
            kl, dkl = torch.expm1(-D) + D, 1 - torch.exp(-D)
        out = {"loss": (w * (case["coef"] * kl - obj)).sum(), "logp": logp, "kl": kl * mask}
        g = w * (case["coef"] * dkl - torch.where(low, torch.zeros_like(r), rho * A * r))
    else:
        beta, margin, eps, nll = _pref_numbers(case)
        ref = st["logp_ref"].double() if st["logp_ref"] is not None else torch.zeros(T, **f64)
        tot = torch.stack([((logp - ref) * mask)[a:b].sum() for a, b in zip(cu, cu[1:])])
        like = torch.stack([-(logp * mask)[a:b].sum() for a, b in zip(cu, cu[1:])])[0::2] / n[0::2]
        per = n if case["mean"] else torch.ones_like(n)
        ratio = tot / per
        diff = ratio[0::2] - ratio[1::2]
        if case["kind"] == "sigmoid":
            h = beta * diff - margin
            pair = -(1 - eps) * torch.log(torch.sigmoid(h)) - eps * torch.log(torch.sigmoid(-h))
            slope = beta * (torch.sigmoid(h) - (1 - eps))
        else:
            pair, slope = (diff - 0.5 / beta) ** 2, 2 * diff - 1 / beta
        P = S // 2
        pair = pair + nll * like
        coef = torch.zeros(S, **f64)
        coef[0::2] = (slope / per[0::2] - nll / n[0::2]) / P
        coef[1::2] = -slope / per[1::2] / P
        g = coef[owner] * mask
        out = {"loss": pair.mean(), "logp": logp * mask, "ratio": ratio, "pair": pair}

    dz = torch.empty((T, V), **f64)
    for b in blocks:
        p = torch.softmax(z64(b), 1).neg_()
        p.scatter_add_(1, y[b, None], torch.ones_like(p[:, :1]))
        dz[b] = p.mul_(g[b, None])
    out["dlogits"] = dz
    return out


def _exact_distill(st, case, mask, n, blocks, z64, f64):
    T, S, V, tau = st["T"], st["S"], st["V"], case["temperature"]
    w = mask / n.sum() if case["per_token"] else mask / (S * n[st["seq"]])
    kl, dz = torch.empty(T, **f64), torch.empty((T, V), **f64)
    for b in blocks:
        lp = z64(b).div_(tau)
        lp -= torch.logsumexp(lp, 1, keepdim=True)
        # the teacher's log-probs over the vocabulary, and a truth value for its own entries
        rows, cols = (st["ids"][b] >= 0).nonzero(as_tuple=True)
        at = st["ids"][b].long()[rows, cols]
        lq = torch.full_like(lp, -math.inf)
        lq[rows, at] = st["vals"][b].double()[rows, cols]
        if case["mode"] == "renorm":
            lq -= torch.logsumexp(lq, 1, keepdim=True)
        top = lq > -math.inf
        q, p = lq.exp(), lp.exp()
        qo = (1 - q.sum(1, keepdim=True)).clamp_min(1e-9) if case["mode"] == "tail" else torch.zeros_like(lp[:, :1])
        po = torch.where(top, 0.0, p).sum(1, keepdim=True)
        if case["direction"] == "forward":
            kl[b] = torch.where(top, q * (lq - lp), 0.0).sum(1)
            d = p * (q.sum(1, keepdim=True) + qo) - q
            if case["mode"] == "tail":
                kl[b] += (qo * (qo.log() - po.log()))[:, 0]
                d -= torch.where(top, 0.0, p * qo / po)
        else:
            a = torch.where(top, lp - torch.where(top, lq, 0.0), (po / qo).log())
            kl[b] = torch.where(top, p * a, 0.0).sum(1) + (po * (po / qo).log())[:, 0]
            d = p * (a - kl[b, None])
        dz[b] = d.mul_(w[b, None] / tau)
    return {"loss": (w * kl).sum(), "kl": kl * mask, "dlogits": dz}


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    lengths = _lengths(case)
    T, S, V, op = sum(lengths), len(lengths), case["vocab"], case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    used = T * (1 - case["masked"])  # rows whose logits are needed (the masked share is drawn around this)
    if op == "logp":
        return {"bytes": used * V * es + T * (4 + 1 + 4 + (4 if case["entropy"] else 0)),
                "flops": used * V * (5 if case["entropy"] else 3)}
    if op == "policy":  # the log-probs of masked tokens are returned too
        return {"bytes": 2 * T * V * es + T * (4 * 4 + 1 + 8) + S * 8, "flops": T * V * 6}
    if op == "distill":
        return {"bytes": (used + T) * V * es + T * (case["k"] * 8 + 1 + 4) + S * 4, "flops": used * V * 6}
    return {"bytes": (used + T) * V * es + T * (4 + 4 + 1 + 4) + S * 12, "flops": used * V * 6}
