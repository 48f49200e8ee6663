"""Post-training operators without a GPU: the refusals of their entry points, and the 64-bit gradients the
GPU tests compare with, against differences of the 64-bit losses."""
import ctypes

import numpy as np
import pytest

import post_helpers as ph
from rl_post_loss_gb300 import build as nvbuild
from rl_post_loss_gb300 import capi

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every check below returns before any CUDA call
C = capi.CODES


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return capi.load()


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "rl_loss.h"\nint main(void) {\n'
    structs = (capi.rl_loss_kl, capi.rl_loss_distill_config, capi.rl_loss_pref_config)
    for s in structs:
        src += f'printf("%zu\\n", sizeof({s.__name__}));\n'
        for name, _ in s._fields_:
            src += f'printf("%zu\\n", offsetof({s.__name__}, {name}));\n'
    (tmp_path / "a.c").write_text(src + "return 0; }\n")
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"), "-o",
                           str(tmp_path / "a")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "a")]).split()]
    want = []
    for s in structs:
        want.append(ctypes.sizeof(s))
        want += [getattr(s, name).offset for name, _ in s._fields_]
    assert got == want


def test_token_logp_refusals(lib):
    def call(dtype=capi.RL_BF16, T=4, V=64, logits=FAKE, ld=64, targets=FAKE, logp=FAKE, entropy=None):
        return lib.rl_loss_token_logp(dtype, T, V, logits, ld, targets, None, logp, entropy, None, None)
    assert call(dtype=5) == C["RL_ERR_DTYPE"]
    assert call(T=-1) == C["RL_ERR_SHAPE"]
    assert call(V=0) == C["RL_ERR_SHAPE"]
    assert call(V=1 << 24) == C["RL_ERR_SHAPE"]
    assert call(ld=63) == C["RL_ERR_SHAPE"]
    assert call(ld=65) == C["RL_ERR_ALIGNMENT"]
    assert call(logits=ctypes.c_void_p(0x10008)) == C["RL_ERR_ALIGNMENT"]
    assert call(logits=None) == C["RL_ERR_INVALID_ARG"]
    assert call(targets=None) == C["RL_ERR_INVALID_ARG"]
    assert call(logp=None) == C["RL_ERR_INVALID_ARG"]
    assert call(logp=ctypes.c_void_p(0x10002)) == C["RL_ERR_ALIGNMENT"]
    assert call(T=0, logits=None, targets=None, logp=None) == 0


def test_distill_refusals(lib):
    T, S = 4, 2
    need = capi.rl_loss_distill_workspace_bytes(T, S)
    good = dict(dtype=capi.RL_F32, V=64, k=4, mode=1, reverse=0, norm=0, tau=1.0, scale=1.0, floor=0.0)

    def call(T=T, S=S, logits=FAKE, ld=64, ids=FAKE, ldk=4, mask=FAKE, cu=FAKE, loss=FAKE, dz=FAKE, ldd=64, ws=FAKE,
             nbytes=need, **over):
        c = dict(good, **over)
        cfg = capi.rl_loss_distill_config(c["dtype"], c["V"], c["k"], c["mode"], c["reverse"], c["norm"], c["tau"],
                                          c["scale"], c["floor"])
        return lib.rl_loss_distill(ctypes.byref(cfg), T, S, logits, ld, ids, FAKE, ldk, mask, cu, loss, None, dz, ldd,
                                   None, ws, nbytes, None, None)
    assert lib.rl_loss_distill_max_k() == 1024
    assert call(dtype=9) == C["RL_ERR_DTYPE"]
    for over in (dict(T=-1), dict(S=0), dict(V=0), dict(ld=60), dict(ldd=60), dict(ldk=3)):
        assert call(**over) == C["RL_ERR_SHAPE"], over
    for over in (dict(k=0), dict(k=1025, ldk=2000), dict(mode=0, reverse=1)):
        assert call(**over) == C["RL_ERR_UNSUPPORTED"], over
    nan, inf = float("nan"), float("inf")
    for over in (dict(mode=2), dict(reverse=2), dict(norm=2), dict(tau=0.0), dict(tau=nan), dict(tau=inf), dict(scale=inf),
                 dict(floor=1.0), dict(floor=-1e-9), dict(floor=nan), dict(logits=None), dict(ids=None), dict(mask=None),
                 dict(cu=None), dict(loss=None), dict(dz=None), dict(ws=None), dict(dz=FAKE, ldd=68)):
        assert call(**over) == C["RL_ERR_INVALID_ARG"], over
    for over in (dict(logits=ctypes.c_void_p(0x10004)), dict(ld=66), dict(ws=ctypes.c_void_p(0x10010)),
                 dict(ids=ctypes.c_void_p(0x10001))):
        assert call(**over) == C["RL_ERR_ALIGNMENT"], over
    assert call(nbytes=need - 1) == C["RL_ERR_CAPACITY"]
    assert lib.rl_loss_distill(None, T, S, FAKE, 64, FAKE, FAKE, 4, FAKE, FAKE, FAKE, None, FAKE, 64,
                               None, FAKE, need, None, None) == C["RL_ERR_INVALID_ARG"]


def test_preference_refusals(lib):
    T, S = 4, 2
    need = capi.rl_loss_preference_workspace_bytes(T, S)
    good = dict(dtype=capi.RL_BF16, V=64, kind=0, mean=0, beta=0.1, margin=0.0, eps=0.0, nll=0.0)

    def call(T=T, S=S, logits=FAKE, ld=64, targets=FAKE, mask=FAKE, cu=FAKE, loss=FAKE, dz=ctypes.c_void_p(0x20000), ldd=64,
             ws=FAKE, nbytes=need, **over):
        c = dict(good, **over)
        cfg = capi.rl_loss_pref_config(c["dtype"], c["V"], c["kind"], c["mean"], c["beta"], c["margin"], c["eps"], c["nll"])
        return lib.rl_loss_preference(ctypes.byref(cfg), T, S, logits, ld, targets, None, mask, cu, loss, None, dz, ldd,
                                      None, None, None, ws, nbytes, None, None)
    assert call(dtype=2) == C["RL_ERR_DTYPE"]
    for over in (dict(S=1), dict(S=3), dict(S=0), dict(T=-1), dict(V=0), dict(ld=56), dict(ldd=56)):
        assert call(**over) == C["RL_ERR_SHAPE"], over
    nan, inf = float("nan"), float("inf")
    for over in (dict(kind=3), dict(mean=2), dict(beta=0.0), dict(beta=nan), dict(margin=inf), dict(eps=0.5), dict(eps=-0.1),
                 dict(nll=-1.0), dict(nll=inf), dict(logits=None), dict(targets=None), dict(mask=None), dict(cu=None),
                 dict(loss=None), dict(dz=None), dict(ws=None), dict(dz=FAKE, ldd=72)):
        assert call(**over) == C["RL_ERR_INVALID_ARG"], over
    for over in (dict(ld=68), dict(dz=ctypes.c_void_p(0x10002)), dict(ws=ctypes.c_void_p(0x10080))):
        assert call(**over) == C["RL_ERR_ALIGNMENT"], over
    assert call(nbytes=need - 1) == C["RL_ERR_CAPACITY"]


def test_kl_refusals(lib):
    inp, out = capi.rl_loss_inputs(), capi.rl_loss_outputs()
    args = lambda kl: (None, ctypes.byref(inp), kl, ctypes.byref(out), None)
    assert lib.rl_loss_forward_backward_kl(*args(None)) == C["RL_ERR_INVALID_ARG"]
    for coef, est in ((-1.0, 0), (float("nan"), 0), (float("inf"), 0), (0.1, 3), (0.1, -1), (0.1, 2)):
        kl = capi.rl_loss_kl(FAKE, coef, est, None, None)  # the last one fails for the missing handle
        assert lib.rl_loss_forward_backward_kl(*args(ctypes.byref(kl))) == C["RL_ERR_INVALID_ARG"]


def test_python_argument_checks():
    import torch
    z = torch.zeros(3, 8)
    y = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        capi.token_logp(z, y)
    with pytest.raises(ValueError, match="mode"):
        capi.distill_loss(z, y, y, y, y, mode="other")
    with pytest.raises(ValueError, match="loss_type"):
        capi.preference_loss(z, y, None, y, y, loss_type="other")


# ---------------------------------------------------------------- the 64-bit gradients against differences

def _central(f, z, direction, h=1e-5):
    return (f(z + h * direction) - f(z - h * direction)) / (2 * h)


@pytest.mark.parametrize("mode,reverse", [("renorm", 0), ("tail", 0), ("tail", 1)])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_gradient_against_differences(mode, reverse, tau):
    rng = np.random.default_rng(3)
    T, V, K = 4, 23, 5
    z = rng.normal(size=(T, V)) * 2
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    ids[1, 3:] = -1
    vals = np.log(rng.dirichlet(np.ones(K + 1), size=T)[:, :K]).astype(np.float32)
    mask = np.array([1, 1, 0, 1], np.uint8)
    cu = np.array([0, 2, 4])
    f = lambda x: ph.distill(x, ids, vals, mask, cu, mode, reverse, tau, 1.7, 1e-6, False)[0]
    d = ph.distill(z, ids, vals, mask, cu, mode, reverse, tau, 1.7, 1e-6, False)[2]
    for seed in range(3):
        u = np.random.default_rng(seed).normal(size=z.shape)
        assert _central(f, z, u) == pytest.approx((d * u).sum(), rel=1e-6, abs=1e-9)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("mean", [0, 1])
def test_preference_gradient_against_differences(kind, mean):
    rng = np.random.default_rng(4)
    T, V = 9, 17
    z = rng.normal(size=(T, V))
    y = rng.integers(0, V, T)
    ref = rng.normal(size=T)
    mask = np.array([1, 1, 0, 1, 1, 1, 0, 1, 1], np.uint8)
    cu = np.array([0, 3, 5, 6, 9])
    args = (y, ref, mask, cu, kind, mean, 0.3, 0.1, 0.05, 0.2)
    f = lambda x: ph.preference(x, *args)["loss"]
    q = ph.preference(z, *args)
    d, _ = ph.onehot_grad(q["rows"], q["g"], y, np.zeros(T), np.zeros(T), "f32")
    for seed in range(3):
        u = np.random.default_rng(seed).normal(size=z.shape)
        assert _central(f, z, u) == pytest.approx((d * u).sum(), rel=1e-6, abs=1e-9)


@pytest.mark.parametrize("kind", ["k1", "k2", "k3"])
def test_kl_gradient_against_differences(kind):
    rng = np.random.default_rng(5)
    T, V = 6, 13
    z = rng.normal(size=(T, V))
    y = rng.integers(0, V, T)
    ref = np.log(1.0 / V) + 0.4 * rng.normal(size=T)
    mask = np.array([1, 0, 1, 1, 1, 1], np.uint8)
    w, _ = ph.weights(mask, np.array([0, 2, 6]), False)

    def part(x):
        r = ph.Rows(x)
        return ph.kl_loss_part(r.lp[np.arange(T), y], ref, mask, w, kind, 0.3)
    g = part(z)[2]
    d, _ = ph.onehot_grad(ph.Rows(z), g, y, np.zeros(T), np.zeros(T), "f32")
    u = rng.normal(size=z.shape)
    assert _central(lambda x: part(x)[0], z, u) == pytest.approx((d * u).sum(), rel=1e-6, abs=1e-9)
