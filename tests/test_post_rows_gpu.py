"""The post-training losses where their rows change ways: rows a warp takes by itself (up to 24 KB) and rows over
rings, on either side of the border, with many rows per cluster; a row's outputs do not depend on its place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import test_post_ops_gpu as ops  # noqa: E402
from rl_post_loss_gb300 import capi  # noqa: E402

pytestmark = pytest.mark.gpu

BORDER = [(12288, "bf16"), (12295, "bf16"), (12296, "bf16"), (6144, "f32"), (6147, "f32"), (6149, "f32")]
MANY = [(1300, 12801, "bf16"), (1700, 6401, "f32"), (900, 25013, "bf16"), (2100, 4096, "bf16")]


@pytest.mark.parametrize("V,dtype", BORDER)
def test_token_logp_at_the_border(V, dtype):
    ops.test_token_logp(90, V, 1, dtype)


@pytest.mark.parametrize("T,V,dtype", MANY)
def test_token_logp_of_many_rows(T, V, dtype):
    ops.test_token_logp(T, V, 0, dtype)


@pytest.mark.parametrize("mode,reverse,tau", [("renorm", 0, 2.0), ("tail", 0, 1.0), ("tail", 1, 1.0)])
@pytest.mark.parametrize("K", [5, 130])
@pytest.mark.parametrize("V,dtype", BORDER)
def test_distill_at_the_border(V, dtype, K, mode, reverse, tau):
    ops.test_distill(30, V, K, mode, reverse, tau, dtype)


@pytest.mark.parametrize("mode,reverse,tau", [("renorm", 0, 1.0), ("tail", 1, 1.0)])
@pytest.mark.parametrize("T,V,dtype", MANY)
def test_distill_of_many_rows(T, V, dtype, mode, reverse, tau):
    ops.test_distill(T, V, 40, mode, reverse, tau, dtype)


@pytest.mark.parametrize("V,dtype", BORDER)
def test_preference_at_the_border(V, dtype):
    ops.check_pref([7, 0, 21, 9], V, dtype, "sigmoid", 1, True)


@pytest.mark.parametrize("T,V,dtype", MANY)
def test_preference_of_many_rows(T, V, dtype):
    a = T // 8
    ops.check_pref([a, 2 * a, 1, 3 * a, 0, T - 6 * a - 1], V, dtype, "sigmoid", 0, True)


@pytest.mark.parametrize("case_id,V,lengths", [
    (0, 6144, [9, 4, 0, 7, 12, 1, 30, 5]), (0, 6147, [9, 4, 0, 7, 12, 1, 30, 5]), (0, 6149, [9, 4, 0, 7, 12, 1, 30, 5]),
    (1, 12288, [9, 4, 0, 7, 12, 1, 30, 5]), (1, 12296, [9, 4, 0, 7, 12, 1, 30, 5]),
    (1, 12801, [160, 90, 400, 31, 250, 70, 3, 120]), (0, 6401, [160, 90, 400, 31, 250, 70, 3, 120]),
    (1, 4096, [160, 90, 700, 31, 250, 70, 3, 520]), (2, 25013, [100, 90, 200, 31, 50, 70, 3, 120])])
def test_loss_with_kl_at_the_border_and_of_many_rows(case_id, V, lengths, monkeypatch):
    monkeypatch.setattr(ops, "KLC", [(case_id, lengths, V, {})])
    ops.test_loss_with_kl(0, "k3")


@pytest.mark.parametrize("V,dtype", [(4099, "bf16"), (12801, "bf16"), (4097, "f32"), (6401, "f32")])
def test_a_row_does_not_depend_on_its_place(V, dtype):
    """The same row at two places of a batch: the same bits. (How a row is cut depends on the number of rows.)"""
    g = torch.Generator().manual_seed(5)
    T, K = 1100, 9
    z = ops.logits_of(T, V, dtype, 3).cuda()
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    z[700], y[700] = z[2], y[2]
    one = torch.ones(T, dtype=torch.uint8, device="cuda")
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]).to(torch.int32).cuda()
    ids[700] = ids[2]
    vals = torch.log_softmax(torch.randn(T, K, generator=g), 1).cuda() - 0.1
    vals[700] = vals[2]

    def outputs(rows):
        n = len(rows)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        zc, yc, m = z[rows].contiguous(), y[rows].contiguous(), one[:n].contiguous()
        logp, ent = capi.token_logp(zc, yc, m, vocab=V, want_entropy=True)
        out = capi.distill_loss(zc, ids[rows].contiguous(), vals[rows].contiguous(), m, cu, vocab=V, mode="tail",
                                direction="reverse", tail_floor=1e-6, scale=float(n), loss_norm=capi.RL_NORM_PER_TOKEN)
        return logp, ent, out["kl"], out["dlogits"][:, :V]

    for a in outputs(list(range(T))):
        assert torch.equal(a[2], a[700])
