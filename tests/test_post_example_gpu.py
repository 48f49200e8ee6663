"""The post-training losses used together, as examples/post_training.py does, and on a stream given by address."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
from rl_post_loss_gb300 import capi  # noqa: E402

pytestmark = pytest.mark.gpu


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "post_training.py")
    spec = importlib.util.spec_from_file_location("post_training_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("vocab", [5003, 4096])
def test_the_example_lowers_each_loss(vocab):
    report = load_example().main(vocab=vocab, steps=8)
    assert report["status"] == [0]
    assert report["KL to the reference"][0] == pytest.approx(0.0, abs=1e-6)  # the first step is the reference
    assert max(report["KL to the reference"]) > 0.0
    for name in ("policy loss", "distillation loss", "preference loss"):
        assert report[name][-1] < report[name][0], name


def test_outputs_that_a_call_allocates_belong_to_its_stream():
    """With stream=: the outputs left out come from that stream's memory, the current stream stays as it was,
    and the values are those of the current stream."""
    V, T = 1000, 12
    g = torch.Generator().manual_seed(3)
    z = torch.randn(T, V, generator=g).cuda()
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 5, T], dtype=torch.int32, device="cuda")
    ids = torch.topk(z, 4, dim=1).indices.to(torch.int32).contiguous()
    vals = torch.gather(z, 1, ids.long()).contiguous()
    calls = [lambda s: dict(zip(("logp", "entropy"), capi.token_logp(z, y, mask, want_entropy=True, stream=s))),
             lambda s: capi.distill_loss(z, ids, vals, mask, cu, stream=s),
             lambda s: capi.preference_loss(z, y, None, mask, cu, stream=s)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        before = torch.cuda.current_stream()
        got = call(side.cuda_stream)
        assert torch.cuda.current_stream() == before
        side.synchronize()
        for name in want:
            assert torch.equal(want[name], got[name]), name
