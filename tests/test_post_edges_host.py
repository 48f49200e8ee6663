"""The post-training losses' binding without a GPU: what it keeps between calls."""
import threading

import pytest

torch = pytest.importorskip("torch")
from rl_post_loss_gb300 import capi  # noqa: E402


def test_threads_do_not_share_a_workspace(monkeypatch):
    """Two threads that enqueue on one stream: a call's launches hand results on in its workspace."""
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    cpu, stream = torch.device("cpu"), 7
    kept, both = {}, threading.Barrier(2, timeout=30)

    def work(name):
        first = capi._post_workspace(1000, cpu, stream)
        both.wait()
        kept[name] = first, capi._post_workspace(2000, cpu, stream), capi._post_workspace(1000, cpu, stream + 1)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert sorted(kept) == [0, 1]
    for first, again, other in kept.values():
        assert again is first and other is not first  # kept between a thread's calls, by stream
    assert kept[0][0] is not kept[1][0]
    grown = capi._post_workspace(1 << 20, cpu, stream)
    assert grown.numel() >= 1 << 20 and capi._post_workspace(10, cpu, stream) is grown


def test_status_words_and_workspaces_are_checked():
    """Of the right place, size and layout, whatever the call: checked on CPU tensors, whose device index is None / -1."""
    here = torch.device("cuda", 0)
    word, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    assert capi._status_word(None, here) is None
    with pytest.raises(ValueError, match="device_status"):
        capi._status_word(word, here)
    with pytest.raises(ValueError, match="workspace"):
        capi._workspace_of(ws, here)


def test_loss_with_kl_refuses_logits_that_are_not_on_a_gpu():
    rl = capi.RlLoss.__new__(capi.RlLoss)
    rl.handle = None
    rl.config = capi.rl_loss_config(8, 1, 4, 1)
    z, f = torch.zeros(4, 8), torch.zeros(4)
    y, cu = torch.zeros(4, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rl.forward_backward_kl(z, y, f, f, y.to(torch.uint8), cu, f[:1], f, kl_coef=0.1, loss=f[:1], dlogits=z)
