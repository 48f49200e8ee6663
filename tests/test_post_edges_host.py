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
