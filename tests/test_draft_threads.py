"""Calls of several host threads on one stream, without a GPU: stand-ins for the
library's calls note what they are given."""

import os
import threading

import pytest
import torch

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(R, "_is_elsewhere", lambda stream, dev: False)
    monkeypatch.setattr(R, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(R, "_capturing", lambda: False)


def verify(seqs, vocab=50):
    b = R.kv_batch([2] * seqs, [9] * seqs, [[0]] * seqs, device="cpu")
    i, f = torch.zeros(2 * seqs, dtype=torch.int32), torch.zeros(2 * seqs)
    return R.verify(b, i, i, torch.zeros(2 * seqs, vocab), f, f[:seqs])


def test_verify_calls_under_way_at_once_share_no_workspace(on_host, monkeypatch):
    """pi_verify is two launches, and the second reads what the first left in the workspace: another
    thread's call on the same stream may lie between them."""
    both, seen = threading.Barrier(2, timeout=30), []

    def pi_verify(n_seq, n_tok, vocab, *a):
        ws, size = a[-3], a[-2]
        assert size >= B.pi_verify_workspace_size(n_seq, n_tok, vocab) and ws.numel() * ws.element_size() >= size
        seen.append((ws.data_ptr(), ws.data_ptr() + size))
        both.wait()   # both calls are inside the library
        return B.PI_OK

    monkeypatch.setattr(B, "pi_verify", pi_verify)
    failed = []

    def work(seqs):
        try:
            for _ in range(3):
                verify(seqs)
        except Exception as e:   # a thread's exception would be lost
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in (3, 40)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(seen) == 6
    for i in range(0, 6, 2):   # the two that were under way together
        (a0, a1), (b0, b1) = seen[i:i + 2]
        assert a1 <= b0 or b1 <= a0


def test_a_threads_verify_calls_share_a_workspace(on_host, monkeypatch):
    seen = []
    monkeypatch.setattr(B, "pi_verify", lambda *a: seen.append(a[-3].data_ptr()) or B.PI_OK)
    for seqs in (20, 3, 20):
        verify(seqs)
    assert len(set(seen)) == 1
