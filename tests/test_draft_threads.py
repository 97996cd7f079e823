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


class Growing:
    """A kept workspace that another thread replaces by a larger one after its first reading."""

    def __init__(self):
        self.bufs = [torch.zeros(64, dtype=torch.uint8), torch.zeros(1 << 30, dtype=torch.uint8, device="meta")]

    @property
    def buf(self):
        return self.bufs.pop(0) if len(self.bufs) > 1 else self.bufs[0]

    def get(self, nbytes):
        b = torch.zeros(nbytes, dtype=torch.uint8)
        return b, nbytes


@pytest.mark.parametrize("tree", [False, True])
def test_a_workspace_replaced_meanwhile_is_not_taken_for_the_larger(on_host, monkeypatch, tree):
    """What the library is told of a workspace's size is that of the buffer it gets."""
    seen = []

    def note(a):
        ws, size = a[-3], a[-2]
        seen.append((0 if ws is None else ws.numel(), size))
        return B.PI_OK if size >= 4096 else B.PI_ERR_WORKSPACE

    monkeypatch.setattr(B, "pi_kv_attend", lambda *a: note(a))
    monkeypatch.setattr(B, "pi_kv_attend_tree", lambda *a: note(a))
    device = torch.device("cpu")
    monkeypatch.setattr(R, "_KV_WS", {(d, 7): Growing() for d in (device.index, -1)})
    c, b = R.kv_cache(4, 2, 64, device="cpu"), R.kv_batch([1], [5], [[0]], device="cpu")
    q, x = torch.zeros(1, 4, 64).half(), torch.zeros(1, 2, 64).half()
    if tree:
        R.kv_attend_tree(c, q, x, x, b, torch.ones(1, 1, dtype=torch.int64))
    else:
        R.kv_attend(c, q, b)
    assert seen and all(have == told for have, told in seen)


def test_a_grown_workspace_is_returned_with_its_own_size():
    class Racing(R.Workspace):
        """Every reading of buf after the first finds a larger one."""
        def __init__(self):
            super().__init__("cpu")
            self.reads = 0

        def __getattribute__(self, name):
            if name != "buf" or "reads" not in super().__getattribute__("__dict__"):
                return super().__getattribute__(name)
            self.reads += 1
            return torch.zeros(256 * self.reads, dtype=torch.uint8)

    w = Racing()
    buf, size = w.get(100)
    assert buf.numel() == size
