"""Where the buffers of the 4-bit step come from when a call names its stream, without a GPU."""

import contextlib

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def skv():
    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


class Step:
    """A Kv4Step whose calls reach no GPU, and the stream that each of its allocations is made under."""

    def __init__(self, skv, monkeypatch):
        from top_sparse_kv_gb300 import binding, step

        p = skv.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=5, n_sink=1, n_local=2,
                        block_size=16, seq_lens=torch.zeros(4, dtype=torch.int32))
        self.step = skv.Kv4Step(p, skv.Kv4Pool.empty(10, 2, 16, torch.zeros((4, 7), dtype=torch.int32)))
        self.q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
        self.made, self.current = [], None
        empty = torch.empty

        def recorded(*args, **kw):
            self.made.append(self.current)
            return empty(*args, **kw)

        @contextlib.contextmanager
        def under(stream):
            old, self.current = self.current, stream
            yield
            self.current = old

        monkeypatch.setattr(torch, "empty", recorded)
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(binding, "raw_stream", lambda device, stream=None: 0)
        monkeypatch.setattr(binding, "skv_topk", lambda *args: None)
        assert step.B is binding
        for name in ("_score", "_attn", "_step", "_gather"):
            monkeypatch.setattr(self.step, name, lambda *args: 0)


CALLS = {
    "score": lambda s, q, st: s.score(q, stream=st),
    "topk": lambda s, q, st: s.topk(stream=st),
    "attend": lambda s, q, st: s.attend(q, stream=st),
    "attend_all": lambda s, q, st: s.attend_all(q, stream=st),
    "run": lambda s, q, st: s.run(q, stream=st),
    "gather": lambda s, q, st: s.gather(stream=st),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_first_call_on_a_stream(skv, monkeypatch, name):
    """Whatever a first call allocates comes from the pool of the stream that writes it: the current stream's may
    hand out memory that work of its own, queued before, has still to use."""
    s = Step(skv, monkeypatch)
    CALLS[name](s.step, s.q, "side")
    assert all(x == "side" for x in s.made), s.made
    if name == "run":
        assert s.step.scores.shape == (4, 2, 100) and s.step.idx.shape == (4, 2, 5)
    made = len(s.made)
    CALLS[name](s.step, s.q, "other")  # what the step owns is there now
    assert s.made[made:] == (["other"] * 2 if name == "gather" else [])


def test_without_a_stream(skv, monkeypatch):
    s = Step(skv, monkeypatch)
    assert s.step.score(s.q) is s.step.scores and s.step.run(s.q)[0] is s.step.out and s.step.topk() is s.step.idx
    assert set(s.made) == {None}
