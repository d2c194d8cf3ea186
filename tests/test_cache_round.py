"""run_round_cached's order of calls and what it does with refused requests,
without a GPU: the library's calls are replaced."""

import types

import pytest

torch = pytest.importorskip("torch")


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


class Cache:
    def __init__(self, granted, log):
        self.granted, self.log = granted, log

    def reserve(self, ell, gamma):
        self.log.append(("reserve", ell.tolist(), gamma))
        return self.granted

    def commit(self, n_acc):
        self.log.append(("commit", n_acc.tolist()))


def test_a_refused_request_keeps_its_anchor(monkeypatch):
    from semi_ar_draft_round_amd import device_round as DR
    log = []
    d = types.SimpleNamespace(gamma=4, x0=i32(30, 40, 50, 60), ell=i32(3, 2, 1, 0), n_acc=i32(0, 0, 0, 0),
                              next_tok=i32(0, 0, 0, 0))

    def verify(d, ell=None):
        log.append(("verify", (d.ell if ell is None else ell).tolist()))
        d.n_acc.copy_(i32(2, 1, 1, 0))
        d.next_tok.copy_(i32(7, 8, 9, 10))

    monkeypatch.setattr(DR, "sample_conf", lambda d: log.append(("draft",)))
    monkeypatch.setattr(DR, "schedule", lambda d: log.append(("schedule",)))
    monkeypatch.setattr(DR, "verify", verify)
    DR.run_round_cached(d, Cache(i32(3, -1, 1, -1), log), lambda d, cache, ell: log.append(("forward", ell.tolist())))
    assert d.next_tok.tolist() == [7, 40, 9, 60]       # refused: drafts from the same anchor again
    assert d.n_acc.tolist() == [2, -1, 1, -1]
    assert d.x0.tolist() == [30, 40, 50, 60]
    assert log == [("draft",), ("schedule",), ("reserve", [3, 2, 1, 0], 4), ("forward", [3, -1, 1, -1]),
                   ("verify", [3, -1, 1, -1]), ("commit", [2, -1, 1, -1])]
