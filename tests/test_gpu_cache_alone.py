"""A request's rows come out the same whatever batch they are in: what the
header promises of the append's queries and of the cache's contents."""

import sys

import numpy as np
import pytest

from cache_cases import BF16, FP4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from semi_ar_draft_round_amd import binding
    binding.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("rot,adjacent", [(128, False), (64, True)])
def test_append_alone_and_in_a_batch(rot, adjacent, dev):
    """The rows of one request alone and among 200, over both page formats:
    the same queries bit for bit in all four, the same pages per format."""
    from semi_ar_draft_round_amd import binding as B
    say(f"[alone] append rot {rot}")
    Hq, Hkv, D, P, gamma, R, me = 32, 8, 128, 32, 63, 200, 77
    g = torch.Generator(device=dev).manual_seed(rot)
    x = torch.randn((R * (gamma + 1), Hq + 2 * Hkv, D), generator=g, device=dev).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn((2, D), generator=g, device=dev)).to(torch.bfloat16)
    freq = 1e4 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=dev) / rot)
    i32 = dict(dtype=torch.int32, device=dev)
    length = torch.arange(R, **i32) * 37 + 5
    pages = -(-(int(length.max()) + gamma + 1) // P)
    queries, contents = [], []
    for fmt in (BF16, FP4):
        for reqs in ([me], list(range(R))):
            n = len(reqs)
            table = torch.full((n, pages), -1, **i32)    # pages of the new rows alone
            for r, q in enumerate(reqs):
                first = int(length[q]) // P
                table[r, first:first + 3] = torch.arange(3 * r, 3 * r + 3, **i32)[:pages - first]
            pool = torch.zeros((3 * n, B.dspark_cache_page_bytes(fmt, Hkv, D, P)), dtype=torch.uint8, device=dev)
            rows = x.view(R, gamma + 1, Hq + 2 * Hkv, D)[reqs].flatten(0, 1)
            out = B.dspark_cache_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], pool, table,
                                        length[reqs].contiguous(), torch.full((n,), gamma, **i32), gamma, fmt=fmt, page=P,
                                        wq=w[0].contiguous(), wk=w[1].contiguous(), freq=freq, adjacent=adjacent)
            r = reqs.index(me)
            queries.append(out.view(n, gamma + 1, Hq, D)[r].view(torch.int16))
            contents.append(pool[3 * r:3 * r + 3])
    torch.cuda.synchronize()
    for q in queries[1:]:
        assert int((q != queries[0]).sum()) == 0
    assert torch.equal(contents[0], contents[1]) and torch.equal(contents[2], contents[3])
