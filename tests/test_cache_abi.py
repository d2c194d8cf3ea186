"""The paged cache's C ABI and its binding without a GPU: exports, sizes and
refusals of host-checkable arguments (nothing here reaches the device)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dspark_cache.h")
LIB = os.path.join(ROOT, "semi_ar_draft_round_amd", "libdspark.so")

EINVAL, EDTYPE, EWORKSPACE = 1, 2, 3
P = ctypes.c_void_p
FAKE = P(0x1000)   # never dereferenced
ODD = P(0x1008)    # not 16-byte aligned


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(dspark_cache_\w+)\s*\(", text)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from semi_ar_draft_round_amd import build
        build.build()
    from semi_ar_draft_round_amd import binding
    return binding.load_library(LIB)


def test_exports(lib):
    from semi_ar_draft_round_amd import binding
    assert sorted(binding.CACHE_EXPORTED) == declared()
    for name in declared():
        assert hasattr(lib, name), name
    assert "pages" in binding.dspark_status_string(binding.ENOPAGES)


def test_page_bytes(lib):
    from semi_ar_draft_round_amd import binding as B
    assert B.dspark_cache_page_bytes(1, 8, 128, 64) == 8 * 64 * 128 * 4
    # 4 bits: half a byte a value, a scale byte per 32 dims of K, four bytes per token of V
    assert B.dspark_cache_page_bytes(2, 8, 128, 64) == 8 * 64 * (64 + 4 + 64 + 4)
    for bad in ((0, 8, 128, 64), (3, 8, 128, 64), (1, 0, 128, 64), (1, 1025, 128, 64), (1, 8, 96, 64), (1, 8, 512, 64),
                (1, 8, 128, 8), (1, 8, 128, 48), (1, 8, 128, 256)):
        assert B.dspark_cache_page_bytes(*bad) == 0, bad
    for fmt in (1, 2):
        for D in (64, 128, 256):
            for page in (16, 32, 64, 128):
                assert B.dspark_cache_page_bytes(fmt, 3, D, page) % 16 == 0


def test_workspace_sizes(lib):
    from semi_ar_draft_round_amd import binding as B
    w = B.dspark_cache_workspace_size
    assert w(B.CACHE_WS_ATTENTION, 4, 16, 32, 8, 128) > 0
    for bad in ((0, 16, 32, 8, 128), (4097, 16, 32, 8, 128), (4, -1, 32, 8, 128), (4, 1024, 32, 8, 128),
                (4, 16, 33, 8, 128), (4, 16, 32, 0, 128), (4, 16, 32, 8, 100)):
        assert w(B.CACHE_WS_ATTENTION, *bad) == 0, bad
    assert w(B.CACHE_WS_RESERVE, 4, 0, 10, 1000) >= 4000
    assert w(B.CACHE_WS_FORK, 4, 0, 10, 1000) >= 4 * 4 * 11
    assert w(B.CACHE_WS_COMPACT, 4, 0, 10, 1000) >= 4004
    for kind in (B.CACHE_WS_RESERVE, B.CACHE_WS_FORK, B.CACHE_WS_COMPACT):
        assert w(kind, 4, 0, 0, 1000) == 0
        assert w(kind, 4, 0, 10, (1 << 20) + 1) == 0
        assert w(kind, 4096, 0, 1 << 19, 1000) == 0     # R * max_pages reaches 2^31
    assert w(9, 4, 0, 10, 1000) == 0


def test_append_refusals(lib):
    def call(fmt=1, R=4, gamma=3, Hq=8, Hkv=2, D=128, page=64, n_pages=50, mp=4, q=FAKE, ldq=1024, ldk=256, ldv=256,
             eps=1e-6, freq=FAKE, rot=128, adj=0, ptr=FAKE, pool=FAKE):
        return lib.dspark_cache_append(fmt, R, gamma, Hq, Hkv, D, page, n_pages, mp, q, ldq, ptr, ldk, ptr, ldv, ptr, ptr,
                                       eps, freq, rot, adj, None, ptr, ptr, ptr, ptr, pool, None)
    assert call(fmt=0) == EDTYPE and call(fmt=3) == EDTYPE
    for bad in (dict(R=0), dict(R=4097), dict(gamma=-1), dict(gamma=1024), dict(Hq=0), dict(Hkv=0), dict(D=96),
                dict(page=20), dict(n_pages=0), dict(n_pages=(1 << 20) + 1), dict(mp=0), dict(ldq=1016), dict(ldq=1028),
                dict(ldk=248), dict(ldv=260), dict(ldq=1 << 31), dict(rot=-2), dict(rot=130), dict(rot=7),
                dict(rot=24), dict(freq=None), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")),
                dict(q=None), dict(ptr=None), dict(pool=None), dict(q=ODD), dict(pool=ODD)):
        assert call(**bad) == EINVAL, bad


def test_attention_refusals(lib):
    def call(fmt=1, R=4, gamma=3, Hq=8, Hkv=2, D=128, page=64, n_pages=50, mp=4, q=FAKE, scale=0.1, window=0, sinks=0,
             ptr=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
        return lib.dspark_cache_attention(fmt, R, gamma, Hq, Hkv, D, page, n_pages, mp, q, scale, window, sinks, None, ptr,
                                          ptr, ptr, ptr, out, None, ws, n, None)
    assert call(fmt=7) == EDTYPE
    for bad in (dict(R=0), dict(gamma=1024), dict(Hq=9), dict(D=80), dict(page=0), dict(n_pages=0), dict(mp=0),
                dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                dict(ptr=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None) == EWORKSPACE
    assert call(n=16) == EWORKSPACE


def test_read_refusals(lib):
    def call(fmt=1, R=4, T=3, Hkv=2, D=128, page=64, n_pages=50, mp=4, ptr=FAKE, pool=FAKE):
        return lib.dspark_cache_read(fmt, R, T, Hkv, D, page, n_pages, mp, None, ptr, ptr, pool, ptr, ptr, None)
    assert call(fmt=0) == EDTYPE
    for bad in (dict(R=0), dict(T=0), dict(T=(1 << 26) + 1), dict(T=1 << 29), dict(Hkv=0), dict(D=1), dict(page=1), dict(n_pages=0), dict(mp=0),
                dict(ptr=None), dict(pool=ODD)):
        assert call(**bad) == EINVAL, bad


def test_page_call_refusals(lib):
    big = 1 << 30

    def reserve(R=4, gamma=3, page=16, n=64, mp=8, ptr=FAKE, ws=FAKE, b=big):
        return lib.dspark_cache_reserve(R, gamma, page, n, mp, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, None, ws, b, None)

    def commit(R=4, gamma=3, page=16, n=64, mp=8, window=0, sinks=0, ptr=FAKE):
        return lib.dspark_cache_commit(R, gamma, page, n, mp, window, sinks, ptr, ptr, ptr, ptr, ptr, ptr, None)

    def fork(R=4, page=16, n=64, mp=8, ptr=FAKE, ws=FAKE, b=big):
        return lib.dspark_cache_fork(R, page, n, mp, ptr, ptr, ptr, ptr, ptr, ws, b, None)

    def compact(R=4, n=64, mp=8, ptr=FAKE, ws=FAKE, b=big):
        return lib.dspark_cache_compact(R, n, mp, ptr, ptr, ptr, ptr, ptr, ws, b, None)

    def reset(R=4, n=64, mp=8, ptr=FAKE):
        return lib.dspark_cache_reset(R, n, mp, ptr, ptr, ptr, ptr, None)

    def copy(layers=1, lb=0, pb=4096, n=64, m=4, ptr=FAKE, pool=FAKE):
        return lib.dspark_cache_copy(layers, lb, pb, n, ptr, ptr, m, pool, None)

    for call in (reserve, commit, fork, compact, reset):
        for bad in (dict(R=0), dict(R=4097), dict(n=0), dict(n=(1 << 20) + 1), dict(mp=0), dict(R=4096, mp=1 << 19),
                    dict(ptr=None)):
            assert call(**bad) == EINVAL, (call.__name__, bad)
    for call in (reserve, commit, fork):
        assert call(page=17) == EINVAL
    for call in (reserve, commit):
        assert call(gamma=-1) == EINVAL and call(gamma=1024) == EINVAL
    assert commit(window=-1) == EINVAL and commit(sinks=-1) == EINVAL
    for call in (reserve, fork, compact):
        assert call(ws=None) == EWORKSPACE and call(b=4) == EWORKSPACE
    for bad in (dict(layers=0), dict(pb=0), dict(pb=24), dict(pb=1 << 31), dict(n=0), dict(m=0), dict(m=(1 << 20) + 1),
                dict(layers=2, lb=4096), dict(layers=2, lb=64 * 4096 + 8), dict(ptr=None), dict(pool=None),
                dict(pool=ODD)):
        assert copy(**bad) == EINVAL, bad


def test_binding_refuses_before_the_library(lib):
    """Shapes, types, strides and places that the binding turns down."""
    import torch
    from semi_ar_draft_round_amd import binding as B
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    table, ell, length = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    pool = torch.zeros(9, B.dspark_cache_page_bytes(1, 2, 64, 16), dtype=torch.uint8)
    q, k = torch.zeros(4, 4, 64, **bf), torch.zeros(4, 2, 64, **bf)

    def append(q=q, k=k, v=k, pool=pool, table=table, gamma=1, **kw):
        return B.dspark_cache_append(q, k, v, pool, table, length, ell, gamma, fmt=1, page=16, **kw)

    with pytest.raises(ValueError, match="not on the current GPU"):
        append()
    for bad, what in ((dict(q=q.float()), "dtype"), (dict(q=q[..., :32]), "shape|heads"), (dict(gamma=2), "row0"),
                      (dict(k=k[:3]), "shape"), (dict(q=torch.zeros(4, 5, 64, **bf)[:, 1:].transpose(0, 1)), "rows|heads"),
                      (dict(pool=pool[:, :-16]), "shape"), (dict(pool=pool.view(9, 2, -1)), "n_pages"),
                      (dict(table=table.long()), "dtype"), (dict(freq=torch.zeros(32)), "dtype"),
                      (dict(wq=torch.zeros(63, **bf)), "shape"), (dict(q_out=torch.zeros(4, 4, 64)), "dtype"),
                      (dict(q=torch.zeros(4 * 4 * 64 + 4, **bf)[4:].view(4, 4, 64)), "aligned")):
        with pytest.raises(ValueError, match=what):
            append(**bad)
    with pytest.raises(ValueError, match="lse"):
        B.dspark_cache_attention(q, pool, table, length, ell, 1, fmt=1, page=16, heads_kv=2, lse=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="not on the current GPU"):
        B.dspark_cache_attention(q, pool, table, length, ell, 1, fmt=1, page=16, heads_kv=2)
    with pytest.raises(ValueError, match="no page format"):
        B.dspark_cache_attention(q, pool, table, length, ell, 1, fmt=5, page=16, heads_kv=2)
    ref, bits = torch.zeros(40, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="bits"):
        B.dspark_cache_reset(table, length, ref, torch.zeros(1, **i32))
    with pytest.raises(ValueError, match="pairs"):
        B.dspark_cache_compact(table, ref, bits, pairs=torch.zeros(19, 2, **i32))
    with pytest.raises(ValueError, match="current GPU"):
        B.dspark_cache_fork(table, length, ref, bits, ell, page=16)
    with pytest.raises(ValueError, match="pool"):
        B.dspark_cache_copy(pool[0], ell.view(1, 2), n_pairs=ell[:1])
