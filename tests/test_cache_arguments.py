"""Refusals of the paged cache's calls and of its binding, without a GPU
(nothing here reaches the device): what the header asks of workspaces and
numbers."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "semi_ar_draft_round_amd", "libdspark.so")

EINVAL, EWORKSPACE = 1, 3
P = ctypes.c_void_p
FAKE = P(0x1000)   # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from semi_ar_draft_round_amd import build
        build.build()
    from semi_ar_draft_round_amd import binding
    return binding.load_library(LIB)


@pytest.mark.parametrize("at", [0x1001, 0x1004, 0x1008])
def test_workspaces_are_16_byte_aligned(at, lib):
    ws = P(at)
    p = FAKE
    assert lib.dspark_cache_reserve(4, 3, 16, 64, 8, p, p, p, p, p, p, p, p, None, ws, BIG, None) == EINVAL
    assert lib.dspark_cache_fork(4, 16, 64, 8, p, p, p, p, p, ws, BIG, None) == EINVAL
    assert lib.dspark_cache_compact(4, 64, 8, p, p, p, p, p, ws, BIG, None) == EINVAL
    assert lib.dspark_cache_attention(1, 4, 3, 8, 2, 128, 64, 50, 4, p, 0.1, 0, 0, None, p, p, p, p, p, None, ws, BIG,
                                      None) == EINVAL
    for call in (lambda w: lib.dspark_cache_reserve(4, 3, 16, 64, 8, p, p, p, p, p, p, p, p, None, w, BIG, None),
                 lambda w: lib.dspark_cache_fork(4, 16, 64, 8, p, p, p, p, p, w, BIG, None),
                 lambda w: lib.dspark_cache_compact(4, 64, 8, p, p, p, p, p, w, BIG, None)):
        assert call(None) == EWORKSPACE


def test_the_binding_checks_a_given_workspace(lib):
    import torch
    from semi_ar_draft_round_amd import binding as B
    ws = torch.zeros(4096 + 64, dtype=torch.uint8)
    lead = -ws.data_ptr() % 16
    kind = B.CACHE_WS_RESERVE
    assert B._cache_ws(ws[lead:], kind, 4, 0, 8, 64, 0, -1) is not None
    for off in (1, 4, 8):
        with pytest.raises(ValueError, match="aligned"):
            B._cache_ws(ws[lead + off:], kind, 4, 0, 8, 64, 0, -1)


def test_the_attention_workspace_holds_what_a_device_uses(lib):
    """Two parts for each of at most 512 work groups (256 with 256 dims): 32
    rows a row tile of D fp32 sums, a maximum and a sum; and the descriptors,
    32 bytes a work group.  No more than that, rounded to 256 bytes."""
    from semi_ar_draft_round_amd import binding as B
    for D in (64, 128, 256):
        for gamma, heads, tiles in ((0, 4, 1), (16, 4, 3), (1023, 1, 4), (1023, 8, 4)):
            groups = 256 if D == 256 else 512
            need = 512 * 32 + groups * 2 * tiles * 32 * (4 * D + 8)
            got = B.dspark_cache_workspace_size(B.CACHE_WS_ATTENTION, 7, gamma, 8 * heads, 8, D)
            assert need <= got < need + 256, (D, gamma, heads)


def test_inline_assembly_leaves_m0_as_it_was():
    """The compiler keeps M0 for itself and is not told of writes to it, so an
    asm statement that writes it saves it first and puts it back."""
    import glob
    import re
    seen = 0
    for path in glob.glob(os.path.join(ROOT, "semi_ar_draft_round_amd", "csrc", "*.h*")):
        for text in re.findall(r"\basm volatile\((.*?)\);", open(path).read(), flags=re.S):
            lines = [x.strip() for x in "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split("\n      :")[0])).replace(
                "\\t", "").split("\\n")]
            if not any(re.match(r"\w+ m0\b", x) for x in lines):
                continue
            seen += 1
            save = re.match(r"s_mov_b32 (%\d), m0$", lines[0])
            assert save and lines[-1] == f"s_mov_b32 m0, {save.group(1)}", path
    assert seen == 1


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 126 * 1.001, float("inf"), float("nan")])
def test_scales_that_overflow_in_base_two(scale, lib):
    """The kernel works with scale * log2 e, which has to be finite; the
    workspace is checked after it, so an accepted scale gets as far as that."""
    p = FAKE
    call = lambda s: lib.dspark_cache_attention(1, 4, 3, 8, 2, 128, 64, 50, 4, p, s, 0, 0, None, p, p, p, p, p, None, p, 16,
                                                None)
    assert call(scale) == EINVAL
    assert call(2.0 ** 126) == EWORKSPACE and call(-2.0 ** 126) == EWORKSPACE and call(0.0) == EWORKSPACE


def test_numbers_past_32_bits_are_refused(lib):
    """Cut to 32 bits, a window of 2^32 tokens would be none at all, 2^32 + 4
    first tokens would be 4."""
    import torch
    from semi_ar_draft_round_amd import binding as B
    from semi_ar_draft_round_amd.cache import PagedCache
    i32, wide = dict(dtype=torch.int32), 1 << 32
    table, ell, length = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    ref, bits = torch.zeros(9, **i32), torch.zeros(1, **i32)
    pool = torch.zeros(9, B.dspark_cache_page_bytes(1, 2, 64, 16), dtype=torch.uint8)
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    state = (table, length, ref, bits)
    for call in (lambda x: B.dspark_cache_page_bytes(1, 2, 64, x + 16),
                 lambda x: B.dspark_cache_workspace_size(B.CACHE_WS_ATTENTION, 4, x + 3, 8, 2, 64),
                 lambda x: B.dspark_cache_append(q, k, k, pool, table, length, ell, x + 1, fmt=1, page=16, row0=ell),
                 lambda x: B.dspark_cache_append(q, k, k, pool, table, length, ell, 1, fmt=1, page=x + 16),
                 lambda x: B.dspark_cache_attention(q, pool, table, length, ell, 1, fmt=1, page=16, heads_kv=2, window=x),
                 lambda x: B.dspark_cache_attention(q, pool, table, length, ell, 1, fmt=1, page=16, heads_kv=2, window=5,
                                                    sinks=x + 4),
                 lambda x: B.dspark_cache_read(pool, table, None, ell, 1, fmt=1, page=x + 16, heads_kv=2, dim=64),
                 lambda x: B.dspark_cache_reserve(*state, ell, x + 1, page=16),
                 lambda x: B.dspark_cache_reserve(*state, ell, 1, page=x + 16),
                 lambda x: B.dspark_cache_commit(*state, ell, ell, 1, page=16, window=x),
                 lambda x: B.dspark_cache_commit(*state, ell, ell, 1, page=16, window=8, sinks=x + 4),
                 lambda x: B.dspark_cache_commit(*state, ell, ell, x + 1, page=16),
                 lambda x: B.dspark_cache_fork(*state, ell, page=x + 16)):
        with pytest.raises(ValueError, match="32 bits"):
            call(wide)
        with pytest.raises(ValueError, match="32 bits"):
            call(-wide)
    for bad in (dict(window=wide), dict(sinks=wide + 4)):
        with pytest.raises(ValueError, match="window and sinks"):
            PagedCache(1, 2, 10, 4, 1, 64, device="cpu", **bad)
