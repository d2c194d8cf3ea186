"""dspark_logits.h's C ABI, the new cache calls and their bindings without a
GPU: exports, sizes and refusals (nothing here reaches the device)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dspark_logits.h")
LIB = os.path.join(ROOT, "semi_ar_draft_round_amd", "libdspark.so")

EINVAL, EDTYPE = 1, 2
P = ctypes.c_void_p
FAKE = P(0x1000)   # never dereferenced
ODD = P(0x1008)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from semi_ar_draft_round_amd import build
        build.build()
    from semi_ar_draft_round_amd import binding
    return binding.load_library(LIB)


def test_exports(lib):
    from semi_ar_draft_round_amd import binding
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dspark_\w+)\s*\(", text)))
    assert sorted(binding.LOGITS_EXPORTED) == names
    import semi_ar_draft_round_amd as pkg
    for name in names + ["dspark_cache_weigh", "dspark_cache_evict"]:
        assert hasattr(lib, name) and getattr(pkg, name) is getattr(binding, name)


def test_page_bytes_of_8_bits(lib):
    from semi_ar_draft_round_amd import binding as B
    for D in (64, 128, 256):
        for page in (16, 32, 64, 128):
            assert B.dspark_cache_page_bytes(B.CACHE_FP8, 3, D, page) == 3 * (2 * page * D + 16)
    for bad in ((4, 0, 128, 64), (4, 8, 96, 64), (4, 8, 128, 8)):
        assert B.dspark_cache_page_bytes(*bad) == 0


def test_logits_refusals(lib):
    def call(dt=0, R=4, gamma=3, V=100, logits=FAKE, ell=FAKE, x0=FAKE, x=FAKE, state=FAKE, nb=2, tok=FAKE, bias=FAKE,
             out=FAKE):
        return lib.dspark_logits(dt, R, gamma, V, logits, None, ell, x0, x, state, None, None, None, nb, tok, bias, None,
                                 out, None)
    assert call(dt=2) == EDTYPE and call(dt=-1) == EDTYPE
    for bad in (dict(R=0), dict(R=4097), dict(gamma=-1), dict(gamma=1024), dict(V=1), dict(V=1 << 24), dict(logits=None),
                dict(ell=None), dict(x0=None), dict(out=None), dict(nb=-1), dict(nb=(1 << 20) + 1), dict(tok=None),
                dict(bias=None), dict(logits=ODD), dict(out=ODD), dict(state=ODD)):
        assert call(**bad) == EINVAL, bad

    def prompt(R=4, V=100, n=10, tokens=FAKE, start=FAKE, count=FAKE, state=FAKE):
        return lib.dspark_logits_prompt(R, V, n, tokens, start, count, state, None)
    for bad in (dict(R=0), dict(R=4097), dict(V=1), dict(V=1 << 24), dict(n=-1), dict(n=1 << 31), dict(tokens=None),
                dict(start=None), dict(count=None), dict(state=None), dict(state=ODD)):
        assert prompt(**bad) == EINVAL, bad

    def commit(R=4, gamma=3, V=100, ptr=FAKE, x=FAKE, state=FAKE):
        return lib.dspark_logits_commit(R, gamma, V, ptr, ptr, ptr, x, state, None)
    for bad in (dict(R=0), dict(gamma=-1), dict(gamma=1024), dict(V=1), dict(ptr=None), dict(state=None),
                dict(state=ODD)):
        assert commit(**bad) == EINVAL, bad


def test_weigh_and_evict_refusals(lib):
    def weigh(fmt=4, R=4, gamma=3, Hq=8, Hkv=2, D=128, page=64, n_pages=50, mp=4, q=FAKE, scale=0.1, window=0, sinks=0,
              ptr=FAKE, pool=FAKE, keep=1.0, mass=FAKE):
        return lib.dspark_cache_weigh(fmt, R, gamma, Hq, Hkv, D, page, n_pages, mp, q, scale, window, sinks, ptr, None, ptr,
                                      ptr, ptr, pool, keep, mass, None)
    assert weigh(fmt=3) == EDTYPE and weigh(fmt=0) == EDTYPE
    inf, nan = float("inf"), float("nan")
    for bad in (dict(R=0), dict(R=4097), dict(gamma=1024), dict(Hq=9), dict(Hq=0), dict(Hkv=0), dict(D=80), dict(page=0),
                dict(n_pages=0), dict(mp=0), dict(R=4096, mp=1 << 19), dict(window=-1), dict(sinks=-1), dict(scale=nan),
                dict(scale=2.0 ** 126 * 1.001), dict(keep=-0.5), dict(keep=inf), dict(keep=nan), dict(q=None),
                dict(ptr=None), dict(pool=None), dict(mass=None), dict(q=ODD), dict(pool=ODD)):
        assert weigh(**bad) == EINVAL, bad

    def evict(R=4, page=16, n=64, mp=8, sinks=0, recent=0, ptr=FAKE):
        return lib.dspark_cache_evict(R, page, n, mp, sinks, recent, ptr, ptr, ptr, ptr, ptr, ptr, None, None)
    for bad in (dict(R=0), dict(R=4097), dict(page=17), dict(n=0), dict(n=(1 << 20) + 1), dict(mp=0),
                dict(R=4096, mp=1 << 19), dict(sinks=-1), dict(recent=-1), dict(ptr=None)):
        assert evict(**bad) == EINVAL, bad


def test_binding_refuses_before_the_library(lib):
    import torch
    from semi_ar_draft_round_amd import binding as B
    from semi_ar_draft_round_amd.cache import PagedCache
    from semi_ar_draft_round_amd.logits import Conditions
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    R, gamma, V = 2, 1, 70
    x = torch.zeros(4, V, dtype=torch.bfloat16)
    state, ell, x0, d = torch.zeros(R, V, dtype=torch.int16), torch.zeros(R, **i32), torch.zeros(R, **i32), torch.zeros(
        R, gamma, **i32)

    def call(x=x, state=state, ell=ell, gamma=gamma, x0=x0, d=d, **kw):
        return B.dspark_logits(x, state, ell, gamma, x0, d, **kw)

    with pytest.raises(ValueError, match="not on the current GPU"):
        call()
    with pytest.raises(ValueError, match="not on the current GPU"):
        call(x=x.view(R, 2, V), mask=torch.zeros(4, 3, **i32))
    for bad, what in ((dict(x=x.half()), "neither"), (dict(x=x[:, ::2]), "logits"), (dict(x=x[:3]), "row0"),
                      (dict(x=x.view(R, 2, V), row0=x0), "without row0"), (dict(x=x[0]), "rows"),
                      (dict(state=state.int()), "int16"), (dict(state=state[:, :-1]), "shape"), (dict(ell=ell.long()), "dtype"),
                      (dict(x0=x0[:1]), "shape"), (dict(d=d.long()), "dtype"), (dict(d=torch.zeros(R, 2, **i32)), "shape"),
                      (dict(repetition=torch.ones(R, dtype=torch.float64)), "dtype"), (dict(presence=torch.ones(3)), "shape"),
                      (dict(mask=torch.zeros(4, 2, **i32)), "shape"), (dict(mask=torch.zeros(4, 3)), "dtype"),
                      (dict(bias_tok=torch.zeros(R, 4, **i32), bias=torch.zeros(R, 3)), "shape"),
                      (dict(out=x.float()), "dtype"), (dict(gamma=1 << 32), "32 bits")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    with pytest.raises(ValueError, match="together"):
        call(bias_tok=torch.zeros(R, 4, **i32))
    with pytest.raises(ValueError, match="current GPU"):
        B.dspark_logits_prompt(state, ell, x0, x0)
    with pytest.raises(ValueError, match="current GPU"):
        B.dspark_logits_commit(state, ell, ell, x0)

    table, ref, bits = torch.zeros(R, 3, **i32), torch.zeros(40, **i32), torch.zeros(2, **i32)
    pool = torch.zeros(9, B.dspark_cache_page_bytes(4, 2, 64, 16), dtype=torch.uint8)
    q, lse, mass = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 4), torch.zeros(R, 3)

    def weigh(q=q, lse=lse, mass=mass, fmt=4, **kw):
        return B.dspark_cache_weigh(q, lse, pool, table, ell, ell, 1, mass, fmt=fmt, page=16, heads_kv=2, **kw)

    with pytest.raises(ValueError, match="current GPU"):
        weigh()
    for bad, what in ((dict(lse=lse[:, :3]), "lse"), (dict(mass=mass[:, :2]), "mass"), (dict(mass=mass.double()), "mass"),
                      (dict(q=q.float()), "dtype"), (dict(fmt=3), "no page format"), (dict(window=1 << 32), "32 bits")):
        with pytest.raises(ValueError, match=what):
            weigh(**bad)
    state4 = (table, ell, ref, bits)
    with pytest.raises(ValueError, match="current GPU"):
        B.dspark_cache_evict(*state4, mass, ell, page=16)
    for bad, what in ((dict(mass=mass.double()), "mass"), (dict(budget=ell.long()), "budget"), (dict(recent=1 << 32), "32 bits"),
                      (dict(freed=torch.zeros(3, **i32)), "freed")):
        with pytest.raises(ValueError, match=what):
            B.dspark_cache_evict(*state4, bad.pop("mass", mass), bad.pop("budget", ell), page=16, **bad)
    for bad in (dict(budget=-1), dict(budget=1, fade=float("nan")), dict(budget=1, fade=-1.0), dict(keep_first=-1),
                dict(keep_last=1 << 31)):
        with pytest.raises(ValueError):
            PagedCache(1, 2, 10, 4, 1, 64, device="cpu", **bad)
    for bad in ((0, 10), (1, 1), (1, 10, -1)):
        with pytest.raises(ValueError):
            Conditions(*bad, device="cpu")


def test_a_mask_needs_conditions():
    import types
    from semi_ar_draft_round_amd import device_round as DR
    with pytest.raises(ValueError, match="conditions"):
        DR.run_round_cached(types.SimpleNamespace(), None, None, mask=1)
