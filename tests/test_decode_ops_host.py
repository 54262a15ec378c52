"""The operators between the GEMVs without a GPU: sizes of the cache, refusals of the C ABI (argument errors are
found before anything touches a device), and the plain implementation's own round trips."""
import ctypes

import numpy as np
import pytest

import quant_dequant_gemv_q4_b200 as qg
import kv4_ref as ref

A = 1 << 20  # an aligned address that is never read: every call here is refused or has nothing to do


@pytest.fixture(scope="module")
def L():
    from quant_dequant_gemv_q4_b200 import build
    build.build()
    return qg.lib()


def heads(ptr=A, token=256, head=256, dim=1, kind=qg.QG_TYPE_F32):
    return ctypes.byref(qg.qg_heads(ptr, token, head, dim, kind))


def test_cache_bytes(L):
    assert qg.qg_kv4_bytes(1, 16, 1, 256) == 4608
    assert qg.qg_kv4_bytes(7, 64, 4, 128) == 7 * 4 * 4 * 18 * 128
    assert qg.qg_kv4_bytes(0, 16, 4, 64) == 0
    for bad in [(1, 8, 1, 64), (1, 24, 1, 64), (1, 16, 0, 64), (1, 16, 1, 96), (-1, 16, 1, 64), (1, 16, 1025, 64),
                (1 << 60, 16, 8, 256)]:
        assert qg.qg_kv4_bytes(*bad) == 0, bad


def norm_rope(L, **kw):
    a = dict(q=heads(), k=heads(), T=3, Hq=4, Hk=1, D=256, wq=A, wk=A, eps=1e-6, pos=A, freq=A, R=64, pairing=0,
             qo=heads(), ko=heads())
    a.update(kw)
    return L.qg_qk_norm_rope(a["q"], a["k"], a["T"], a["Hq"], a["Hk"], a["D"], a["wq"], a["wk"], a["eps"], a["pos"],
                             a["freq"], a["R"], a["pairing"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=96), qg.QG_ERR_SHAPE), (dict(T=-1), qg.QG_ERR_SHAPE), (dict(Hq=-1), qg.QG_ERR_SHAPE),
    (dict(Hk=1025), qg.QG_ERR_SHAPE), (dict(R=65), qg.QG_ERR_SHAPE), (dict(R=258), qg.QG_ERR_SHAPE),
    (dict(R=-2), qg.QG_ERR_SHAPE), (dict(pairing=2), qg.QG_ERR_VARIANT), (dict(eps=-1.0), qg.QG_ERR_RANGE),
    (dict(eps=float("nan")), qg.QG_ERR_RANGE), (dict(pos=None), qg.QG_ERR_NULL), (dict(freq=None), qg.QG_ERR_NULL),
    (dict(pos=A + 2), qg.QG_ERR_ALIGN), (dict(freq=A + 4), qg.QG_ERR_ALIGN), (dict(wq=A + 1), qg.QG_ERR_ALIGN),
    (dict(q=None), qg.QG_ERR_NULL), (dict(qo=heads(ptr=None)), qg.QG_ERR_NULL),
    (dict(k=heads(ptr=A + 2)), qg.QG_ERR_ALIGN), (dict(ko=heads(kind=30)), qg.QG_ERR_FMT),
    (dict(T=0), qg.QG_OK), (dict(Hq=0, Hk=0), qg.QG_OK)])
def test_norm_rope_refusals(L, kw, want):
    assert norm_rope(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(D=32), qg.QG_ERR_SHAPE), (dict(H=0), qg.QG_ERR_SHAPE), (dict(page=20), qg.QG_ERR_SHAPE),
    (dict(page=0), qg.QG_ERR_SHAPE), (dict(pages=-1), qg.QG_ERR_SHAPE), (dict(pages=1 << 60), qg.QG_ERR_SHAPE),
    (dict(T=-1), qg.QG_ERR_SHAPE), (dict(cache=None), qg.QG_ERR_NULL), (dict(cache=A + 8), qg.QG_ERR_ALIGN),
    (dict(slot=None), qg.QG_ERR_NULL), (dict(slot=A + 4), qg.QG_ERR_ALIGN), (dict(k=None), qg.QG_ERR_NULL),
    (dict(v=heads(kind=8)), qg.QG_ERR_FMT), (dict(R=64, pos=None), qg.QG_ERR_NULL), (dict(eps=-1e-9), qg.QG_ERR_RANGE),
    (dict(T=0), qg.QG_OK), (dict(pages=0, cache=None), qg.QG_OK)])
def test_append_refusals(L, kw, want):
    a = dict(k=heads(), v=heads(), T=3, H=2, D=128, wk=None, eps=0.0, pos=A, freq=A, R=0, pairing=0, slot=A, cache=A,
             pages=4, page=32)
    a.update(kw)
    assert L.qg_kv4_append(a["k"], a["v"], a["T"], a["H"], a["D"], a["wk"], a["eps"], a["pos"], a["freq"], a["R"],
                           a["pairing"], a["slot"], a["cache"], a["pages"], a["page"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), qg.QG_ERR_SHAPE), (dict(slot=None), qg.QG_ERR_NULL), (dict(T=-3), qg.QG_ERR_SHAPE),
    (dict(out=None), qg.QG_ERR_NULL), (dict(cache=A + 1), qg.QG_ERR_ALIGN), (dict(T=0), qg.QG_OK)])
def test_read_refusals(L, kw, want):
    a = dict(cache=A, pages=4, page=32, H=2, D=128, slot=A, T=3, out=heads())
    a.update(kw)
    assert L.qg_kv4_read(a["cache"], a["pages"], a["page"], a["H"], a["D"], a["slot"], a["T"], a["out"], heads(), None) == want


H16 = dict(kind=qg.QG_TYPE_F16)


@pytest.mark.parametrize("kw,want", [
    (dict(D=192), qg.QG_ERR_SHAPE), (dict(Hq=5), qg.QG_ERR_SHAPE), (dict(Hk=0), qg.QG_ERR_SHAPE),
    (dict(Hq=2048), qg.QG_ERR_SHAPE), (dict(page=17), qg.QG_ERR_SHAPE), (dict(width=-1), qg.QG_ERR_SHAPE),
    (dict(width=1 << 30), qg.QG_ERR_SHAPE), (dict(T=-1), qg.QG_ERR_SHAPE), (dict(nseq=-1), qg.QG_ERR_SHAPE),
    (dict(pages=-1), qg.QG_ERR_SHAPE), (dict(max_q=-1), qg.QG_ERR_SHAPE), (dict(start=None), qg.QG_ERR_NULL),
    (dict(lens=None), qg.QG_ERR_NULL), (dict(table=None), qg.QG_ERR_NULL), (dict(cache=None), qg.QG_ERR_NULL),
    (dict(ws=None), qg.QG_ERR_NULL), (dict(q=None), qg.QG_ERR_NULL), (dict(q=heads()), qg.QG_ERR_FMT),
    (dict(out=heads()), qg.QG_ERR_FMT), (dict(q=heads(ptr=A + 1, **H16)), qg.QG_ERR_ALIGN),
    (dict(cache=A + 8), qg.QG_ERR_ALIGN), (dict(ws=A + 16), qg.QG_ERR_ALIGN), (dict(start=A + 2), qg.QG_ERR_ALIGN),
    (dict(T=0), qg.QG_OK), (dict(nseq=0), qg.QG_OK)])
def test_attention_refusals(L, kw, want):
    a = dict(q=heads(**H16), T=3, nseq=2, start=A, max_q=2, Hq=4, Hk=2, D=128, cache=A, pages=9, page=32, table=A, width=4,
             lens=A, out=heads(**H16), ws=A, wb=1 << 40)
    a.update(kw)
    assert L.qg_attn_kv4(a["q"], a["T"], a["nseq"], a["start"], a["max_q"], a["Hq"], a["Hk"], a["D"], a["cache"], a["pages"],
                         a["page"], a["table"], a["width"], a["lens"], 1.0, a["out"], a["ws"], a["wb"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), qg.QG_ERR_SHAPE), (dict(V=0), qg.QG_ERR_SHAPE), (dict(V=1 << 31), qg.QG_ERR_SHAPE),
    (dict(logits=None), qg.QG_ERR_NULL), (dict(token=None), qg.QG_ERR_NULL), (dict(u=None), qg.QG_ERR_NULL),
    (dict(logits=A + 2), qg.QG_ERR_ALIGN), (dict(top_k=A + 1), qg.QG_ERR_ALIGN), (dict(ws=A + 2), qg.QG_ERR_ALIGN),
    (dict(es=2, ws=A, wb=799), qg.QG_ERR_SCRATCH), (dict(rows=0), qg.QG_OK)])
def test_sample_refusals(L, kw, want):
    a = dict(logits=A, rows=2, V=100, es=1, t=A, top_k=A, p=A, mp=A, u=A, token=A, ws=None, wb=0)
    a.update(kw)
    assert L.qg_sample(a["logits"], a["rows"], a["V"], a["V"], a["es"], a["t"], a["top_k"], a["p"], a["mp"], a["u"], a["token"], a["ws"],
                       a["wb"], None) == want


def test_sample_workspace(L):
    assert qg.qg_sample_workspace(16, 1000, 16) == 64000
    assert qg.qg_sample_workspace(16, 1000, 1) == 0 and qg.qg_sample_workspace(1, 1000, 16) == 0


def test_wrappers_refuse_host_tensors(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the check is of a machine without a GPU's tensors")
    with pytest.raises(Exception):
        qg.qg_sample(torch.zeros(1, 4), None, None, None, None, torch.zeros(1), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_reference_cache_round_trip(D):
    rng = np.random.default_rng(D)
    cache = rng.integers(0, 256, (3, 2, 2, 18 * D), dtype=np.uint8)
    before = cache.copy()
    x = rng.normal(size=(5, 2, D))
    slot = np.array([0, 95, 33, -1, 96])
    code, d, m = ref.quantize(x)
    ref.store(cache, 32, slot, 0, code, d, m)
    got = [ref.load(cache, 32, p, 0) for p in range(3)]
    for i, p in enumerate(slot):
        if 0 <= p < 96:
            assert np.array_equal(got[p // 32][:, p % 32].astype(np.float32), ref.values(code, d, m)[i])
    # K of three tokens: their codes and scales changed, nothing else
    assert np.array_equal(cache[..., 9 * D:], before[..., 9 * D:])
    assert (cache != before).sum() <= 3 * 2 * (D // 2 + D // 16)
    # a value is off by half a step, and by what rounding d and m to fp16 moves it
    err = np.abs(ref.values(code, d, m).astype(np.float64) - x)
    step = d.astype(np.float64).repeat(64, -1)
    assert (err <= step * (0.5 + 15 * 2.0 ** -11) + np.abs(m.astype(np.float64)).repeat(64, -1) * 2.0 ** -11 + 2.0 ** -24).all()


def test_reference_samples_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert ref.sample(x, 1.0, None, None, None, 0.05) == 0
    assert ref.sample(x, 1.0, None, None, None, 0.6) == 2
    assert ref.sample(x, 1.0, 2, None, None, 0.99) == 3      # 1 and 3 stay
    assert ref.sample(x, 1.0, None, 0.35, None, 0.99) == 1   # 1 alone
    assert ref.sample(x, 1.0, None, None, 0.6, 0.99) == 3    # 1 and 3 stay
    assert ref.sample(x, 0.0, None, None, None, 0.99) == 1
    assert ref.sample(np.full(3, -np.inf), 1.0, None, None, None, 0.5) == -1
    assert ref.sample(np.zeros(4), 1.0, 2, None, None, 0.75) == 1  # ties: the lower indices stay


@pytest.mark.parametrize("kw", [dict(V=1 << 20), dict(rows=16 * 65535 + 1)])
def test_sample_sizes_past_the_sums_and_the_grid(L, kw):
    """2^20 weights of 2^44 would not fit 64 bits; a grid has 65535 rows of blocks."""
    a = dict(rows=2, V=100)
    a.update(kw)
    assert L.qg_sample(A, a["rows"], a["V"], a["V"], 1, A, A, A, A, A, A, None, 0, None) == qg.QG_ERR_SHAPE
    assert qg.qg_sample_workspace(a["rows"], a["V"], 2) == 0
