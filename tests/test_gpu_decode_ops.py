"""The operators between the GEMVs on the GPU, against the plain 64-bit implementations of kv4_ref: head norms
and rotation, the 4-bit cache, the attention over it, sampling, and a run of them together with the GEMVs."""
import numpy as np
import pytest

import kv4_ref as ref
from quant_dequant_gemv_q4_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quant_dequant_gemv_q4_b200 import build
    build.build()
    import quant_dequant_gemv_q4_b200 as q
    return q


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def frequencies(R, base=1e7):
    return np.array([base ** (-2.0 * i / R) for i in range(R // 2)]) if R else np.zeros(0)


def layout(x, how):
    """A [T, H, D] tensor with the values of x (numpy) in one of the layouts a caller has."""
    import torch
    T, H, D = x.shape
    if how == "rows":
        return dev(x)
    if how == "gemv":  # [H D][T], what a GEMV leaves and takes
        return dev(x.transpose(1, 2, 0)).permute(2, 0, 1)
    if how == "heads first":
        return dev(x.transpose(1, 0, 2)).permute(1, 0, 2)
    # rows of a wider array at an odd offset: no wide accesses
    wide = torch.zeros(T, H * D + 3, dtype=dev(x[:1, :1, :1]).dtype, device="cuda")
    v = wide[:, 1:1 + H * D].unflatten(1, (H, D))
    v.copy_(dev(x))
    return v


LAYOUTS = ["rows", "gemv", "heads first", "odd"]


# ---------------------------------------------------------------------------------------------
# Head norms and rotation
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hk,R,pairing,norm,first", [
    (1, 48, 4, 64, 0, True, 70001), (3, 5, 1, 16, 1, True, 2000000000), (17, 8, 8, 64, 0, False, 0),
    (2, 1, 0, 2, 0, True, 9), (33, 12, 2, 64, 1, False, -5), (5, 0, 3, 0, 0, True, 0), (700, 6, 1, 6, 0, True, 250000)])
@pytest.mark.parametrize("how,src,dst", [("rows", "f4", "f2"), ("gemv", "f4", "f2"), ("odd", "f2", "f4"), ("heads first", "f2", "f2")])
def test_norm_rope(qg, D, T, Hq, Hk, R, pairing, norm, first, how, src, dst):
    """Bound: the sum of squares takes at most 8 + 5 additions of fp32 and the factor 4 more roundings, each
    product one; sine and cosine are off by 2^-25 turns (3.2 half ulps of 1) and 2 ulps; two products and a sum:
    24 half ulps of |x_i| + |x_j| in all.  An fp16 output adds half a step, 2^-11 of itself or 2^-25."""
    import torch
    rng = np.random.default_rng(D + T)
    pos = (first + np.arange(T)).astype(np.int32)
    freq = frequencies(R)
    w = rng.uniform(0.5, 1.5, (2, D)).astype(np.float32)
    ins, outs, xs = [], [], []
    for H in (Hq, Hk):
        x = (rng.normal(size=(T, H, D)) * 3).astype(src)
        xs.append(x)
        ins.append(layout(x, how) if H else None)
        y = layout(np.full((T, H, D), np.nan, dst), how) if H else None
        outs.append(y)
    qg.qg_qk_norm_rope(ins[0], ins[1], dev(w[0]) if norm else None, dev(w[1]) if norm else None, 1e-6,
                       dev(pos) if R else None, dev(freq) if R else None, pairing, outs[0], outs[1])
    torch.cuda.synchronize()
    for x, y, ww in zip(xs, outs, w):
        if y is None:
            continue
        n = ref.norm(x.astype(np.float64), ww.astype(np.float64) if norm else None, 1e-6)
        want = ref.rope(n, pos, freq, pairing)
        size = np.abs(want)
        if R:
            r = n[..., :R]
            i = np.arange(R // 2)
            a, b = (i, i + R // 2) if pairing == 0 else (2 * i, 2 * i + 1)
            both = np.abs(r[..., a]) + np.abs(r[..., b])
            size = size.copy()
            size[..., a] = both
            size[..., b] = both
        tol = 24 * 2.0 ** -24 * size
        if dst == "f2":
            tol = tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25
        err = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
        assert (err <= tol).all(), (err - tol).max()


def test_norm_rope_in_place(qg):
    import torch
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(50, 9, 128))).astype("f4")
    a, b, y = dev(x), dev(x), torch.empty(50, 9, 128, device="cuda")
    pos, f, w = dev(np.arange(50, dtype=np.int32)), dev(frequencies(128)), dev(np.ones(128, "f4"))
    qg.qg_qk_norm_rope(a, None, w, None, 1e-6, pos, f, 0, y, None)
    qg.qg_qk_norm_rope(b, None, w, None, 1e-6, pos, f, 0, b, None)
    assert torch.equal(b, y)


def test_norm_rope_leaves_what_lies_between(qg):
    """Strided outputs: nothing but the rows' own elements is written."""
    import torch
    x = dev(np.ones((4, 2, 64), "f4"))
    wide = torch.full((4, 200), 7.0, device="cuda")
    qg.qg_qk_norm_rope(x, None, None, None, 0.0, None, None, 0, wide[:, 5:133].unflatten(1, (2, 64)), None)
    assert (wide[:, 5:133] == 1).all() and (wide[:, :5] == 7).all() and (wide[:, 133:] == 7).all()


# ---------------------------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page,R,pairing,norm", [
    (1, 4, 16, 64, 0, True), (16, 4, 64, 64, 0, True), (37, 1, 16, 0, 0, False), (5, 3, 128, 64, 1, False),
    (130, 2, 32, 16, 0, True), (400, 1, 48, 2, 1, True)])
@pytest.mark.parametrize("how,src", [("rows", "f4"), ("gemv", "f4"), ("odd", "f2"), ("rows", "f2")])
def test_append_and_read(qg, D, T, H, page, R, pairing, norm, how, src):
    """Every byte of the cache is the plain implementation's: the codes and scales of the tokens written, and
    all others as they were.  What is read back is d * code + m, rounded once."""
    import torch
    rng = np.random.default_rng(T + D)
    pages = (T + 60) // page + 2
    cache = rng.integers(0, 256, (pages, H, page // 16, 18 * D), dtype=np.uint8)
    k, v = ((rng.normal(size=(T, H, D)) * 2).astype(src) for _ in range(2))
    k[0, 0, :64] = 0.5   # a group without a range: d = 0
    v[-1, -1] *= 1000
    pos = (rng.integers(0, 300000, T)).astype(np.int32)
    freq = frequencies(R)
    w = rng.uniform(0.5, 1.5, D).astype("f4") if norm else None
    slot = rng.permutation(pages * page)[:T].astype(np.int64)
    slot[rng.random(T) < 0.1] = -1
    if T > 4:
        slot[1], slot[2] = pages * page, 1 << 60  # outside: not written
    d_cache = dev(cache)
    qg.qg_kv4_append(layout(k, how), layout(v, how), None if w is None else dev(w), 1e-6, dev(pos) if R else None,
                     dev(freq) if R else None, pairing, dev(slot), d_cache, page)
    kk = ref.rope(ref.norm(k.astype(np.float64), None if w is None else w.astype(np.float64), 1e-6), pos, freq, pairing)
    held = []
    for part, x in ((0, kk), (1, v.astype(np.float64))):
        q = ref.quantize(x)
        ref.store(cache, page, slot, part, *q)
        held.append(ref.values(*q))
    assert np.array_equal(d_cache.cpu().numpy(), cache)
    ok = ((slot >= 0) & (slot < pages * page))[:, None, None]
    for kind in ("f4", "f2"):
        out = [layout(np.full((T, H, D), np.nan, kind), how) for _ in range(2)]
        qg.qg_kv4_read(d_cache, page, dev(slot), *out)
        for y, x in zip(out, held):
            assert np.array_equal(y.cpu().numpy(), np.where(ok, x, 0).astype(kind))


def test_append_extremes(qg):
    """Ties between two levels go to the even one; ranges past fp16 saturate and stay finite; tiny ranges and
    a single value hold their minimum."""
    import torch
    x = np.zeros((4, 1, 64), "f4")
    x[0, 0, :31] = np.arange(31) * 0.5 + 4     # d = 1, m = 4: halves lie between two codes
    x[0, 0, 31:] = 19
    x[1, 0, ::2] = 3e6                          # d = 65504 at most
    x[2, 0, ::2] = 1e-9                         # d rounds to 0
    x[3] = -2.5
    cache = torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8, device="cuda")
    slot = dev(np.arange(4, dtype=np.int64))
    qg.qg_kv4_append(dev(x), dev(-x), None, 0.0, None, None, 0, slot, cache, 16)
    k, v = torch.empty(4, 1, 64, device="cuda"), torch.empty(4, 1, 64, device="cuda")
    qg.qg_kv4_read(cache, 16, slot, k, v)
    k, v = k.cpu().numpy(), v.cpu().numpy()
    assert np.array_equal(k[0, 0, :31], 4 + np.rint(np.arange(31) * 0.5))
    assert np.isfinite(k).all() and np.isfinite(v).all()
    assert (k[2] == 0).all() and (k[3] == -2.5).all() and (v[3] == 2.5).all()


# ---------------------------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------------------------
def attention_case(seed, lens, nq, Hk, G, D, page, how="rows", peaked=False, spare=3, tail=0, width=None):
    """Inputs of a ragged batch: a cache of random entries (NaN scales wherever no place is), shuffled pages."""
    rng = np.random.default_rng(seed)
    nseq = len(lens)
    nq = np.asarray(nq if np.ndim(nq) else [nq] * nseq)
    width = width or max(1, (max(lens) + page - 1) // page)
    pages = sum((n + page - 1) // page for n in lens) + spare
    cache = np.full((pages, Hk, page // 16, 18 * D), 0xff, np.uint8)  # 0xffff is a NaN in fp16
    table = np.full((nseq, width), -7, np.int32)
    order = rng.permutation(pages)
    at = 0
    for s, n in enumerate(lens):
        for i in range((n + page - 1) // page):
            table[s, i] = order[at]
            at += 1
            used = min(page, n - i * page)
            x = rng.normal(size=(2, used, Hk, D)) * (2.0 if peaked else 1.0)
            slot = table[s, i] * page + np.arange(used)
            for part in (0, 1):
                ref.store(cache, page, slot, part, *ref.quantize(x[part]))
    start = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    T = int(start[-1]) + tail
    q = (rng.normal(size=(T, Hk * G, D)) * (1.5 if peaked else 0.5)).astype(np.float16)
    return dict(q=q, start=start, cache=cache, page=page, table=table, lens=np.asarray(lens, np.int32), scale=D ** -0.5,
                how=how, max_q=int(nq.max()) if nseq else 0)


def run_attention(qg, c, out=None, **kw):
    y = layout(np.full(c["q"].shape, 9, np.float16), c["how"]) if out is None else out
    qg.qg_attn_kv4(layout(c["q"], c["how"]), dev(c["start"]), c["max_q"], dev(c["cache"]), c["page"], dev(c["table"]),
                   dev(c["lens"]), c["scale"], y, **kw)
    return y


def check_attention(qg, c):
    got = run_attention(qg, c).cpu().numpy().astype(np.float64)
    want, bound = ref.attention(c["q"], c["start"], c["cache"], c["page"], c["table"], c["lens"], c["scale"],
                                np.full(c["q"].shape, 9.0))
    err = np.abs(got - want)
    assert (err <= bound).all(), ((err - bound).max(), np.argwhere(~(err <= bound))[:5])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hk,G", [(1, 1), (2, 4), (4, 12), (1, 16), (3, 17)])
@pytest.mark.parametrize("lens,nq", [
    ([1], 1), ([15, 16, 17], 1), ([0], 1), ([63, 64, 65, 0, 1], 1), ([300], 1), ([130, 5], 2), ([20, 3, 0, 90], [5, 3, 1, 0]),
    ([64], 16)])
def test_attention(qg, D, Hk, G, lens, nq):
    check_attention(qg, attention_case(D + G, lens, nq, Hk, G, D, 16 if D == 64 else 32))


@pytest.mark.parametrize("D,page,how,peaked", [
    (256, 64, "gemv", False), (256, 16, "odd", True), (128, 128, "heads first", True), (128, 48, "gemv", False),
    (64, 256, "odd", False), (64, 32, "rows", True)])
def test_attention_layouts_pages_and_peaked_scores(qg, D, page, how, peaked):
    check_attention(qg, attention_case(5, [777, 33, 1300], [1, 4, 3], 2, 6, D, page, how, peaked))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,nq", [([40], 40), ([500], 37), ([130, 90], [70, 90])])
def test_attention_of_a_prompt(qg, D, lens, nq):
    check_attention(qg, attention_case(7, lens, nq, 2, 4, D, 64))


def test_attention_more_queries_than_places(qg):
    """The first queries of a sequence with more new tokens than places see nothing: zeros."""
    c = attention_case(3, [3, 1], [6, 4], 1, 4, 128, 16)
    got = run_attention(qg, c).cpu().numpy()
    assert (got[:3] == 0).all() and (got[6:9] == 0).all()
    check_attention(qg, c)


def test_attention_long_context_is_cut_between_ctas(qg):
    """One long sequence on one key head, thousands of units over every CTA, and its join."""
    check_attention(qg, attention_case(11, [40001], 1, 1, 8, 128, 64, spare=0))
    check_attention(qg, attention_case(12, [9001, 0, 70], [2, 1, 1], 1, 12, 256, 32))


def test_attention_many_sequences(qg):
    """More items than CTAs, lengths from nothing up."""
    rng = np.random.default_rng(0)
    check_attention(qg, attention_case(13, list(rng.integers(0, 90, 400)), 1, 2, 2, 64, 16))
    check_attention(qg, attention_case(14, list(rng.integers(1, 200, 160)), list(rng.integers(0, 4, 160)), 1, 7, 64, 32))


def test_attention_rows_of_no_sequence_stay(qg):
    c = attention_case(2, [50, 20], [1, 2], 1, 4, 64, 16, tail=5)
    got = run_attention(qg, c).cpu().numpy()
    assert (got[3:] == 9).all() and (got[:3] != 9).any()
    check_attention(qg, c)


def test_attention_skips_bad_pages(qg):
    c = attention_case(4, [200, 64], [1, 2], 2, 4, 128, 32)
    c["table"][0, 2] = len(c["cache"])
    c["table"][0, 5] = -1
    c["table"][1, :] = [2 ** 31 - 1, -2 ** 31] + [0] * (c["table"].shape[1] - 2)
    got = run_attention(qg, c).cpu().numpy()
    assert (got[1:] == 0).all()  # no page of the second sequence is there
    check_attention(qg, c)


def test_attention_lengths_out_of_range(qg):
    """A length past the table is taken as all of it, a negative one as none; query starts out of range or
    falling give rows of no sequence."""
    c = attention_case(6, [64, 32], 1, 1, 2, 64, 32)
    c["lens"] = np.array([5000, -3], np.int32)
    c["table"] = c["table"][:, :2].copy()
    check_attention(qg, c)
    d = attention_case(6, [64, 32, 40], 1, 1, 2, 64, 32)
    d["start"] = np.array([1, 0, 90, 2], np.int32)
    y = run_attention(qg, d).cpu().numpy()
    assert (y[0] == 0).sum() >= 0  # no fault; what the call means is not defined


def test_attention_is_the_same_every_time_and_on_any_stream(qg):
    import torch
    c = attention_case(8, [5000, 1, 700], [2, 1, 3], 2, 6, 128, 64)
    first = run_attention(qg, c).clone()
    for _ in range(3):
        assert torch.equal(run_attention(qg, c), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run_attention(qg, c)
    s.synchronize()
    assert torch.equal(other, first)
    ws = torch.full((qg.qg_attn_kv4_workspace(12, 2, 128, c["max_q"]),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(run_attention(qg, c, workspace=ws), first)  # a workspace's contents do not matter
    assert ws[:4].view(torch.int32).item() == 0
    with pytest.raises(qg.QgError):
        run_attention(qg, c, workspace=ws[:-256])
    with pytest.raises(ValueError):
        run_attention(qg, c, stream=s)


def test_attention_graphs_do_not_share_a_workspace(qg):
    """Two graphs captured on one stream, replayed on two at once, many times."""
    import torch
    cs = [attention_case(20 + i, [6000, 3000 + i], 1, 2, 4, 128, 64) for i in range(2)]
    want = [run_attention(qg, c).clone() for c in cs]
    graphs, outs = [], []
    for c in cs:
        t = [layout(c["q"], "rows"), dev(c["start"]), dev(c["cache"]), dev(c["table"]), dev(c["lens"])]
        y = torch.zeros_like(t[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.qg_attn_kv4(t[0], t[1], 1, t[2], c["page"], t[3], t[4], c["scale"], y)
        graphs.append((g, t))
        outs.append(y)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for y, w in zip(outs, want):
        assert torch.equal(y, w)


def test_attention_far_pages(qg):
    """Pages past 2^32 bytes of a cache."""
    import torch
    c = attention_case(9, [100, 40], 1, 2, 4, 256, 64)
    pages = (5 << 30) // (2 * 4 * 18 * 256)
    big = torch.empty(pages, 2, 4, 18 * 256, dtype=torch.uint8, device="cuda")
    n = len(c["cache"])
    big[pages - n:] = dev(c["cache"])
    y = layout(np.full(c["q"].shape, 9, np.float16), "rows")
    table = np.where(c["table"] >= 0, c["table"] + pages - n, c["table"]).astype(np.int32)
    qg.qg_attn_kv4(layout(c["q"], "rows"), dev(c["start"]), 1, big, 64, dev(table), dev(c["lens"]), c["scale"], y)
    assert torch.equal(y, run_attention(qg, c))
    # the append and the read reach them too
    slot = dev(np.array([pages * 64 - 1, 0], np.int64))
    x = torch.randn(2, 2, 256, device="cuda")
    k, v = torch.empty_like(x), torch.empty_like(x)
    qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, big, 64)
    qg.qg_kv4_read(big, 64, slot, k, v)
    assert torch.equal(k, v) and (k - x).abs().max() < 0.5


# ---------------------------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------------------------
def run_sample(qg, x, t=None, k=None, p=None, mp=None, u=None, major="row"):
    import torch
    R = x.shape[0]
    lx = dev(x) if major == "row" else dev(x.T).t()
    tok = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    f = lambda a, kind: None if a is None else dev(np.asarray(a, kind))  # noqa: E731
    qg.qg_sample(lx, f(t, "f4"), f(k, "i4"), f(p, "f4"), f(mp, "f4"), f(u, "f4"), tok)
    return tok.cpu().numpy()


def check_sample(qg, x, t=None, k=None, p=None, mp=None, u=None, major="row"):
    got = run_sample(qg, x, t, k, p, mp, u, major)
    at = lambda a, i, kind: None if a is None else np.asarray(a, kind)[i]  # noqa: E731
    want = [ref.sample(x[i], at(t, i, "f4"), at(k, i, "i4"), at(p, i, "f4"), at(mp, i, "f4"), at(u, i, "f4")) for i in range(len(x))]
    assert got.tolist() == want


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1025, 8193, 50257, 151936])
@pytest.mark.parametrize("major", ["row", "vocabulary"])
@pytest.mark.parametrize("kind", ["plain", "topk", "topp", "both", "minp", "all", "wide"])
def test_sample(qg, V, major, kind):
    rng = np.random.default_rng(V)
    R = 9
    x = (rng.normal(size=(R, V)) * 2.5).astype("f4")
    x[:, rng.integers(0, V, 5)] += 7
    u = rng.random(R).astype("f4")
    u[0], u[1] = 0.0, np.float32(1 - 2.0 ** -24)
    t = rng.uniform(0.3, 1.6, R)
    k = rng.integers(1, 60, R)
    p = rng.uniform(0.05, 0.99, R)
    mp = rng.uniform(0.001, 0.3, R)
    use = {"plain": {}, "topk": dict(k=k), "topp": dict(p=p), "both": dict(k=k, p=p), "minp": dict(mp=mp),
           "all": dict(k=k * 3, p=p, mp=mp), "wide": dict(k=k * 100, p=1 - (1 - p) * 0.01)}[kind]
    check_sample(qg, x, t=t, u=u, major=major, **use)


@pytest.mark.parametrize("V", [5, 3000, 40000])
def test_sample_ties(qg, V):
    """Rows of few different values: the lower index goes first, through lists and through finer histograms."""
    rng = np.random.default_rng(V)
    R = 12
    x = rng.integers(-2, 3, (R, V)).astype("f4") * 0.5
    x[3] = 1.25           # all equal
    x[4, ::2] = -0.0      # the two zeros are equal
    x[4, 1::2] = 0.0
    x[5] = np.nextafter(np.float32(2), np.float32(3)) if V == 5 else x[5]
    u = rng.random(R)
    for kw in (dict(), dict(k=rng.integers(1, V + 3, R)), dict(p=rng.uniform(0, 1, R)),
               dict(k=rng.integers(1, V + 3, R), p=rng.uniform(0, 1, R), mp=rng.uniform(0, 0.9, R)), dict(t=np.zeros(R))):
        check_sample(qg, x, u=u, **kw)


@pytest.mark.parametrize("equal", [1000, 1500, 2500])
def test_sample_many_equal_at_the_top(qg, equal):
    """The cut among so many equal logits that a list holds them, just so, or does not."""
    rng = np.random.default_rng(equal)
    R, V = 10, 9000
    x = rng.normal(size=(R, V)).astype("f4")
    for i in range(R):
        x[i, rng.permutation(V)[:equal]] = 5.0 if i % 2 else x[i].max() - 1.0
    u = rng.random(R)
    p = np.array([0.0, 0.0, 1e-9, 1e-9, 0.2, 0.2, 0.5, 0.5, 0.97, 0.97])
    for kw in (dict(p=p), dict(p=p, k=np.full(R, 1300)), dict(p=p, mp=np.full(R, 0.3)), dict(k=np.full(R, equal - 3))):
        check_sample(qg, x, u=u, **kw)


@pytest.mark.parametrize("V", [700, 50257])
def test_sample_share_against_min_p(qg, V):
    """Either of top-p and min-p may be the one that cuts, far from the other's cut or next to it."""
    rng = np.random.default_rng(V)
    R = 24
    x = (rng.normal(size=(R, V)) * 2).astype("f4")
    u = rng.random(R)
    p = rng.uniform(0.05, 0.999, R)
    for least in (1e-30, 1e-4, 0.02, 0.3, 1.0, 1.5):
        mp = least * rng.uniform(0.7, 1.0, R) if least < 1 else np.full(R, least)
        check_sample(qg, x, u=u, p=p, mp=mp)
        check_sample(qg, x, u=u, p=p, mp=mp, k=rng.integers(1, 3 * V // 2, R))
    # min_p next to the weight of the last token that top-p keeps
    z = np.sort(x.astype(np.float64), 1)[:, ::-1]
    w = np.exp(z - z[:, :1])
    n = (np.cumsum(w, 1) - w < p[:, None] * w.sum(1, keepdims=True)).sum(1)
    edge = w[np.arange(R), n - 1]
    for f in (0.97, 0.999, 1.001, 1.03):
        check_sample(qg, x, u=u, p=p, mp=np.minimum(edge * f, 1.0))
    x[:, ::7] = x.max()  # equal logits at the top: only the first is never dropped
    check_sample(qg, x, u=u, mp=np.full(R, 1.25), p=p)


def test_sample_masked_rows_and_odd_settings(qg):
    rng = np.random.default_rng(5)
    V = 9000
    x = rng.normal(size=(16, V)).astype("f4")
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 1:] = -np.inf
    x[3, ::3] = np.nan
    x[4, 5:] = -np.inf
    x[5] = np.finfo("f4").min      # masked with the type's lowest value
    x[5, 77] = 0
    x[6, [10, 500]] = np.inf       # two infinite logits share everything
    x[7] *= 1e30
    u = rng.random(16)
    k = rng.integers(-1, 30, 16)
    k[4] = 4000                    # more than are left
    p = rng.uniform(0, 1, 16)
    p[8], p[9], p[10] = 0.0, 1.0, 2.0
    mp = rng.uniform(0, 1, 16)
    mp[11], mp[12] = 0.0, 1.0
    t = rng.uniform(0.1, 3, 16)
    t[13], t[14], t[15] = 0.0, -1.0, 1e-20
    for kw in (dict(), dict(k=k), dict(p=p), dict(mp=mp), dict(k=k, p=p, mp=mp), dict(p=p, mp=mp), dict(t=t, k=k, p=p, mp=mp)):
        check_sample(qg, x, u=u, **kw)
    # u of 1 or NaN takes the last kept token
    assert run_sample(qg, np.zeros((2, 50), "f4"), k=[7, 7], u=[1.0, np.nan]).tolist() == [6, 6]
    assert run_sample(qg, np.zeros((2, 50), "f4"), u=[1.0, np.nan]).tolist() == [49, 49]


def test_sample_large_vocabulary_and_many_rows(qg):
    """More logits than a cluster's shared memory holds, and more rows than the card takes at once."""
    rng = np.random.default_rng(2)
    x = (rng.normal(size=(3, 600_001)) * 2).astype("f4")
    check_sample(qg, x, u=[0.1, 0.5, 0.9], p=[0.2, 0.9, 0.999], k=[0, 20, 5000])
    check_sample(qg, x, u=[0.1, 0.5, 0.9])
    x = (rng.normal(size=(300, 700)) * 2).astype("f4")
    check_sample(qg, x, u=rng.random(300), p=rng.uniform(0, 1, 300))


def test_sample_rows_that_no_cluster_holds(qg):
    """Rows too long for the shared memory of eight processors, of more rows than sixteen are taken for; and the longest."""
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(9, 420_001)) * 2).astype("f4")
    x[2] = rng.integers(-3, 3, x.shape[1])  # ties past any list
    u = rng.random(9)
    check_sample(qg, x, u=u, p=rng.uniform(0.1, 1, 9), k=rng.integers(0, 3000, 9))
    check_sample(qg, x, u=u, p=rng.uniform(0.1, 1, 9), mp=rng.uniform(0, 0.1, 9), major="vocabulary")
    x = np.zeros((2, (1 << 20) - 1), "f4")
    x[1] = rng.normal(size=x.shape[1])
    check_sample(qg, x, u=[0.999, 0.25])


def test_sample_tiny_temperatures_and_random_numbers_below_zero(qg):
    x = np.array([[0, 1, 3, 3, 2], [-1, 0, 0, 0, -2]], "f4").repeat(3, 0)
    for t in (1.2e-38, 1e-40, 1.5e-45):
        check_sample(qg, x, t=np.full(6, t, "f4"), u=[0.1, 0.6, 0.9, 0.1, 0.5, 0.9], p=[1, 0.9, 0.4, 1, 0.9, 0.2])
    assert run_sample(qg, x[:2], u=[-1.0, -np.inf]).tolist() == [0, 0]


def test_sample_side_by_side_without_a_workspace(qg):
    """The C entry takes rows side by side as they are where it gets no workspace."""
    import torch
    rng = np.random.default_rng(9)
    x = (rng.normal(size=(5, 30_011)) * 2).astype("f4")
    u, p = rng.random(5).astype("f4"), rng.uniform(0.3, 0.99, 5).astype("f4")
    lx, du, dp = dev(x.T), dev(u), dev(p)
    tok = torch.full((7,), -9, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert qg.lib().qg_sample(lx.data_ptr(), 5, 30_011, 1, 5, None, None, dp.data_ptr(), None, du.data_ptr(), tok.data_ptr(), None, 0,
                              st) == qg.QG_OK
    assert tok.cpu().tolist() == [ref.sample(x[i], None, None, p[i], None, u[i]) for i in range(5)] + [-9, -9]


def test_calls_on_two_streams_at_once(qg):
    """Attention and sampling on two streams, launched so that they may overlap, give what they give alone."""
    import torch
    rng = np.random.default_rng(11)
    cache = qg.kv4_cache(40, 64, 2, 128)
    kv = torch.randn(40 * 64, 2, 128, device="cuda")
    qg.qg_kv4_append(kv, kv, None, 0.0, None, None, 0, torch.arange(40 * 64, device="cuda"), cache, 64)
    sets = []
    for i in range(2):
        q = torch.randn(3, 8, 128, device="cuda", dtype=torch.float16)
        table = dev(np.stack([rng.permutation(40) for _ in range(3)]).astype(np.int32))
        lens = dev(rng.integers(1, 2560, 3).astype(np.int32))
        x = torch.randn(4, 60_000, device="cuda").t().contiguous().t()
        u = torch.rand(4, device="cuda")
        sets.append((q, table, lens, x, u))
    start = dev(np.arange(4, dtype=np.int32))

    def go(s, out, tok):
        q, table, lens, x, u = s
        qg.qg_attn_kv4(q, start, 1, cache, 64, table, lens, 0.1, out)
        qg.qg_sample(x, None, None, None, None, u, tok)

    fresh = lambda: (torch.zeros(3, 8, 128, device="cuda", dtype=torch.float16), torch.zeros(4, device="cuda", dtype=torch.int32))  # noqa: E731
    want = [fresh() for _ in sets]
    for s, w in zip(sets, want):
        go(s, *w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[fresh() for _ in range(20)] for _ in sets]
    torch.cuda.synchronize()
    for r in range(20):
        for s, g, st in zip(sets, got, streams):
            with torch.cuda.stream(st):
                go(s, *g[r])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for out, tok in g:
            assert torch.equal(out, w[0]) and torch.equal(tok, w[1])


def test_sample_follows_the_weights(qg):
    """Evenly spread random numbers reach every token in proportion to its weight."""
    import torch
    x = np.log(np.array([1, 2, 3, 4, 0.5], "f4"))[None].repeat(1050, 0)
    u = (np.arange(1050) + 0.5) / 1050
    got = np.bincount(run_sample(qg, x, u=u), minlength=5)
    assert np.abs(got - np.array([100, 200, 300, 400, 50])).max() <= 1


def test_sample_in_a_graph(qg):
    import torch
    x = torch.randn(4, 30000, device="cuda")
    u = torch.rand(4, device="cuda")
    tok, p = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((4,), 0.9, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qg_sample(x, None, None, p, None, u, tok)
    for _ in range(3):
        x.normal_()
        u.uniform_()
        g.replay()
        check = torch.zeros_like(tok)
        qg.qg_sample(x, None, None, p, None, u, check)
        assert torch.equal(tok, check)


def test_wrappers_refuse(qg):
    import torch
    x = torch.zeros(2, 2, 64, device="cuda")
    cache = qg.kv4_cache(2, 16, 2, 64)
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        qg.qg_kv4_append(x.cpu(), x, None, 0.0, None, None, 0, slot, cache, 16)
    with pytest.raises(ValueError):
        qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot.int(), cache, 16)
    with pytest.raises(ValueError):
        qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, cache, 32)
    with pytest.raises(ValueError):
        qg.qg_kv4_append(x.double(), x, None, 0.0, None, None, 0, slot, cache, 16)
    with pytest.raises(ValueError):
        qg.qg_kv4_append(x[:, :1], x[:, :1], None, 0.0, None, None, 0, slot, cache, 16)
    with pytest.raises(ValueError):
        qg.qg_qk_norm_rope(x, None, None, None, 0.0, None, torch.ones(4, dtype=torch.float64, device="cuda"), 0, x, None)
    with pytest.raises(ValueError):
        qg.qg_attn_kv4(x, slot, 1, cache, 16, slot, slot, 1.0, x)
    with pytest.raises(ValueError):
        qg.qg_sample(x[0], None, None, torch.ones(3, device="cuda"), None, torch.ones(2, device="cuda"),
                     torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(qg.QgError):
        qg.kv4_cache(2, 24, 2, 64)


def test_wrappers_refuse_what_the_c_abi_cannot_see(qg):
    """Types, shapes, missing arguments and foreign streams, before anything is launched."""
    import torch
    x = torch.zeros(2, 2, 64, device="cuda")
    h = x.half()
    cache = qg.kv4_cache(2, 16, 2, 64)
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    start = torch.arange(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    f = torch.ones(2, device="cuda")
    cols = torch.zeros(9, 2, device="cuda").t()
    side = torch.cuda.Stream()
    bad = [
        lambda: qg.qg_kv4_append(x, None, None, 0.0, None, None, 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x[0], x[0], None, 0.0, None, None, 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x, x[:1], None, 0.0, None, None, 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x, x, torch.ones(128, device="cuda")[::2], 0.0, None, None, 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x, x, None, 0.0, i32, torch.ones(8, device="cuda"), 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x, x, None, 0.0, i32, torch.ones(512, dtype=torch.float64, device="cuda"), 0, slot, cache, 16),
        lambda: qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, cache.view(-1), 16),
        lambda: qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, cache[:, :1], 16),
        lambda: qg.qg_kv4_read(cache, 16, slot, x, x[:, :1]),
        lambda: qg.qg_kv4_read(cache, 16, slot[:1], x, x),
        lambda: qg.qg_qk_norm_rope(None, None, None, None, 0.0, None, None, 0, None, None),
        lambda: qg.qg_qk_norm_rope(x, None, None, None, 0.0, None, None, 0, None, None),
        lambda: qg.qg_qk_norm_rope(x, x[:1], None, None, 0.0, None, None, 0, x, x[:1]),
        lambda: qg.qg_attn_kv4(h, start, 1, cache, 16, table, i32, 1.0, x),
        lambda: qg.qg_attn_kv4(h, start[:2], 1, cache, 16, table, i32, 1.0, h),
        lambda: qg.qg_attn_kv4(h, start, 1, cache, 16, table, slot, 1.0, h),
        lambda: qg.qg_attn_kv4(h, start, 1, cache, 16, table.t(), i32, 1.0, h),
        lambda: qg.qg_attn_kv4(h, start, 1 << 40, cache, 16, table, i32, 1.0, h),
        lambda: qg.qg_attn_kv4(h, start, 1, cache, 16, table, i32, 1.0, torch.empty_like(h), stream=side),
        lambda: qg.qg_sample(cols, None, None, None, None, f, i32, stream=side),
        lambda: qg.qg_sample(cols, None, None, None, None, f, slot),
        lambda: qg.qg_sample(cols.half(), None, None, None, None, f, i32),
        lambda: qg.qg_sample(cols, None, f, None, None, f, i32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: qg.qg_attn_kv4(h[:, :1], start, 1, cache, 16, table, i32, 1.0, h[:, 1:]),  # one query head of two
                 lambda: qg.qg_qk_norm_rope(x, None, None, None, -1.0, None, None, 0, x, None)):
        with pytest.raises(qg.QgError):
            call()
    for call in (lambda: qg.qg_sample(cols, None, None, None, None, f, i32, stream="x"),
                 lambda: qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, cache, "16")):
        with pytest.raises((AttributeError, TypeError)):
            call()
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------------------------
def test_a_decode_step(qg, orc):
    """One attention layer and the sampler as a decode step runs them, for three columns of three sequences:
    the Q, K and V projections (GEMVs), norms and rotation, append, attention, the output projection with its
    residual, the output head, the token; captured in one graph.  Each stage is checked from the inputs that
    it really had, by its own reference."""
    import torch
    K, Hq, Hk, D, B, R, V, page = 512, 8, 2, 64, 3, 16, 1000, 16
    rng = np.random.default_rng(0)
    fmt = qg.QG_FMT_Q4_K
    W = {n: synth.weights(fmt, rows, k, seed=i) for i, (n, rows, k) in enumerate(
        [("q", Hq * D, K), ("k", Hk * D, K), ("v", Hk * D, K), ("o", K, Hq * D), ("head", V, K)])}
    Wd = {n: dev(w) for n, w in W.items()}
    lens = np.array([40, 17, 1], np.int32)   # the new token included
    c = attention_case(1, [int(n) for n in lens], 1, Hk, 1, D, page)
    cache, table = dev(c["cache"]), dev(c["table"])
    slot = np.array([c["table"][s, (n - 1) // page] * page + (n - 1) % page for s, n in enumerate(lens)], np.int64)
    x = synth.activations(K, B, seed=3)
    xd = dev(x.view(np.uint16)).view(torch.float16)
    wq, wk = (rng.uniform(0.5, 1.5, D).astype("f4") for _ in range(2))
    pos, freq, u = (lens - 1).astype(np.int32), frequencies(R), rng.random(B).astype("f4")
    t = {n: dev(a) for n, a in dict(wq=wq, wk=wk, pos=pos, freq=freq, u=u, slot=slot, lens=lens,
                                    start=np.arange(B + 1, dtype=np.int32), p=np.full(B, 0.9, "f4")).items()}
    f = lambda n: torch.empty(n, B, device="cuda")  # noqa: E731
    yq, yk, yv, res, logits = f(Hq * D), f(Hk * D), f(Hk * D), torch.zeros(K, B, device="cuda"), f(V)
    q16, a16 = (torch.empty(Hq * D, B, dtype=torch.float16, device="cuda") for _ in range(2))
    h16 = torch.empty(K, B, dtype=torch.float16, device="cuda")
    tok = torch.zeros(B, dtype=torch.int32, device="cuda")
    view = lambda y, H: y.view(H, D, B).permute(2, 0, 1)  # noqa: E731
    scale = D ** -0.5

    def step():
        qg.qg_gemv(Wd["q"], fmt, Hq * D, K, xd, B, yq)
        qg.qg_gemv(Wd["k"], fmt, Hk * D, K, xd, B, yk)
        qg.qg_gemv(Wd["v"], fmt, Hk * D, K, xd, B, yv)
        qg.qg_qk_norm_rope(view(yq, Hq), None, t["wq"], None, 1e-6, t["pos"], t["freq"], qg.QG_ROPE_HALVES, view(q16, Hq), None)
        qg.qg_kv4_append(view(yk, Hk), view(yv, Hk), t["wk"], 1e-6, t["pos"], t["freq"], qg.QG_ROPE_HALVES, t["slot"], cache, page)
        qg.qg_attn_kv4(view(q16, Hq), t["start"], 1, cache, page, table, t["lens"], scale, view(a16, Hq))
        qg.qg_gemv_residual(Wd["o"], fmt, K, Hq * D, a16, B, res, res)
        h16.copy_(res)
        qg.qg_gemv(Wd["head"], fmt, V, K, h16, B, logits)
        qg.qg_sample(logits.t(), None, None, t["p"], None, t["u"], tok)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # the GEMVs make their workspaces, one a stream
    torch.cuda.synchronize()
    cache.copy_(dev(c["cache"]))
    res.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    g.replay()
    torch.cuda.synchronize()
    host = lambda a: a.cpu().numpy()  # noqa: E731
    rows = lambda y, H: host(view(y, H)).astype(np.float64)  # noqa: E731
    for y, n, H in ((yq, "q", Hq), (yk, "k", Hk), (yv, "v", Hk)):
        want, A = orc.gemv(W[n], fmt, H * D, K, x, B)
        assert (np.abs(host(y) - want) <= 1e-5 * A + 1e-6).all()
    want = ref.rope(ref.norm(rows(yq, Hq), wq.astype(np.float64), 1e-6), pos, freq, 0)
    assert np.abs(rows(q16, Hq) - want).max() <= 2.0 ** -10 * np.abs(want).max()
    plain = c["cache"].copy()
    kk = ref.rope(ref.norm(rows(yk, Hk), wk.astype(np.float64), 1e-6), pos, freq, 0)
    ref.store(plain, page, slot, 0, *ref.quantize(kk))
    ref.store(plain, page, slot, 1, *ref.quantize(rows(yv, Hk)))
    assert np.array_equal(host(cache), plain)
    q = host(view(q16, Hq))
    want, bound = ref.attention(q, np.arange(B + 1), plain, page, c["table"], lens, scale, np.zeros(q.shape))
    assert (np.abs(rows(a16, Hq) - want) <= bound).all()
    want, A = orc.gemv(W["o"], fmt, K, Hq * D, host(a16), B)
    assert (np.abs(host(res) - want) <= 1e-5 * A + 1e-6).all()
    lg = host(logits)
    assert host(tok).tolist() == [ref.sample(lg[:, b], None, None, np.float32(0.9), None, u[b]) for b in range(B)]
