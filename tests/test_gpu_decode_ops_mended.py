"""The operators between the GEMVs where they had gone wrong, or were not compared with anything: views that run
backwards, many tokens, wrong guesses of max_q, sizes at the ends of their ranges."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref
import test_gpu_decode_ops as decode
from test_gpu_decode_ops import attention_case, check_attention, dev, frequencies, layout, qg, run_attention, run_sample  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------
# Views with negative strides, which torch has not, through the C ABI
# ---------------------------------------------------------------------------------------------
def backwards(qg, t, tokens, heads):
    """A contiguous [T, H, D] tensor as the view whose tokens and / or heads run from the last to the first."""
    T, H, D = t.shape
    at = t.data_ptr() + t.element_size() * D * ((T - 1) * H * tokens + (H - 1) * heads)
    kind = qg.QG_TYPE_F32 if t.element_size() == 4 else qg.QG_TYPE_F16
    return ctypes.byref(qg.qg_heads(at, -H * D if tokens else H * D, -D if heads else D, 1, kind))


@pytest.mark.parametrize("lens,nq", [([90, 20], [1, 3]), ([5000], 2), ([700, 300], [40, 9])])  # whole items; cut ones
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tokens,heads", [(1, 0), (0, 1), (1, 1)])
def test_attention_of_views_that_run_backwards(qg, lens, nq, D, tokens, heads):
    """The result is that of the same values in order, and goes where the view says."""
    import torch
    c = attention_case(31, lens, nq, 2, 4, D, 32)
    want = run_attention(qg, c).cpu().numpy()
    flip = tuple(a for a, on in ((0, tokens), (1, heads)) if on)
    q, out = dev(np.flip(c["q"], flip)), dev(np.full(c["q"].shape, 9, np.float16))
    t = [dev(c[n]) for n in ("start", "cache", "table", "lens")]
    T, Hq, _ = c["q"].shape
    ws = torch.empty(qg.qg_attn_kv4_workspace(Hq, 2, D, c["max_q"]), dtype=torch.uint8, device="cuda")
    rc = qg.lib().qg_attn_kv4(backwards(qg, q, tokens, heads), T, len(lens), t[0].data_ptr(), c["max_q"], Hq, 2, D, t[1].data_ptr(),
                              len(c["cache"]), 32, t[2].data_ptr(), t[2].shape[1], t[3].data_ptr(), c["scale"],
                              backwards(qg, out, tokens, heads), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == qg.QG_OK
    assert np.array_equal(np.flip(out.cpu().numpy(), flip), want)


@pytest.mark.parametrize("tokens,heads", [(1, 0), (0, 1), (1, 1)])
def test_head_operators_on_views_that_run_backwards(qg, tokens, heads):
    """Norm and rotation, append and read give what they give in order."""
    import torch
    rng = np.random.default_rng(3)
    T, H, D, page = 21, 6, 128, 16
    x = rng.normal(size=(T, H, D)).astype("f4")
    flip = tuple(a for a, on in ((0, tokens), (1, heads)) if on)
    w, pos, freq = dev(rng.uniform(0.5, 1.5, D).astype("f4")), dev(np.arange(T, dtype=np.int32)), dev(frequencies(64))
    slot = dev(rng.permutation(4 * page)[:T].astype(np.int64))
    st = torch.cuda.current_stream().cuda_stream
    fwd, y = dev(x), torch.empty(T, H, D, device="cuda")
    back, z = dev(np.flip(x, flip)), torch.empty(T, H, D, device="cuda")
    qg.qg_qk_norm_rope(fwd, None, w, None, 1e-6, pos, freq, 0, y, None)
    v = lambda t: backwards(qg, t, tokens, heads)  # noqa: E731
    assert qg.lib().qg_qk_norm_rope(v(back), None, T, H, 0, D, w.data_ptr(), None, 1e-6, pos.data_ptr(), freq.data_ptr(), 64, 0, v(z),
                                    None, st) == qg.QG_OK
    assert torch.equal(z.flip(flip), y)
    one, two = qg.kv4_cache(4, page, H, D), qg.kv4_cache(4, page, H, D)
    qg.qg_kv4_append(fwd, fwd, w, 1e-6, pos, freq, 0, slot, one, page)
    assert qg.lib().qg_kv4_append(v(back), v(back), T, H, D, w.data_ptr(), 1e-6, pos.data_ptr(), freq.data_ptr(), 64, 0, slot.data_ptr(),
                                  two.data_ptr(), 4, page, st) == qg.QG_OK
    assert torch.equal(one, two)
    a, b, k, u = (torch.empty(T, H, D, device="cuda") for _ in range(4))
    qg.qg_kv4_read(one, page, slot, a, b)
    assert qg.lib().qg_kv4_read(one.data_ptr(), 4, page, H, D, slot.data_ptr(), T, v(k), v(u), st) == qg.QG_OK
    assert torch.equal(k.flip(flip), a) and torch.equal(u.flip(flip), b)


# ---------------------------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("V", [20_000, 151_936])
def test_sample_share_on_the_border_of_two_threads_bins(qg, V):
    """Shares whose bounds fall on the border between two threads' bins of the histogram, where the two add up the
    weight after it in another order: the bins next to the cut are the same for every CTA of a cluster, and the
    token that of the definition, every time."""
    import torch
    rng = np.random.default_rng(V)
    R = 160
    x = (rng.normal(size=(1, V)) * 2).astype("f4").repeat(R, 0)
    t = (x[0].max() - x[0].astype(np.float64)) * np.log2(np.e)
    count = np.bincount(np.rint(64 * t).astype(int), minlength=4096)
    b = np.arange(4096)
    total = np.exp2(-t).sum()
    p = np.empty(R, "f4")
    for i in range(R):
        border = 4 * (32 * (1 + i // 40) if i % 2 else 20 + i)  # between warps, and within one
        part = (count * np.exp2(-(b + (-0.5 if i % 4 < 2 else 0.5)) / 64) * (1.0002 if i % 4 < 2 else 0.9998))[border:].sum()
        p[i] = 1 - part / total
    assert 0 < p.min() and p.max() < 1
    u = rng.random(R).astype("f4")
    want = [ref.sample(x[i], None, None, p[i], None, u[i]) for i in range(R)]
    lx, du = dev(x), dev(u)
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    for _ in range(5):
        qg.qg_sample(lx, None, None, dev(p), None, du, tok)
        assert tok.tolist() == want
    one = torch.zeros(1, dtype=torch.int32, device="cuda")  # a row alone: a larger cluster
    for i in range(R):
        qg.qg_sample(lx[:1], None, None, dev(p[i:i + 1]), None, du[i:i + 1], one)
        assert one.item() == want[i]


@pytest.mark.parametrize("V", [151_936, (1 << 20) - 1])
@pytest.mark.parametrize("deep", [43.01, 44.4, 40.3, 43.5, 36.7, 45.5, 24.0])
def test_sample_of_one_logit_and_a_long_flat_tail(qg, V, deep):
    """Weights next to the least that counts, a vocabulary full of them.  A weight is off by 2^-45 at most and 2^-30 of
    itself, so a token is right for a u that is off by V 2^-45 and 2^-29 (the sum and the total)."""
    x = np.full((2, V), -deep * np.log(2), "f4")
    x[0, V - 1] = 0   # the tail first
    x[1, 0] = 0       # ... and last
    w = np.exp(x.astype(np.float64))
    c = np.cumsum(w, 1)
    total = c[:, -1]
    near = np.array([0.03, 0.2, 0.5, 0.8, 0.97]) * w[0, 0] * (V - 1)
    u = np.stack([near / total[0], (1 + near) / total[1]]).clip(0, 1 - 2.0 ** -24).astype("f4")
    far = V * 2.0 ** -45 + 2.0 ** -29
    for i in range(u.shape[1]):
        got = run_sample(qg, x, u=u[:, i])
        for r in range(2):
            j = got[r]
            assert 0 <= j < V
            at, before = c[r, j] / total[r], (c[r, j] - w[r, j]) / total[r]
            assert before - far <= u[r, i] <= at + far, (r, i, j, u[r, i], before, at)


@pytest.mark.parametrize("middle", [900, 1200, 1800, 2040, 2300, 3000, 20_000])  # lists sorted, listed, and over the row
def test_sample_share_that_ends_where_a_deep_tail_begins(qg, middle):
    """A share of 1 - 2^-24 that ends just behind the middle weights, by the weight of a million of the smallest that
    there are: all of the middle is kept (what the tail weighs decides no more than the tail), through every path."""
    V = (1 << 20) - 1
    rng = np.random.default_rng(middle)
    x = np.empty((4, V), "f4")
    level = 12 + np.log2(middle / 3000)
    x[:] = -(44 - np.log2(1.7)) * np.log(2)             # the tail: 1.7 x 2^-44 each, less than 2^-24 of all
    x[:, rng.permutation(V)[:middle]] = -level * np.log(2)
    x[:, V // 2] = 0
    p = np.full(4, 1 - 2.0 ** -24, "f4")
    u = np.array([0.05, 0.4, 0.6, 0.95], "f4")
    w = np.exp(x[0].astype(np.float64))
    kept = np.where(x[0] > -20, w, 0.0)
    assert w.sum() - kept.sum() < (1 - float(p[0])) * w.sum()
    c = np.cumsum(kept)
    got = run_sample(qg, x, p=p, u=u)
    for i in range(4):
        j = got[i]
        assert kept[j] > 0 and (c[j] - kept[j]) / c[-1] - 2.0 ** -22 <= u[i] <= c[j] / c[-1] + 2.0 ** -22


# ---------------------------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------------------------
def test_attention_over_the_longest_table(qg):
    """A table of as many places as one may have, 2^31 - 256, its first and its last page alone there: what the same
    pages give side by side.  (All values of v lie in 1 .. 1.15.  Both results are off by the weights' and values'
    rounding to fp16, 2^-11 each, the scores' (below 2^-8 here) and the output's: less than 2^-6 together.)"""
    import torch
    page, width, D = 16 * 178481, 752, 64
    assert page * width == 0x7fffff00
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, (2, 1, page // 16, 18 * D), dtype=torch.uint8, device="cuda", generator=gen)
    for part, m in ((0, -0.075), (1, 1.0)):
        at = cache[..., part * 9 * D + 8 * D:(part + 1) * 9 * D]
        at.copy_(torch.tensor([0.01, m], dtype=torch.float16, device="cuda").view(torch.uint8).repeat(16))
    q = torch.randn(3, 4, D, device="cuda", generator=gen).half()
    start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = 0, 1
    far, near = torch.zeros_like(q), torch.zeros_like(q)
    qg.qg_attn_kv4(q, start, 3, cache, page, table, torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda"), 1.0, far)
    qg.qg_attn_kv4(q, start, 3, cache, page, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                   torch.tensor([2 * page], dtype=torch.int32, device="cuda"), 1.0, near)
    assert (near.float() - 1.075).abs().max() < 0.08
    assert (far.float() - near.float()).abs().max() <= 2 * 2.0 ** -6


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("nq", [1, 40])
def test_attention_with_a_hole_in_every_other_tile(qg, D, page, nq):
    """Pages that are not there all along long sequences: the ring's stages are zeroed in part and filled again, over
    and over."""
    c = attention_case(17, [2600, 1900], nq, 2, 4, D, page)
    c["table"][0, 3::128 * 2 // page] = -1
    c["table"][1, 1::128 * 3 // page] = 2 ** 30
    check_attention(qg, c)


# ---------------------------------------------------------------------------------------------
# Errors
# ---------------------------------------------------------------------------------------------
def test_a_launch_that_failed_leaves_no_error_behind(qg):
    """While some stream is captured in the global mode, nothing can be launched on the legacy stream: QG_ERR_CUDA.
    The next call, of the GEMVs' kind, launches and says so."""
    import torch
    rt = ctypes.CDLL("libcudart.so.12")
    x, y = torch.ones(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    h, out = x.half(), torch.zeros(2, 2, 64, device="cuda", dtype=torch.float16)
    cache = qg.kv4_cache(2, 16, 2, 64)
    slot, i32 = torch.arange(2, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    start, table = torch.arange(3, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    u = torch.zeros(2, device="cuda")
    ws = torch.empty(qg.qg_attn_kv4_workspace(2, 2, 64, 1), dtype=torch.uint8, device="cuda")
    src, dst = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    calls = [lambda: qg.qg_qk_norm_rope(x, None, None, None, 0.0, None, None, 0, y, None, stream=0),
             lambda: qg.qg_kv4_append(x, x, None, 0.0, None, None, 0, slot, cache, 16, stream=0),
             lambda: qg.qg_kv4_read(cache, 16, slot, x, y, stream=0),
             lambda: qg.qg_attn_kv4(h, start, 1, cache, 16, table, i32, 1.0, out, workspace=ws, stream=0),
             lambda: qg.qg_sample(x.view(2, 128), None, None, None, None, u, i32, stream=0)]
    for call in calls:
        call()  # what is set up once is
    qg.qg_hbm_copy(src, dst, 256)
    torch.cuda.synchronize()
    for call in calls:
        s = ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
        assert rt.cudaStreamBeginCapture(s, 0) == 0
        with pytest.raises(qg.QgError) as e:
            call()
        g = ctypes.c_void_p()
        rt.cudaStreamEndCapture(s, ctypes.byref(g))  # (invalidated: no graph)
        rt.cudaGetLastError()
        assert rt.cudaStreamDestroy(s) == 0
        assert e.value.status == qg.QG_ERR_CUDA
        dst.zero_()
        qg.qg_hbm_copy(src, dst, 256)
        assert torch.equal(src, dst)


def test_empty_tensors(qg):
    """No tokens, no rows, no sequences, no places: nothing is done, nothing is refused."""
    import torch
    x, h = torch.empty(0, 2, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda", dtype=torch.float16)
    i32, i64, f = (torch.empty(0, dtype=t, device="cuda") for t in (torch.int32, torch.int64, torch.float32))
    freq, w = dev(frequencies(32)), torch.ones(64, device="cuda")
    cache = qg.kv4_cache(2, 16, 2, 64).fill_(7)
    qg.qg_qk_norm_rope(x, x[:, :1], w, w, 1e-6, i32, freq, 0, h, h[:, :1])
    qg.qg_kv4_append(x, x, w, 1e-6, i32, freq, 0, i64, cache, 16)
    qg.qg_kv4_append(x, x, w, 1e-6, i32, freq, 0, i64, cache[:0], 16)
    qg.qg_kv4_read(cache, 16, i64, x, h)
    start, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    qg.qg_attn_kv4(h, start, 0, cache, 16, table, i32, 1.0, torch.empty_like(h))
    out = torch.full((3, 2, 64), 9.0, device="cuda", dtype=torch.float16)
    q = torch.ones_like(out)
    qg.qg_attn_kv4(q, start, 0, cache, 16, table, i32, 1.0, out)  # rows, but no sequences
    assert (out == 9).all()
    one = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    qg.qg_attn_kv4(q, one, 3, cache[:0], 16, torch.empty(1, 0, dtype=torch.int32, device="cuda"), one[1:], 1.0, out)  # no pages at all
    assert (out == 0).all()
    qg.qg_sample(torch.empty(0, 50, device="cuda"), f, i32, f, f, f, i32)
    torch.cuda.synchronize()
    assert (cache == 7).all()


# ---------------------------------------------------------------------------------------------
# The cache's scales
# ---------------------------------------------------------------------------------------------
def test_scales_are_rounded_to_fp32_and_then_to_fp16(qg):
    """A group whose least value is 1 + 2^-11 + 2^-40 (a rotation by 2^-41 makes it): as fp32 that is 1 + 2^-11, a tie
    of fp16 that goes to 1; one rounding would give 1 + 2^-10.  d likewise: fp16(fp32(range / 15))."""
    import torch
    D, page = 64, 16
    x = np.full((2, 1, D), 2.0, "f4")
    x[0, 0, 0] = 1 + 2.0 ** -11
    x[1, 0, 1], x[1, 0, 33] = 2 - 15 * (1 + 2.0 ** -11), -3.75   # a range of 15 (1 + 2^-11 + 2^-40), nearly
    freq = np.zeros(32)
    freq[:2] = 2.0 ** -41, 2.0 ** -38
    pos = np.array([-1, -1], np.int32)
    kk = ref.rope(x.astype(np.float64), pos, freq, 0)
    assert kk[0].min() == 1 + 2.0 ** -11 + 2.0 ** -40
    once = kk[0].min().astype(np.float16)
    code, d, m = ref.quantize(kk)
    assert m[0, 0, 0] == 1 and once == np.float16(1 + 2.0 ** -10)
    assert d[1, 0, 0] == 1 and ((kk[1].max() - kk[1].min()) / 15).astype(np.float16) == np.float16(1 + 2.0 ** -10)
    cache, slot = torch.zeros(1, 1, 1, 18 * D, dtype=torch.uint8, device="cuda"), torch.arange(2, device="cuda")
    qg.qg_kv4_append(dev(x), dev(x), None, 0.0, dev(pos), dev(freq), 0, slot, cache, page)
    want = np.zeros((1, 1, 1, 18 * D), np.uint8)
    ref.store(want, page, np.arange(2), 0, code, d, m)
    ref.store(want, page, np.arange(2), 1, *ref.quantize(x.astype(np.float64)))
    assert np.array_equal(cache.cpu().numpy(), want)


def test_attention_says_whether_it_gave_up(qg):
    """No wait has run out in the calls of these tests, with workspaces of their own or torch's, on any stream."""
    import torch
    c = attention_case(2, [3000, 50], [1, 2], 1, 4, 64, 16)
    run_attention(qg, c)
    assert qg.qg_attn_kv4_device_error() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run_attention(qg, c)
        assert qg.qg_attn_kv4_device_error() == 0
    assert qg.qg_attn_kv4_device_error(s) == 0


# ---------------------------------------------------------------------------------------------
# Many tokens: blocks of four, whose tables stand side by side
# ---------------------------------------------------------------------------------------------
def many(over):
    """A number of tokens from which on a block takes four (16 a multiprocessor), and `over` more."""
    import torch
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count + over


@pytest.mark.parametrize("over", [0, 1, 2, 3, 1731])  # whole blocks and a last one of one, two and three tokens
@pytest.mark.parametrize("D,Hq,Hk,R,pairing,norm,how,src,dst", [
    (64, 3, 2, 64, 0, True, "rows", "f2", "f2"), (64, 17, 0, 6, 1, True, "odd", "f4", "f4"), (128, 12, 3, 128, 0, True, "rows", "f4", "f2"),
    (128, 1, 1, 10, 0, False, "heads first", "f2", "f2"), (256, 9, 2, 64, 1, True, "rows", "f2", "f2"),
    (256, 1, 0, 0, 0, True, "rows", "f4", "f4"), (256, 2, 1, 20, 0, True, "gemv", "f4", "f2")])
def test_norm_rope_of_many_tokens(qg, over, D, Hq, Hk, R, pairing, norm, how, src, dst):
    decode.test_norm_rope(qg, D, many(over), Hq, Hk, R, pairing, norm, 250000, how, src, dst)


@pytest.mark.parametrize("over", [1, 3, 1731])
@pytest.mark.parametrize("D,H,page,R,pairing,norm,how,src", [
    (64, 5, 16, 64, 0, True, "rows", "f2"), (64, 1, 48, 2, 1, True, "odd", "f2"), (128, 2, 32, 10, 0, True, "rows", "f4"),
    (128, 3, 16, 0, 0, False, "rows", "f2"), (256, 1, 64, 64, 1, False, "heads first", "f4"), (256, 2, 16, 256, 0, True, "gemv", "f4")])
def test_append_and_read_of_many_tokens(qg, over, D, H, page, R, pairing, norm, how, src):
    decode.test_append_and_read(qg, D, many(over), H, page, R, pairing, norm, how, src)


def test_append_of_the_same_token_twice(qg):
    """Two tokens of one slot, the same values: the slot holds them, and nothing else is touched."""
    import torch
    x = torch.randn(1, 3, 128, device="cuda")
    slot = torch.tensor([37], device="cuda")
    one, two = qg.kv4_cache(4, 16, 3, 128).fill_(85), qg.kv4_cache(4, 16, 3, 128).fill_(85)
    qg.qg_kv4_append(x, -x, None, 0.0, None, None, 0, slot, one, 16)
    qg.qg_kv4_append(x.expand(9, 3, 128), -x.expand(9, 3, 128), None, 0.0, None, None, 0, slot.repeat(9), two, 16)
    assert torch.equal(one, two)


# ---------------------------------------------------------------------------------------------
# Attention told less than the truth
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("max_q", [0, 1, 2, 9, 33, 100_000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_with_any_max_q(qg, D, max_q):
    """How many query rows are worked through together is only a matter of time; items cut between CTAs among them."""
    for lens, nq, Hk, G in (([777, 33, 1300, 0], [1, 4, 3, 2], 2, 4), ([3000, 90], [37, 5], 1, 7)):
        c = attention_case(41, lens, nq, Hk, G, D, 32)
        c["max_q"] = max_q
        check_attention(qg, c)


def test_attention_leaves_rows_outside_of_falling_starts(qg):
    """Starts that fall or lie outside of 0 .. T: those sequences have no rows.  Rows of none stay, what lies around
    out stays, and so does the cache."""
    import torch
    c = attention_case(6, [64, 32, 40, 50], 2, 1, 2, 64, 32)
    c["start"] = np.array([3, 5, 2, -4, -1], np.int32)
    T = len(c["q"])
    wide = torch.full((T + 4, 2, 64), 9, dtype=torch.float16, device="cuda")
    cache = dev(c["cache"])
    qg.qg_attn_kv4(dev(c["q"]), dev(c["start"]), 2, cache, 32, dev(c["table"]), dev(c["lens"]), c["scale"], wide[2:-2])
    got = wide.cpu().numpy()
    assert (np.delete(got, [5, 6], 0) == 9).all() and np.array_equal(cache.cpu().numpy(), c["cache"])
    one = dict(c, start=np.array([3, 5], np.int32), table=c["table"][:1], lens=c["lens"][:1])
    want, bound = ref.attention(one["q"], one["start"], one["cache"], 32, one["table"], one["lens"], one["scale"], np.full(c["q"].shape, 9.0))
    assert (np.abs(got[2:-2].astype(np.float64) - want) <= bound).all()


# ---------------------------------------------------------------------------------------------
# The ends of the ranges
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("nseq,Hk,G,D", [(1000, 2, 1, 64), (2301, 1, 3, 128)])
def test_attention_of_more_sequences_than_a_block_has_threads(qg, nseq, Hk, G, D):
    """The line of tiles is added up over several rounds of the block; most sequences short, one long, some empty."""
    rng = np.random.default_rng(nseq)
    lens = rng.integers(0, 40, nseq)
    lens[nseq // 2], lens[-1] = 1500, 70
    check_attention(qg, attention_case(nseq, [int(n) for n in lens], list(rng.integers(0, 3, nseq)), Hk, G, D, 16, spare=1))


@pytest.mark.parametrize("Hk,G,D", [(1, 1024, 64), (1024, 1, 64), (2, 300, 128), (1, 129, 256)])
def test_attention_of_many_heads(qg, Hk, G, D):
    check_attention(qg, attention_case(G, [40, 150], [1, 2], Hk, G, D, 32))


def test_attention_with_large_pages_and_scales(qg):
    """Pages of 2048 places and of nine blocks; a scale of zero (the mean of what is seen), a negative and a large one.
    (The reference's bound takes the scale as positive: a negative one is that of -q with its opposite, since
    scale q . k = -scale (-q) . k and a sign costs no rounding.)"""
    c = attention_case(51, [3000, 5], [2, 1], 2, 3, 128, 2048)
    for scale in (0.0, -0.1, 3.0):
        got = run_attention(qg, dict(c, scale=scale)).cpu().numpy().astype(np.float64)
        want, bound = ref.attention(c["q"] if scale >= 0 else -c["q"], c["start"], c["cache"], 2048, c["table"], c["lens"], abs(scale),
                                    np.full(c["q"].shape, 9.0))
        assert (np.abs(got - want) <= bound).all()
    check_attention(qg, attention_case(52, [1000, 290, 144], [1, 3, 2], 1, 5, 64, 144))


@pytest.mark.parametrize("D,R,pairing", [(256, 256, 0), (256, 254, 0), (128, 128, 1), (64, 62, 1), (64, 2, 1)])
def test_norm_rope_of_whole_heads(qg, D, R, pairing):
    decode.test_norm_rope(qg, D, 19, 5, 2, R, pairing, True, 2 ** 31 - 20, "rows", "f2", "f2")
    decode.test_norm_rope(qg, D, 19, 5, 2, R, pairing, True, -2 ** 31, "gemv", "f4", "f2")


@pytest.mark.parametrize("pairing,R", [(0, 128), (0, 20), (1, 128)])
def test_norm_rope_in_place_in_one_projection(qg, pairing, R):
    """q and k side by side in one [T, (Hq + 2 Hk) D] array, each onto itself; v stays."""
    import torch
    T, Hq, Hk, D = 70, 6, 2, 128
    rng = np.random.default_rng(R)
    a = dev(rng.normal(size=(T, (Hq + 2 * Hk) * D)).astype("f2"))
    b = a.clone()
    part = lambda x, at, H: x[:, at * D:(at + H) * D].unflatten(1, (H, D))  # noqa: E731
    wq, wk = (dev(rng.uniform(0.5, 1.5, D).astype("f4")) for _ in range(2))
    pos, freq = dev(np.arange(T, dtype=np.int32)), dev(frequencies(R))
    q, k = torch.empty(T, Hq, D, dtype=torch.float16, device="cuda"), torch.empty(T, Hk, D, dtype=torch.float16, device="cuda")
    qg.qg_qk_norm_rope(part(a, 0, Hq), part(a, Hq, Hk), wq, wk, 1e-6, pos, freq, pairing, q, k)
    qg.qg_qk_norm_rope(part(b, 0, Hq), part(b, Hq, Hk), wq, wk, 1e-6, pos, freq, pairing, part(b, 0, Hq), part(b, Hq, Hk))
    assert torch.equal(part(b, 0, Hq), q) and torch.equal(part(b, Hq, Hk), k)
    assert torch.equal(part(b, Hq + Hk, Hk), part(a, Hq + Hk, Hk))


@pytest.mark.parametrize("major", ["row", "vocabulary"])
def test_sample_of_very_many_rows(qg, major):
    rng = np.random.default_rng(8)
    R, V = 70_001, 5
    x = rng.normal(size=(R, V)).astype("f4")
    u = rng.random(R).astype("f4")
    k = rng.integers(0, 4, R)
    got = run_sample(qg, x, k=k, u=u, major=major)
    at = np.concatenate([rng.integers(0, R, 500), [0, 65535, 65536, R - 1]])
    assert [got[i] for i in at] == [ref.sample(x[i], None, int(k[i]), None, None, u[i]) for i in at]


def test_sample_settings_at_their_ends(qg):
    """An infinite temperature (all equally likely), counts and shares at their ends, logits of one value, strides of zero."""
    import torch
    rng = np.random.default_rng(4)
    R, V = 8, 3001
    x = (rng.normal(size=(R, V)) * 3).astype("f4")
    x[:, ::5] = -np.inf
    u = rng.random(R)
    inf = np.full(R, np.inf)
    for kw in (dict(t=inf), dict(t=inf, p=np.full(R, 0.5)), dict(t=inf, k=np.full(R, 1700), p=np.full(R, 0.9)),
               dict(k=np.full(R, 2 ** 31 - 1)), dict(k=np.full(R, -2 ** 31)), dict(k=np.full(R, V)), dict(k=np.full(R, V - 1), p=np.full(R, 0.999)),
               dict(p=np.full(R, -1.0)), dict(p=np.full(R, 1e-45)), dict(mp=np.full(R, 1e-45)), dict(mp=np.full(R, -3.0))):
        decode.check_sample(qg, x, u=u, **kw)
    one, tok = dev(x[0]), torch.zeros(4, dtype=torch.int32, device="cuda")
    uu = dev(np.array([0.1, 0.3, 0.6, 0.99], "f4"))
    qg.qg_sample(one.expand(4, V), None, None, None, None, uu, tok)   # every row the same memory
    assert tok.tolist() == [ref.sample(x[0], None, None, None, None, v) for v in uu.cpu().numpy()]
    qg.qg_sample(dev(x[:4, :1]).expand(4, 100), None, None, None, None, uu, tok)   # every token the same logit
    assert tok.tolist() == [-1] * 4
    qg.qg_sample(dev(x[:4, 1:2]).expand(4, 100), None, None, None, None, uu, tok)
    assert tok.tolist() == [10, 30, 60, 99]
