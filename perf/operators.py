"""What is measured of the operators around the GEMVs of a decode step: the head norms with the
position rotation (qg_qk_norm_rope), the append to the paged 4-bit cache (qg_kv4_append, read back
with qg_kv4_read), the attention over that cache (qg_attn_kv4) and the sampling of a token from the
logits (qg_sample).

Each operator stands here in its plain form (elementary torch operations, `own` false) and as a
user's program calls the library (`own` true), on the same inputs.

Layout of the 4-bit cache.  uint8 [pages][H][page / 16][18 D]: a block holds 16 tokens of one head,
  [K codes 16 x D/2][K scales 16 x D/64 x (fp16 d, fp16 m)][V codes 16 x D/2][V scales ...].
A token's codes are D nibbles, the even dimension in the low one, as D/32 chunks of 16 bytes; chunk
c of token t is stored at place c ^ (s(t) & (D/32 - 1)), s(t) = (t & 2) | ((t ^ (t >> 2)) & 1) << 2.
A value is d * code + m with the (d, m) of its 64 dimensions.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the 48-query / 4-key head layer, q and k as the GEMVs leave them
        {"name": "norm-rope 1 token", "op": "norm_rope", "T": 1, "Hq": 48, "Hk": 4, "D": 256, "R": 64, "pairing": 0,
         "inputs": "gemv", "first": 70001},
        # a long prompt, token-major fp16 projections, whole heads rotated, an odd length
        {"name": "norm-rope 4099 tokens", "op": "norm_rope", "T": 4099, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "pairing": 0, "inputs": "f16", "first": 0},
        # sixteen sequences, one new token each, from the GEMVs
        {"name": "append 16 tokens", "op": "append", "T": 16, "H": 4, "D": 256, "R": 64, "pairing": 0, "inputs": "gemv",
         "norm": True, "page": 64, "pages": 256, "first": 3000, "dropped": 0.0},
        # a long prompt of one sequence, token-major, with places that are not to be written
        {"name": "append 6001 tokens", "op": "append", "T": 6001, "H": 8, "D": 128, "R": 128, "pairing": 1,
         "inputs": "f32", "norm": False, "page": 16, "pages": 512, "first": 17, "dropped": 0.05},
        # a short conversation, one new token: latency counts
        {"name": "attn 1 x 700", "op": "attn", "nseq": 1, "nq": 1, "ragged_q": False, "shortest": 700, "longest": 700,
         "Hk": 4, "G": 12, "D": 256, "page": 64},
        # a batch of sixteen conversations of very different lengths, one of them empty
        {"name": "attn 16 x 0-16k", "op": "attn", "nseq": 16, "nq": 1, "ragged_q": False, "shortest": 0,
         "longest": 16000, "Hk": 4, "G": 12, "D": 256, "page": 64},
        # one very long context
        {"name": "attn 1 x 200001", "op": "attn", "nseq": 1, "nq": 1, "ragged_q": False, "shortest": 200001,
         "longest": 200001, "Hk": 4, "G": 12, "D": 256, "page": 64},
        # many sequences on the smaller heads
        {"name": "attn 64 x 200-6k", "op": "attn", "nseq": 64, "nq": 1, "ragged_q": False, "shortest": 200,
         "longest": 6000, "Hk": 8, "G": 4, "D": 128, "page": 16},
        # speculative verify: up to five tokens of four sequences at once
        {"name": "attn verify 4 x 30k", "op": "attn", "nseq": 4, "nq": 5, "ragged_q": True, "shortest": 9000,
         "longest": 30000, "Hk": 4, "G": 12, "D": 256, "page": 64},
        # a chunk of a prompt over what the cache holds already
        {"name": "attn chunk 1000 of 7k", "op": "attn", "nseq": 1, "nq": 1000, "ragged_q": False, "shortest": 7003,
         "longest": 7003, "Hk": 4, "G": 12, "D": 256, "page": 64},
        # one conversation, the usual settings
        {"name": "sample 1 x 151936", "op": "sample", "rows": 1, "V": 151936, "major": "row", "kinds": "nucleus"},
        # sixteen columns as the output GEMV leaves them, each user with settings of their own
        {"name": "sample 16 x 248320", "op": "sample", "rows": 16, "V": 248320, "major": "vocabulary", "kinds": "mixed"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attn", "attn", "sample"])
    D = rng.choice([64, 128, 256])
    if op == "norm_rope":
        Hk = rng.choice([1, 2, 4, 8])
        T = _spread(rng, 1, 2200)
        inputs = rng.choice(["gemv", "f16", "f32"]) if T <= 16 else rng.choice(["f16", "f32"])
        return {"op": op, "T": T, "Hq": Hk * rng.choice([1, 4, 6, 7]), "Hk": Hk, "D": D, "R": rng.choice([D // 4, D // 2, D]),
                "pairing": rng.choice([0, 1]), "inputs": inputs, "first": rng.choice([0, 5, 4000, 250000])}
    if op == "append":
        T = _spread(rng, 1, 6000)
        page = rng.choice([16, 32, 64, 128])
        inputs = rng.choice(["gemv", "f16", "f32"]) if T <= 16 else rng.choice(["f16", "f32"])
        return {"op": op, "T": T, "H": rng.choice([1, 2, 4, 8]), "D": D, "R": rng.choice([0, D // 4, D]),
                "pairing": rng.choice([0, 1]), "inputs": inputs, "norm": rng.choice([True, False]), "page": page,
                "pages": (T + 700 + page - 1) // page, "first": rng.choice([0, 9, 5000, 250000]),
                "dropped": rng.choice([0.0, 0.1])}
    if op == "attn":
        nseq = _spread(rng, 1, 64)
        Hk = rng.choice([1, 2, 4, 8])
        longest = _spread(rng, 1, min(150000, 200_000_000 // (nseq * Hk * D)))
        nq = rng.choice([1, 1, 2, 4, 7, 16, _spread(rng, 17, 500)])
        longest = max(longest, nq)
        while nseq * nq > 1000 and nq > 1:
            nq //= 2
        if nq > 16:
            longest = min(longest, 7000)
        return {"op": op, "nseq": nseq, "nq": nq, "ragged_q": rng.choice([True, False]),
                "shortest": min(longest, rng.choice([0, 1, nq, longest // 3])), "longest": longest, "Hk": Hk,
                "G": rng.choice([1, 2, 4, 6, 12, 16] if Hk <= 4 else [1, 2, 4]), "D": D,
                "page": rng.choice([16, 32, 64, 128, 256])}
    rows = _spread(rng, 1, 16)
    return {"op": "sample", "rows": rows, "V": _spread(rng, 300, 248000), "major": rng.choice(["row", "vocabulary"]),
            "kinds": rng.choice(["plain", "greedy", "topk", "nucleus", "mixed"])}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _heads(g, T, H, D, inputs):
    """Projections [T, H, D]: contiguous fp16 or fp32, or a view of what a GEMV leaves, fp32 [H D][T]."""
    if inputs == "gemv":
        return torch.randn(H * D, T, device=DEV, generator=g).mul_(1.7).view(H, D, T).permute(2, 0, 1)
    x = torch.randn(T, H, D, device=DEV, generator=g).mul_(1.7)
    return x.half() if inputs == "f16" else x


def _frequencies(R, base=1e7):
    return torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64, device=DEV)


def _table(g, nseq, wide, pages):
    return torch.randperm(pages, device=DEV, generator=g)[: nseq * wide].to(torch.int32).view(nseq, wide)


def _cache(g, pages, H, page, D):
    """A filled cache: codes as a quantizer leaves normal values, d around a fifteenth of their range."""
    blocks = pages * H * (page // 16)
    out = torch.empty(blocks, 18 * D, dtype=torch.uint8, device=DEV)
    nib = [i for i, n in enumerate([1, 1, 2, 4, 6, 9, 12, 15, 15, 13, 10, 7, 4, 2, 1, 1]) for _ in range(n)]
    pairs = torch.tensor([nib[i % len(nib)] | nib[(i * 37 + 11) % len(nib)] << 4 for i in range(256)], dtype=torch.uint8, device=DEV)
    half = 9 * D
    for p in (0, 1):  # K, then V
        at = out[:, p * half:(p + 1) * half]
        step = 1 << 18
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            raw = torch.randint(0, 256, (n, 8 * D), device=DEV, generator=g, dtype=torch.uint8)
            at[b:b + n, : 8 * D] = pairs[raw.int()]
            d = torch.rand(n, D // 4, 1, device=DEV, generator=g).mul_(0.15).add_(0.25)
            m = d * torch.rand(n, D // 4, 1, device=DEV, generator=g).mul_(2.0).add_(-8.5)
            at[b:b + n, 8 * D:] = torch.cat([d, m], 2).half().view(torch.uint8).view(n, D)
    return out.view(pages, H, page // 16, 18 * D)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op, D = case["op"], case.get("D")
    if op == "norm_rope":
        T, Hq, Hk, R = case["T"], case["Hq"], case["Hk"], case["R"]
        s["q"], s["k"] = _heads(g, T, Hq, D, case["inputs"]), _heads(g, T, Hk, D, case["inputs"])
        s["wq"], s["wk"] = (torch.rand(D, device=DEV, generator=g) + 0.5 for _ in range(2))
        s["pos"] = torch.arange(T, device=DEV, dtype=torch.int32) + case["first"]
        s["freq"] = _frequencies(R)
        s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV)
        s["k_out"] = torch.zeros(T, Hk, D, dtype=torch.float16, device=DEV)
    elif op == "append":
        T, H, page, pages = case["T"], case["H"], case["page"], case["pages"]
        s["k"], s["v"] = _heads(g, T, H, D, case["inputs"]), _heads(g, T, H, D, case["inputs"])
        s["wk"] = torch.rand(D, device=DEV, generator=g) + 0.5 if case["norm"] else None
        s["pos"] = torch.arange(T, device=DEV, dtype=torch.int32) + case["first"]
        s["freq"] = _frequencies(case["R"]) if case["R"] else None
        if T <= 16:  # tokens of different sequences
            slot = torch.randperm(pages * page, device=DEV, generator=g)[:T]
        else:  # consecutive places of one sequence, through its pages
            at = torch.arange(T, device=DEV) + case["first"] % page
            slot = torch.randperm(pages, device=DEV, generator=g)[at // page % pages] * page + at % page
        gone = torch.rand(T, device=DEV, generator=g) < case["dropped"]
        s["slot"] = torch.where(gone, -1, slot)
        s["cache"] = torch.zeros(pages, H, page // 16, 18 * D, dtype=torch.uint8, device=DEV)
        s["k_out"] = torch.zeros(T, H, D, device=DEV)
        s["v_out"] = torch.zeros(T, H, D, device=DEV)
    elif op == "attn":
        nseq, nq, Hk, page = case["nseq"], case["nq"], case["Hk"], case["page"]
        lo, hi = case["shortest"], case["longest"]
        frac = torch.arange(nseq, device=DEV, dtype=torch.float64) / max(1, nseq - 1)
        lens = (hi - (hi - lo) * frac ** 0.5).round().to(torch.int64)
        lens = lens[torch.randperm(nseq, device=DEV, generator=g)]
        n = torch.full((nseq,), nq, device=DEV, dtype=torch.int64)
        if case["ragged_q"]:
            n = torch.randint(0, nq + 1, (nseq,), device=DEV, generator=g)
            n[0] = nq
        start = torch.zeros(nseq + 1, dtype=torch.int32, device=DEV)
        start[1:] = torch.cumsum(n, 0)
        wide = max(1, (hi + page - 1) // page)
        T = nseq * nq
        s["T"], s["len"], s["start"] = T, lens.to(torch.int32), start
        s["q"] = torch.randn(T, Hk * case["G"], D, device=DEV, generator=g).mul_(0.4).half()
        s["table"] = _table(g, nseq, wide, nseq * wide + 3)
        s["cache"] = _cache(g, nseq * wide + 3, Hk, page, D)
        s["out"] = torch.zeros(T, Hk * case["G"], D, dtype=torch.float16, device=DEV)
        s["scale"] = D ** -0.5
    else:
        R, V = case["rows"], case["V"]
        x = torch.randn(R, V, device=DEV, generator=g).mul_(2.0)
        x[torch.arange(R, device=DEV)[:, None], torch.randint(0, V, (R, 12), device=DEV, generator=g)] += \
            torch.rand(R, 12, device=DEV, generator=g) * 6 + 6
        s["logits"] = x if case["major"] == "row" else x.t().contiguous().t()
        kind = case["kinds"]
        row = torch.arange(R, device=DEV)
        t = torch.rand(R, device=DEV, generator=g) * 0.8 + 0.5
        k = torch.randint(1, 100, (R,), device=DEV, generator=g).to(torch.int32)
        p = torch.rand(R, device=DEV, generator=g) * 0.3 + 0.7
        mp = torch.rand(R, device=DEV, generator=g) * 0.1
        if kind == "mixed":  # every row with another set of filters, one greedy
            t[row % 8 == 5] = 0.0
            k[row % 2 == 1] = 0
            p[row % 4 >= 2] = 1.0
            mp[row % 3 != 0] = 0.0
        s["temperature"] = torch.zeros(R, device=DEV) if kind == "greedy" else t
        s["top_k"] = k if kind in ("topk", "mixed") else None
        s["top_p"] = p if kind in ("nucleus", "mixed") else None
        s["min_p"] = mp if kind == "mixed" else None
        s["u"] = torch.rand(R, device=DEV, generator=g)
        s["token"] = torch.zeros(R, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _rotated(x, pos, freq, pairing):
    """x [T, H, D] with its first R dimensions rotated by the angles pos * freq (in 64 bits)."""
    if freq is None:
        return x
    R = 2 * freq.numel()
    a = (pos.double()[:, None] * freq)[:, None, :]
    c, s = a.cos().to(x.dtype), a.sin().to(x.dtype)
    i = torch.arange(R // 2, device=x.device)
    first, second = (i, i + R // 2) if pairing == 0 else (2 * i, 2 * i + 1)
    u, v = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = u * c - v * s
    y[..., second] = v * c + u * s
    return y


def _normed(x, w, eps=1e-6):
    return x if w is None else x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.to(x.dtype)


def _places(D, device):
    """[16][D/32]: where chunk c of token t stands in a block."""
    t = torch.arange(16, device=device)[:, None]
    s = (t & 2) | ((t ^ (t >> 2)) & 1) << 2
    return torch.arange(D // 32, device=device)[None, :] ^ (s & (D // 32 - 1))


def _quantized(x):
    """x [T, H, D] in 64 bits -> codes, d, m of each group of 64."""
    T, H, D = x.shape
    x = x.view(T, H, D // 64, 64)
    lo, hi = x.amin(-1), x.amax(-1)
    d, m = ((hi - lo) / 15).half(), lo.half()
    y = (x - m.double()[..., None]) / d.double()[..., None]
    code = torch.where(d[..., None] == 0, 0.0, y).round().clamp(0, 15).to(torch.uint8)
    return code.view(T, H, D), d, m


def _store(cache, slot, page, part, x):
    """Writes the rows of x [T, H, D] to their slots: part 0 for K, 1 for V."""
    T, H, D = x.shape
    code, d, m = _quantized(x)
    pages = cache.shape[0]
    ok = (slot >= 0) & (slot < pages * page)
    slot, code, d, m = slot[ok], code[ok], d[ok], m[ok]
    pg, blk, t = slot // page, slot % page // 16, slot % 16
    h = torch.arange(H, device=x.device)
    chunks = (code[..., 0::2] | code[..., 1::2] << 4).view(-1, H, D // 32, 16)
    codes = torch.empty_like(chunks)
    codes.scatter_(2, _places(D, x.device)[t][:, None, :, None].expand(-1, H, -1, 16), chunks)
    at = cache.view(pages, H, page // 16, 18 * D)[..., part * 9 * D:(part + 1) * 9 * D]
    cols = t[:, None, None] * (D // 2) + torch.arange(D // 2, device=x.device)
    at[pg[:, None, None], h[None, :, None], blk[:, None, None], cols] = codes.view(-1, H, D // 2)
    scales = torch.stack([d, m], -1).view(torch.uint8).view(-1, H, D // 16)
    cols = 8 * D + t[:, None, None] * (D // 16) + torch.arange(D // 16, device=x.device)
    at[pg[:, None, None], h[None, :, None], blk[:, None, None], cols] = scales


def _unpacked(blocks, D, part):
    """Blocks [..., 18 D] -> values [..., 16, D] of K (part 0) or V (part 1), in 32 bits."""
    at = blocks[..., part * 9 * D:(part + 1) * 9 * D]
    lead = at.shape[:-1]
    codes = at[..., : 8 * D].reshape(*lead, 16, D // 32, 16)
    idx = _places(D, at.device)[..., None].expand(16, D // 32, 16)
    codes = codes.gather(-2, idx.expand(*lead, 16, D // 32, 16)).reshape(*lead, 16, D // 2)
    code = torch.stack([codes & 15, codes >> 4], -1).reshape(*lead, 16, D // 64, 64)
    dm = at[..., 8 * D:].contiguous().view(torch.float16).view(*lead, 16, D // 64, 2).float()
    return (code * dm[..., :1] + dm[..., 1:]).view(*lead, 16, D)


def _read(s, part):
    """The values at the slots, zero where there is none."""
    slot, page, D = s["slot"], s["page"], s["D"]
    ok = (slot >= 0) & (slot < s["cache"].shape[0] * page)
    at = torch.where(ok, slot, 0)
    vals = _unpacked(s["cache"][at // page, :, at % page // 16], D, part)
    vals = vals[torch.arange(slot.numel(), device=slot.device), :, at % 16]
    return torch.where(ok[:, None, None], vals, 0.0)


def _attn(s):
    D, page, nseq, nq, Hk, G = s["D"], s["page"], s["nseq"], s["nq"], s["Hk"], s["G"]
    L = s["table"].shape[1] * page
    blocks = s["cache"][s["table"].long()].permute(0, 2, 1, 3, 4)  # [nseq, H, pages of it, blocks, bytes]
    n = s["start"][1:] - s["start"][:-1]
    i = torch.arange(nq, device=n.device)
    row = (s["start"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][row].float().view(nseq, nq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(nseq, Hk, G * nq, D)
    k = _unpacked(blocks, D, 0).reshape(nseq, Hk, L, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(nseq, Hk, G, nq, L)
    del k
    last = s["len"][:, None] - n[:, None] + i  # the last place that a token sees
    seen = (torch.arange(L, device=n.device) <= last[..., None]) & (i < n[:, None])[..., None]
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = (x - torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _unpacked(blocks, D, 1).reshape(nseq, Hk, L, D)
    o = torch.matmul(x.view(nseq, Hk, G * nq, L), v).view(nseq, Hk, G, nq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(nseq, nq, Hk * G, D).half()
    valid = i < n[:, None]
    s["out"][row[valid]] = o[valid]
    return s["out"]


def _sample(s):
    x = s["logits"]
    R, V = x.shape
    ones = torch.ones(R, device=x.device)
    t = s["temperature"].double()[:, None]
    k = s["top_k"].long()[:, None] if s["top_k"] is not None else torch.zeros(R, 1, dtype=torch.int64, device=x.device)
    p = (s["top_p"] if s["top_p"] is not None else ones).double()[:, None]
    mp = (s["min_p"] if s["min_p"] is not None else ones * 0).double()[:, None]
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    z = xs.double() / torch.where(t > 0, t, 1.0)
    w = (z - z[:, :1]).exp()
    rank = torch.arange(V, device=x.device)
    keep = (rank < k) | (k <= 0)
    w = torch.where(keep, w, 0.0)
    total = w.sum(1, keepdim=True)
    before = torch.cumsum(w, 1) - w
    keep = keep & ((before < p * total) | (p >= 1)) & (w >= mp)
    keep[:, 0] = True
    keep = keep & ((t > 0) | (rank == 0))
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))  # in the vocabulary's order
    cum = torch.cumsum(w, 1)
    past = cum > s["u"].double()[:, None] * cum[:, -1:]
    s["token"].copy_(past.int().argmax(1))
    return s["token"]


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        import quant_dequant_gemv_q4_b200 as qg
        if op == "norm_rope":
            qg.qg_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], 1e-6, s["pos"], s["freq"], s["pairing"], s["q_out"], s["k_out"])
            return [s["q_out"], s["k_out"]]
        if op == "append":
            qg.qg_kv4_append(s["k"], s["v"], s["wk"], 1e-6, s["pos"], s["freq"], s["pairing"], s["slot"], s["cache"], s["page"])
            qg.qg_kv4_read(s["cache"], s["page"], s["slot"], s["k_out"], s["v_out"])
            return [s["k_out"], s["v_out"]]
        if op == "attn":
            qg.qg_attn_kv4(s["q"], s["start"], s["nq"], s["cache"], s["page"], s["table"], s["len"], s["scale"], s["out"])
            return s["out"]
        qg.qg_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"])
        return s["token"]
    if op == "norm_rope":
        for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
            out.copy_(_rotated(_normed(x.float(), w), s["pos"], s["freq"], s["pairing"]))
        return [s["q_out"], s["k_out"]]
    if op == "append":
        # in 64 bits: a code is decided by which side of a border the value lies on
        _store(s["cache"], s["slot"], s["page"], 0, _rotated(_normed(s["k"].double(), s["wk"]), s["pos"], s["freq"], s["pairing"]))
        _store(s["cache"], s["slot"], s["page"], 1, s["v"].double())
        s["k_out"].copy_(_read(s, 0))
        s["v_out"].copy_(_read(s, 1))
        return [s["k_out"], s["v_out"]]
    return _attn(s) if op == "attn" else _sample(s)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _attn_rows(case):
    """Tokens read of the cache and (query, place) pairs, from the lengths that prepare() makes (ragged
    query counts at their mean)."""
    nseq, lo, hi = case["nseq"], case["shortest"], case["longest"]
    lens = [round(hi - (hi - lo) * (i / max(1, nseq - 1)) ** 0.5) for i in range(nseq)]
    nq = case["nq"] if not case["ragged_q"] else max(1, (case["nq"] + case["nq"] * (nseq - 1) / 2) / nseq)
    pairs = sum(max(0.0, nq * L - nq * (nq - 1) / 2) for L in lens)
    return sum(lens), pairs, nseq * nq


def work(case):
    op, D = case["op"], case.get("D")
    if op == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": n * ((2 if case["inputs"] == "f16" else 4) + 2) + 4 * case["T"], "flops": 6 * n}
    if op == "append":  # the inputs, the 4.5-bit rows written and read back, the values read back
        n = 2 * case["T"] * case["H"] * D
        return {"bytes": n * ((2 if case["inputs"] == "f16" else 4) + 2 * 4.5 / 8 + 4) + 12 * case["T"], "flops": 12 * n}
    if op == "attn":
        places, pairs, T = _attn_rows(case)
        Hq = case["Hk"] * case["G"]
        return {"bytes": places * case["Hk"] * 2 * D * 4.5 / 8 + 4 * T * Hq * D, "flops": 4 * pairs * Hq * D}
    return {"bytes": case["rows"] * (case["V"] * 4 + 24), "flops": case["rows"] * case["V"]}


# ---------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def _spun(x, pos, freq, pairing):
    """The rotation as a complex product."""
    if freq is None:
        return x
    R = 2 * freq.numel()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), torch.outer(pos.double(), freq))[:, None]
    rot = x[..., :R]
    pairs = torch.stack(rot.split(R // 2, -1), -1) if pairing == 0 else rot.unflatten(-1, (R // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = torch.cat([y[..., 0], y[..., 1]], -1) if pairing == 0 else y.flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _unit(x, w, eps=1e-6):
    return x if w is None else x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + eps) * w.double()


def _held(x):
    """The values that 4 bits with d and m in fp16 for each 64 stand for."""
    y = x.unflatten(-1, (-1, 64))
    m = y.min(-1, keepdim=True).values
    d = ((y.max(-1, keepdim=True).values - m) / 15).half().double()
    m = m.half().double()
    code = torch.round((y - m) / torch.where(d > 0, d, 1.0)).clamp(0, 15)
    return (torch.where(d > 0, code, 0.0) * d + m).flatten(-2)


def _kv64(block, D, part, tokens):
    """Values [tokens, D] of consecutive blocks [n, 18 D] of one head, byte by byte."""
    at = block[:, part * 9 * D:(part + 1) * 9 * D]
    t = torch.arange(16, device=at.device)
    s = (t & 2) + 4 * ((t & 1) ^ ((t >> 2) & 1))
    dim = torch.arange(D, device=at.device)
    byte = t[:, None] * (D // 2) + ((dim // 32)[None] ^ (s & (D // 32 - 1))[:, None]) * 16 + dim % 32 // 2
    nib = (at[:, byte].long() >> (4 * (dim % 2))) & 15
    dm = at[:, 8 * D:].contiguous().view(torch.float16).double().view(-1, 16, D // 64, 2)
    return (nib * dm[..., 0].repeat_interleave(64, -1) + dm[..., 1].repeat_interleave(64, -1)).view(-1, D)[:tokens]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return [_spun(_unit(x.double(), w), s["pos"], s["freq"], case["pairing"]) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"]))]
    if op == "append":
        ok = (s["slot"] >= 0)[:, None, None]
        k = _spun(_unit(s["k"].double(), s["wk"]), s["pos"], s["freq"], case["pairing"])
        return [torch.where(ok, _held(x), 0.0) for x in (k, s["v"].double())]
    if op == "sample":
        return None  # a token, not a computed number
    D, G, page = case["D"], case["G"], case["page"]
    out = s["out"].double()
    start, lens = s["start"].tolist(), s["len"].tolist()
    for i in range(case["nseq"]):
        a, b, L = start[i], start[i + 1], lens[i]
        if a == b or L == 0:
            continue
        for h in range(case["Hk"]):
            blocks = s["cache"][s["table"][i].long(), h].flatten(0, 1)[: (L + 15) // 16]
            k, v = _kv64(blocks, D, 0, L), _kv64(blocks, D, 1, L)
            q = s["q"][a:b, h * G:(h + 1) * G].double()
            for c in range(0, b - a, 64):
                x = torch.einsum("tgd,ld->tgl", q[c:c + 64], k) * s["scale"]
                last = L - (b - a) + c + torch.arange(x.shape[0], device=x.device)
                hidden = torch.arange(L, device=x.device)[None] > last[:, None]
                x = x.masked_fill(hidden[:, None], -math.inf)
                y = torch.einsum("tgl,ld->tgd", torch.softmax(x, -1), v)
                out[a + c:a + c + x.shape[0], h * G:(h + 1) * G] = torch.where((last >= 0)[:, None, None], y, 0.0)
    return out
