"""The 8-bit paged KV cache's operators as measured cases: block tables and slot
maps, the quantising append, and attention over the cache's pages (all of a
request's pages, or the pages that the indexer picked for each row).

The cache of one layer is k, v (8-bit codes, float8_e4m3fn or int8)
[n_blocks][H][P][D] with fp32 scales [n_blocks][H]; the key at position i of
request b is row i % P of block page_table[b, i // P].
"""

import math

import torch

own = False  # True: run() makes the framework's calls; False: the plain forms

DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MIN_EXP = -100  # the smallest scale is 2^-100


# ------------------------------------------------------------------------ cases
def _tables(name, B, T, P, N, lo, hi, flo, fhi):
    return dict(name=name, op="tables", B=B, T=T, P=P, N=N, lo=lo, hi=hi, flo=flo, fhi=fhi, lens=1)


def _append(name, B, T, H, D, P, fmt, lo, hi, flo, fhi, n_blocks):
    return dict(name=name, op="append", B=B, T=T, H=H, D=D, P=P, fmt=fmt, lo=lo, hi=hi, flo=flo,
                fhi=fhi, n_blocks=n_blocks, lens=2)


def _attn(name, B, T, Q, H, D, P, K, fmt, lo, hi):
    return dict(name=name, op="attention", B=B, T=T, Q=Q, H=H, D=D, P=P, K=K, fmt=fmt, lo=lo,
                hi=hi, lens=3)


def listed():
    return [
        # one decode step of 256 requests, contexts of up to 65536 keys in pages of 64
        _tables("tables_decode", 256, 1, 64, 1025, 1, 65536, 1, 1),
        # a batch of prompts of up to 1024 tokens, small pages, some requests already started
        _tables("tables_prompt", 64, 1024, 16, 256, 0, 3000, 0, 1024),
        # one decode step: a token of each of 256 requests into partly filled pages
        _append("append_decode", 256, 1, 8, 128, 64, "e4m3", 1, 511, 1, 1, 4096),
        # prompts: 16384 tokens in pages of 64
        _append("append_prompt", 8, 2048, 8, 128, 64, "int8", 0, 0, 2048, 2048, 512),
        # ragged chunks, odd heads, pages of 24, a head dim that is no power of two
        _append("append_ragged", 5, 37, 3, 96, 24, "e4m3", 0, 90, 0, 37, 64),
        # one request, one kv head, 256 of 4096 pages: the indexer's single-request decode
        _attn("attn_pages_one", 1, 1, 4, 1, 128, 64, 256, "e4m3", 200000, 262144),
        # the decode batch: 32 requests, 256 selected pages of 64 keys each, 8 kv heads
        _attn("attn_pages_decode", 32, 1, 32, 8, 128, 64, 256, "e4m3", 4096, 32768),
        # four new tokens per request, each with its own page list
        _attn("attn_pages_tokens", 16, 4, 32, 8, 128, 64, 64, "int8", 2048, 16384),
        # dense decode of many short, ragged contexts in small pages
        _attn("attn_dense_ragged", 128, 1, 32, 4, 128, 16, 0, "int8", 1, 4096),
        # a 16-token chunk with 8 query heads per kv head over long contexts
        _attn("attn_dense_chunk", 4, 16, 64, 8, 128, 64, 0, "e4m3", 24000, 32768),
        # prompt chunks of 1024 tokens behind up to 7168 cached keys
        _attn("attn_dense_prompt", 2, 1024, 32, 8, 128, 64, 0, "e4m3", 1024, 8192),
        # small, odd everything: 3 tokens, 5 query heads per kv head, pages of 24, from empty caches on
        _attn("attn_dense_odd", 3, 3, 10, 2, 96, 24, 0, "int8", 0, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: sizes over their logarithms, odd ones among them."""
    most = [work(c) for c in listed()]
    top = (max(w["bytes"] for w in most), max(w["flops"] for w in most))
    while True:
        op = rng.choice(["tables", "append", "append", "attention", "attention", "attention"])
        P = rng.choice([16, 32, 64, 64, 128, 4, 7, 24, 48])
        fmt = rng.choice(["e4m3", "int8"])
        D = rng.choice([64, 128, 128, 256, 96, 48, 112])
        H = rng.choice([1, 2, 3, 4, 8])
        if op == "tables":
            B, T = _log(rng, 1, 512), rng.choice([1, 1, 2, 4, _log(rng, 5, 1024)])
            hi = _log(rng, 1, 65536)
            c = _tables("drawn", B, T, P, -(-(hi + T) // P), rng.randint(0, hi), hi, min(T, 1), T)
            if B * T > 65536 or B * c["N"] > (1 << 20):
                continue
        elif op == "append":
            B, T = _log(rng, 1, 256), rng.choice([1, 1, 3, _log(rng, 4, 2048)])
            if B * T > 16384:
                continue
            hi = rng.choice([0, P - 1, 3 * P + 1])
            need = B * (-(-(hi + T) // P))
            c = _append("drawn", B, T, H, D, P, fmt, 0, hi, rng.choice([0, T]), T, need + rng.randint(1, 64))
            if c["n_blocks"] * H * P * D > (1 << 28):
                continue
        else:
            G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            B, T = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4, 16, _log(rng, 3, 512)])
            K = rng.choice([0, 0, _log(rng, 4, 512)])
            hi = _log(rng, 16, 65536)
            if T > 16:
                K = 0
            lo = rng.choice([T, max(T, hi // 2), hi])
            if hi < lo or (K and hi < K * P):
                continue
            c = _attn("drawn", B, T, H * G, H, D, P, K, fmt, lo, hi)
            pages = -(-hi // P)
            if B * pages * H * P * D > (1 << 31):  # the pool
                continue
            gathered = B * (T * K if K else pages) * P * H
            if gathered * D > (1 << 31) or gathered * G * (1 if K else T) > (1 << 30):
                continue  # the plain form's fp32 keys and scores
        w = work(c)
        if w["bytes"] <= top[0] and w["flops"] <= top[1]:
            del c["name"]
            c["lens"] = rng.randint(4, 1 << 30)
            return c


def _lengths(c):
    """(cached, fresh) per request, from the case alone: lists of B numbers."""
    g = torch.Generator().manual_seed(c["lens"])
    B = c["B"]
    length = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g)
    if c["op"] == "attention":  # length: keys the last token of the chunk sees
        return length, torch.full((B,), c["T"])
    return length, torch.randint(c["flo"], c["fhi"] + 1, (B,), generator=g)


def _pages(n, P):
    return (n + P - 1) // P


def work(case):
    c = case
    B, T, P = c["B"], c["T"], c["P"]
    length, fresh = _lengths(c)
    if c["op"] == "tables":
        new = _pages(length + fresh, P) - _pages(length, P)
        # lengths in; new pages read from the list and written; three maps out
        return {"bytes": int(8 * B + 8 * new.sum() + 12 * B * T), "flops": 0}
    H, D = c["H"], c["D"]
    if c["op"] == "append":
        rows = int(fresh.sum())
        pages = int((_pages(length + fresh, P) - length // P)[fresh > 0].sum())
        # bf16 rows in, codes out, scales of the touched pages in and out
        return {"bytes": rows * H * D * (4 + 2) + 4 * B * T + 16 * pages * H, "flops": 2 * rows * H * D * 2}
    Q, K = c["Q"], c["K"]
    t = torch.arange(T)
    counts = (length[:, None] - (T - 1) + t).clamp(min=0)  # keys that each row sees
    if K:
        seen = counts.clamp(max=K * P)
        # each row has its own list: T lists of a request share pages by chance only
        keys = torch.minimum(seen.sum(1), length)
    else:
        seen, keys = counts, length
    keys, seen = int(keys.sum()), int(seen.sum())
    pages = -(-keys // P)
    b = keys * H * D * 2 + pages * (8 * H + 4) + 4 * B * T * (1 + K) + B * T * Q * (4 * D + 4)
    return {"bytes": b, "flops": 4 * D * Q * seen}


# ----------------------------------------------------------------------- inputs
def _pow2_scale(amax, fmt):
    """The least power of two s (at least 2^-100) with QMAX * s >= amax."""
    m, e = torch.frexp(amax)
    qm, qe = math.frexp(QMAX[fmt])
    e = (e - qe + (m > qm).to(torch.int32)).clamp(min=MIN_EXP)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP))
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """Values in units of the scale, rounded to the code's nearest (ties to even)."""
    x = x.clamp(-QMAX[fmt], QMAX[fmt])
    return (x if fmt == "e4m3" else x.round()).to(CODE[fmt])


def _pool(n, H, P, D, fmt, g):
    """A filled cache of n blocks: normal values whose spread differs by block and head."""
    codes = torch.empty((n, H, P, D), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, H), device=DEV)
    step = max(1, (1 << 27) // (H * P * D))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn((m, H, P, D), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((m, H, 1, 1), generator=g, device=DEV))
        s = _pow2_scale(x.abs().amax((2, 3)), fmt)
        scales[i:i + m] = s
        codes[i:i + m] = _encode(x / s[:, :, None, None], fmt).view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = case
    B, T, P = c["B"], c["T"], c["P"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    length, fresh = _lengths(c)
    s = dict(c)
    if own:
        from page_scoring_top_b200 import binding
        s["ctx"] = binding.Context(torch.device(DEV), max_rows=1, max_n=1, max_k=1)
    if c["op"] == "tables":
        N = c["N"]
        length = torch.minimum(length, N * P - fresh)
        used = int(_pages(length, P).sum())
        n_blocks = int(_pages(length + fresh, P).sum()) + 64
        ids = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
        have = _pages(length, P)
        table = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
        inside = torch.arange(N)[None] < have[:, None]
        table[inside.to(DEV)] = ids[:used]
        s.update(cached=length.to(DEV, torch.int32), fresh=fresh.to(DEV, torch.int32), table=table,
                 n_blocks=n_blocks, free=ids, head=torch.full((1,), used, dtype=torch.int32, device=DEV),
                 head_out=torch.zeros(1, dtype=torch.int32, device=DEV))
        for k in ("slots", "key_counts", "page_counts"):
            s[k] = torch.zeros((B, T), dtype=torch.int32, device=DEV)
        return s
    H, D, fmt = c["H"], c["D"], c["fmt"]
    if c["op"] == "append":
        n = c["n_blocks"]
        ids = torch.randperm(n, generator=g, device=DEV)
        t = torch.arange(T)[None]
        last = _pages(length + fresh, P)
        base = torch.cumsum(last, 0) - last  # each request has blocks of its own
        pos = length[:, None] + t
        slots = ids[((base[:, None] + pos // P).to(DEV)) % n] * P + (pos % P).to(DEV)
        slots = torch.where((t < fresh[:, None]).to(DEV), slots, torch.full_like(slots, -1))
        # one block more than the cache has: where the plain form writes padding rows
        for w in ("k", "v"):
            codes, scales = _pool(n + 1, H, P, D, fmt, g)
            s[w + "_buf"], s[w + "_scale_buf"] = codes.view(CODE[fmt]), scales
            s[w] = torch.randn((B * T, H, D), generator=g, device=DEV).to(torch.bfloat16)
        s["slots"] = slots.reshape(-1).to(torch.int32)
        return s
    Q, K = c["Q"], c["K"]
    pages = _pages(length, P)
    N = int(pages.max())
    n = int(pages.sum()) + 1
    ids = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((B, N), dtype=torch.int32, device=DEV)
    table[(torch.arange(N)[None] < pages[:, None]).to(DEV)] = ids[:n - 1]
    counts = (length[:, None] - (T - 1) + torch.arange(T)).clamp(min=0).to(DEV, torch.int32)
    for w in ("k", "v"):
        codes, s[w + "_scale"] = _pool(n, H, P, D, fmt, g)
        s[w + "_cache"] = codes.view(CODE[fmt])
    s["page_idx"] = None
    if K:  # as the indexer gives them: distinct pages by descending score, -1 behind the last
        score = torch.rand((B, T, N), generator=g, device=DEV)
        score.masked_fill_(torch.arange(N, device=DEV) >= _pages(counts, P)[..., None], -1.0)
        val, idx = score.topk(min(K, N), dim=2)
        idx = torch.where(val < 0, torch.full_like(idx, -1), idx).to(torch.int32)
        s["page_idx"] = torch.nn.functional.pad(idx, (0, K - idx.shape[2]), value=-1).reshape(B * T, K)
    s.update(table=table, key_counts=counts, scale=1.0 / math.sqrt(D),
             q=torch.randn((B, T, Q, D), generator=g, device=DEV).to(torch.bfloat16),
             out=torch.empty((B, T, Q, D), dtype=torch.bfloat16, device=DEV),
             lse=torch.empty((B, T, Q), device=DEV))
    return s


# ------------------------------------------------------------------ plain forms
def _plain_tables(s):
    P, T = s["P"], s["T"]
    table, free, head = s["table"].long(), s["free"].long(), s["head"].long()
    cached, fresh = s["cached"].long()[:, None], s["fresh"].long()[:, None]
    N, F = table.shape[1], free.numel()
    have, want = _pages(cached, P), _pages(cached + fresh, P)
    need = want - have
    start = head + torch.cumsum(need, 0) - need
    j = torch.arange(N, device=DEV)[None]
    src = start + j - have
    ids = torch.where(src < F, free[src.clamp(0, F - 1)], torch.full_like(src, -1))
    table = torch.where((j >= have) & (j < want), ids, table)
    t = torch.arange(T, device=DEV)[None]
    pos = cached + t
    block = table.gather(1, (pos // P).clamp(max=N - 1))
    ok = (t < fresh) & (block >= 0)
    slots = torch.where(ok, block * P + pos % P, torch.full_like(pos, -1))
    keys = torch.where(ok, pos + 1, torch.zeros_like(pos))
    head_out = (head + need.sum()).clamp(max=F)
    return [x.to(torch.int32) for x in (table, slots, keys, _pages(keys, P), head_out)]


def _plain_append_one(x, codes, scales, slots, first, P, fmt):
    """Writes rows x [R][H][D] into codes (one spare block at the end); slots [R] long, the
    spare block's for padding rows; first [B]: each request's first slot."""
    n, H = scales.shape
    x = x.float()
    page, off = slots // P, slots % P
    fits = torch.isfinite(x)
    amax = torch.where(fits, x, torch.zeros_like(x)).abs().amax(2)
    sc = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand_as(amax),
                                                  _pow2_scale(amax, fmt), "amax")
    begins = torch.full((n,), P, device=DEV).scatter_reduce_(0, page, off, "amin")
    sc = torch.where((begins > 0)[:, None], torch.maximum(sc, scales), sc)
    touched = begins < P
    sc = torch.where(touched[:, None], sc, scales)
    # rows already in the first page of each request, in units of the new scale
    fp, fo = first // P, first % P
    old = codes.view(torch.uint8)[fp].view(codes.dtype)
    re = old.float() * (scales[fp] / sc[fp])[:, :, None, None]
    re = _encode(re, fmt).view(torch.uint8)
    keep = (torch.arange(P, device=DEV) >= fo[:, None])[:, None, :, None]
    raw = codes.view(torch.uint8)
    raw[fp] = torch.where(keep, old.view(torch.uint8), re)
    raw[page, :, off] = _encode(x / sc[page][:, :, None], fmt).view(torch.uint8)
    scales.copy_(sc)


def _plain_append(s):
    P, n = s["P"], s["n_blocks"]
    slots = s["slots"].long()
    slots = torch.where(slots >= 0, slots, torch.full_like(slots, n * P))
    first = slots.view(s["B"], s["T"])[:, 0]
    for w in ("k", "v"):
        _plain_append_one(s[w], s[w + "_buf"], s[w + "_scale_buf"], slots, first, P, s["fmt"])
    return [s[w][:n] for w in ("k_buf", "v_buf", "k_scale_buf", "v_scale_buf")]


def _plain_attention(s):
    B, T, Q, H, D, P, K = (s[k] for k in ("B", "T", "Q", "H", "D", "P", "K"))
    G, N = Q // H, s["table"].shape[1]
    counts = s["key_counts"].long()
    if K:
        page = s["page_idx"].long().view(B, T, K)
    else:
        page = torch.arange(N, device=DEV).expand(B, 1, N)  # one list for all tokens
    L = page.shape[1]
    bi = torch.arange(B, device=DEV)[:, None, None]
    block = s["table"].long()[bi, page.clamp(min=0)]

    def gather(w):  # [B][L][H][keys][D], fp32
        codes, scale = s[w + "_cache"], s[w + "_scale"]
        x = codes.view(torch.uint8)[block].view(codes.dtype).float()
        x = x * scale[block][..., None, None]
        return x.permute(0, 1, 3, 2, 4, 5).reshape(B, L, H, -1, D)

    pos = (page[..., None] * P + torch.arange(P, device=DEV)).reshape(B, L, -1)
    there = (page >= 0).repeat_interleave(P, 2)
    ok = there & (pos < counts.view(B, T, 1))  # [B][T][keys]
    # rows that share a list side by side: [B][L][H][(T / L) * G][D]
    q = s["q"].float().view(B, L, T // L, H, G, D).transpose(2, 3).reshape(B, L, H, -1, D)
    sc = (q @ gather("k").transpose(-1, -2)) * s["scale"]
    sc = sc.view(B, L, H, T // L, G, -1).masked_fill(~ok.view(B, L, 1, T // L, 1, -1), -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, L, H, -1, p.shape[-1]) @ gather("v")).view(B, L, H, T // L, G, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l)).squeeze(-1)
    return [o.transpose(2, 3).reshape(B, T, Q, D).to(torch.bfloat16),
            lse.transpose(2, 3).reshape(B, T, Q)]


# -------------------------------------------------------------------------- run
def run(state):
    s = state
    if own:
        from page_scoring_top_b200 import binding
        if s["op"] == "tables":
            binding.kv_block_tables(s["ctx"], s["cached"], s["fresh"], s["P"], s["n_blocks"], s["table"],
                                    s["free"], s["head"], s["head_out"], s["slots"],
                                    s["key_counts"], s["page_counts"])
            return [s[k] for k in ("table", "slots", "key_counts", "page_counts", "head_out")]
        if s["op"] == "append":
            n = s["n_blocks"]
            kc, vc, ks, vs = (s[w][:n] for w in ("k_buf", "v_buf", "k_scale_buf", "v_scale_buf"))
            binding.kv_append(s["ctx"], s["k"], s["v"], s["slots"], kc, vc, ks, vs)
            return [kc, vc, ks, vs]
        binding.kv_attention(s["ctx"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                             s["table"], s["key_counts"], s["out"], lse=s["lse"],
                             page_idx=s["page_idx"], scale=s["scale"])
        return [s["out"], s["lse"]]
    if s["op"] == "tables":
        return _plain_tables(s)
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_attention(s)


# ------------------------------------------------------------------------ exact
def exact(case, seed):
    """Attention and append in 64 bits, request by request; tables are whole numbers (None)."""
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    P, H, D = c["P"], c["H"], c["D"]
    if c["op"] == "append":
        return _exact_append(s, c)
    B, T, Q, K = c["B"], c["T"], c["Q"], c["K"]
    if work(c)["flops"] > 4e11:
        return None
    out = torch.zeros((B, T, Q, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, Q), -math.inf, dtype=torch.float64, device=DEV)
    counts = s["key_counts"].tolist()
    for b in range(B):
        for t in range(T if K else 1):
            last = counts[b][t] if K else counts[b][T - 1]
            if last == 0:
                continue
            if K:
                pages = s["page_idx"][b * T + t]
                pages = pages[pages >= 0].long()
                rows, n_rows = slice(t, t + 1), 1
            else:
                pages = torch.arange(-(-last // P), device=DEV)
                rows, n_rows = slice(0, T), T
            ids = s["table"][b][pages].long()
            keep = (pages[:, None] * P + torch.arange(P, device=DEV)).reshape(-1)
            for h in range(H):
                k = s["k_cache"][ids, h] if c["fmt"] == "int8" else s["k_cache"].view(torch.uint8)[ids, h].view(CODE["e4m3"])
                v = s["v_cache"][ids, h] if c["fmt"] == "int8" else s["v_cache"].view(torch.uint8)[ids, h].view(CODE["e4m3"])
                k = (k.double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)
                v = (v.double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, D)
                heads = slice(h * (Q // H), (h + 1) * (Q // H))
                x = torch.einsum("tgd,nd->tgn", s["q"][b, rows, heads].double(), k) * s["scale"]
                hide = keep[None, :] >= s["key_counts"][b, rows].long()[:, None]
                x = x.masked_fill(hide[:, None, :], -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[..., None]).nan_to_num(0.0)
                out[b, rows, heads] = torch.einsum("tgn,nd->tgd", w, v)
                lse[b, rows, heads] = z
    return [out, lse]


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_append(s, c):
    """Codes before their rounding, in units of the new scale, and the scales."""
    P, n, B, T = c["P"], c["n_blocks"], c["B"], c["T"]
    slots = s["slots"].view(B, T).tolist()
    qmax = QMAX[c["fmt"]]
    result = {}
    for w in ("k", "v"):
        codes = s[w + "_buf"][:n].double()
        scale = s[w + "_scale_buf"][:n].double()
        x = s[w].double().view(B, T, c["H"], c["D"])
        for b in range(B):
            t = 0
            while t < T and slots[b][t] >= 0:
                page, row = divmod(slots[b][t], P)
                rows = min(P - row, sum(1 for i in slots[b][t:t + P - row] if i >= 0))
                part = x[b, t:t + rows]  # [rows][H][D]
                top = part.abs().amax((0, 2))
                exp = torch.log2((top / qmax).clamp(min=2.0 ** MIN_EXP)).floor().long() - 1
                for _ in range(3):  # up to the first power whose range holds every row
                    exp += _two_to(exp) * qmax < top
                new = _two_to(exp.clamp(min=MIN_EXP))
                if row:
                    new = torch.maximum(new, scale[page])
                    codes[page, :, :row] *= (scale[page] / new)[:, None, None]
                codes[page, :, row:row + rows] = (part / new[None, :, None]).transpose(0, 1)
                scale[page] = new
                t += rows
        result[w] = codes, scale
    codes = [result[w][0] if c["fmt"] == "e4m3" else None for w in ("k", "v")]
    return codes + [result[w][1] for w in ("k", "v")]
