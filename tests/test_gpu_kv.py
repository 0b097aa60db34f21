"""GPU parity of the 8-bit paged KV cache (kv_block_tables, kv_append,
kv_attention) with 64-bit plain forms: whole numbers and codes equal, attention
within the error its roundings allow (kv_reference.tolerance)."""

import numpy as np
import pytest

import kv_reference as ref
from page_scoring_top_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

POISON = 0x5A5A5A5A
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from page_scoring_top_b200 import binding
    c = binding.Context(0, max_rows=1, max_n=1, max_k=1)
    yield c
    c.close()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def status(ctx):
    from page_scoring_top_b200 import binding
    return binding.idx_get_status(ctx)[1]


def bf16(x):
    """x rounded to bf16, as float64 and as the device tensor."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


# --------------------------------------------------------------------- tables
def run_tables(ctx, cached, fresh, T, P, N, table, n_blocks, free, head, use_fresh=True):
    from page_scoring_top_b200 import binding
    B = len(cached)
    t = dev(table)
    out = [torch.full((B, T), POISON, dtype=torch.int32, device="cuda") for _ in range(3)]
    ho = torch.full((1,), POISON, dtype=torch.int32, device="cuda")
    binding.kv_block_tables(ctx, dev(np.int32(cached)), dev(np.int32(fresh)) if use_fresh else None, P,
                            n_blocks, t, dev(np.int32(free)), dev(np.int32([head])), ho, *out)
    return [t.cpu().numpy()] + [o.cpu().numpy() for o in out] + [int(ho.item())]


def table_case(seed, B, T, P, cached_hi, fresh_lo):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, cached_hi + 1, B)
    fresh = rng.integers(fresh_lo, T + 1, B)
    have, want = -(-cached // P), -(-(cached + fresh) // P)
    N = int(max(want.max(), 1)) + 1
    n_blocks = int(want.sum()) + 5
    ids = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((B, N), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    return cached, fresh, N, table, n_blocks, ids, at


@pytest.mark.parametrize("B,T,P,hi,lo", [
    (1, 1, 64, 0, 1), (1, 1, 1, 5, 1), (3, 4, 16, 70, 0), (257, 1, 64, 1000, 0), (300, 4, 7, 50, 0),
    (1000, 2, 4, 9, 0), (2, 1500, 16, 33, 0), (1, 5000, 64, 100, 5000), (5, 1025, 3, 10, 1000),
    (4, 37, 128, 1, 0)])
def test_tables(ctx, B, T, P, hi, lo):
    cached, fresh, N, table, n_blocks, ids, head = table_case(B + T, B, T, P, hi, lo)
    got = run_tables(ctx, cached, fresh, T, P, N, table, n_blocks, ids, head)
    want = ref.block_tables(cached, fresh, T, P, N, table, n_blocks, ids, head)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert status(ctx) == 0


def test_tables_without_fresh_counts_or_head(ctx):
    cached, _, N, table, n_blocks, ids, head = table_case(9, 6, 3, 8, 30, 3)
    free = ids[head:]
    got = run_tables(ctx, cached, None, 3, 8, N, table, n_blocks, free, 0, use_fresh=False)
    want = ref.block_tables(cached, np.full(6, 3), 3, 8, N, table, n_blocks, free, 0)
    assert all(np.array_equal(g, w) for g, w in zip(got, want)) and status(ctx) == 0


def test_tables_free_list_ends(ctx):
    cached, fresh, N, table, n_blocks, ids, head = table_case(10, 40, 20, 4, 0, 20)
    free = ids[:head + 77]
    got = run_tables(ctx, cached, fresh, 20, 4, N, table, n_blocks, free, head)
    want = ref.block_tables(cached, fresh, 20, 4, N, table, n_blocks, free, head)
    assert all(np.array_equal(g, w) for g, w in zip(got, want))
    assert (got[1] == -1).any() and got[4] == len(free) and status(ctx) == 8


def test_tables_bad_values_are_reported(ctx):
    # counts outside the table are clamped, block ids outside the pool leave no slot
    table = np.array([[0, -1, -1], [9, -1, -1], [1, 2, 3]], np.int32)
    got = run_tables(ctx, [-4, 2, 99], [2, 5, 5], 2, 4, 3, table, 5, [4, 77], 0)
    want = ref.block_tables([0, 2, 12], [2, 2, 0], 2, 4, 3, table, 5, [4, 77], 0)
    assert all(np.array_equal(g, w) for g, w in zip(got, want))
    assert got[0][0, 0] == 4 and got[1].tolist() == [[16, 17], [-1, -1], [-1, -1]]
    assert status(ctx) == 1 | 4
    got = run_tables(ctx, [0], [1], 1, 4, 1, np.array([[3]], np.int32), 5, [2, 1], -3)
    assert got[1].tolist() == [[8]] and got[4] == 1 and status(ctx) == 1


# --------------------------------------------------------------------- append
def random_cache(rng, n, H, P, D, fmt, nan=False):
    codes = rng.integers(0, 256, (n, H, P, D)).astype(np.uint8)
    if fmt == "e4m3" and not nan:
        codes[(codes & 127) == 127] ^= 64
    if fmt == "int8":
        codes[codes == 128] = 129  # -127 is the least code
    return codes, (2.0 ** rng.integers(-8, 3, (n, H))).astype(np.float32)


def run_append(ctx, kx, vx, slots, kc, vc, ks, vs, fmt):
    from page_scoring_top_b200 import binding
    t = [dev(kc).view(CODE[fmt]), dev(vc).view(CODE[fmt]), dev(ks), dev(vs)]
    binding.kv_append(ctx, kx, vx, dev(np.int32(slots)), *t)
    return [t[0].view(torch.uint8).cpu().numpy(), t[1].view(torch.uint8).cpu().numpy(),
            t[2].cpu().numpy(), t[3].cpu().numpy()]


def check_append(ctx, seed, slots, n, H, P, D, fmt, spread=1.0, edit=None):
    rng = np.random.default_rng(seed)
    R = len(slots)
    kc, ks = random_cache(rng, n, H, P, D, fmt, nan=True)
    vc, vs = random_cache(rng, n, H, P, D, fmt, nan=True)
    x = rng.standard_normal((2, R, H, D)) * np.exp(spread * rng.standard_normal((2, R, H, 1)))
    if edit:
        edit(x)
    (k64, kx), (v64, vx) = bf16(x[0]), bf16(x[1])
    got = run_append(ctx, kx, vx, slots, kc, vc, ks, vs, fmt)
    for c, s, c0, s0, x64 in ((got[0], got[2], kc, ks, k64), (got[1], got[3], vc, vs, v64)):
        wc, ws = ref.append(x64, slots, c0, s0, fmt)
        assert np.array_equal(s, ws)
        assert np.array_equal(c, wc)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H,P,D", [(1, 16, 64), (2, 64, 128), (3, 7, 96), (2, 1, 16), (1, 130, 256), (2, 24, 48)])
def test_append_runs(ctx, fmt, H, P, D):
    # whole pages, starts inside a page, single rows, padding between and at the ends
    runs = [[-1], range(0, 2 * P), [-1, -1], range(3 * P + P // 2, 4 * P), [5 * P + P - 1], [6 * P],
            range(8 * P + P // 3, 9 * P + P // 2), [-1]]
    slots = [s for r in runs for s in r]
    check_append(ctx, H + P + D, slots, 10, H, P, D, fmt)
    assert status(ctx) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_many_rows(ctx, fmt):
    # enough rows for the windowed grid: runs that cross its windows
    P, rng = 24, np.random.default_rng(3)
    slots, at = [], 0
    while len(slots) < 3000:
        start = at * P + rng.integers(0, P)
        slots += list(range(start, start + rng.integers(1, 90)))
        at = slots[-1] // P + 1
        slots += [-1] * rng.integers(0, 3)
    check_append(ctx, 4, slots, at + 1, 4, P, 64, fmt)
    assert status(ctx) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_special_values(ctx, fmt):
    def edit(x):
        x[:, 0] = 0.0                   # a row of zeros: the smallest scale
        x[:, 1, 0, :3] = np.nan, np.inf, -np.inf
        x[:, 2] = np.inf                # nothing finite
        x[:, 3] = 3e38                  # near bf16's end
        x[:, 4] = 1e-38
        x[:, 5, 0, 0] = -0.0
        x[:, 6] = 448 if fmt == "e4m3" else 127   # exactly the range's end
        x[:, 7] = 450 if fmt == "e4m3" else 127.5
    check_append(ctx, 5, [3, 7, 8, 13, 16, 21, 24, 28], 8, 2, 4, 32, fmt, edit=edit)
    assert status(ctx) == 0


def test_append_bad_slots_are_skipped_and_reported(ctx):
    check_append(ctx, 6, [5, 64, -2, 10, 2 ** 31 - 1, -2 ** 31], 16, 1, 4, 64, "int8")
    assert status(ctx) == 4


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_token_by_token_equals_at_once(ctx, fmt):
    # powers of two: e4m3 codes do not depend on how the tokens were cut into
    # calls while none falls below the code's normal range
    rng = np.random.default_rng(7)
    n, H, P, D, R = 3, 2, 16, 64, 40
    x = np.sign(rng.standard_normal((R, H, D))) * rng.uniform(1, 8, (R, H, D)) * np.linspace(1, 16, R)[:, None, None]
    _, xt = bf16(x)
    kc, ks = random_cache(rng, n, H, P, D, fmt)
    once = run_append(ctx, xt, xt, range(R), kc, kc, ks, ks, fmt)
    c = [dev(kc).view(CODE[fmt]), dev(kc).view(CODE[fmt]), dev(ks), dev(ks)]
    from page_scoring_top_b200 import binding
    for r in range(R):
        binding.kv_append(ctx, xt[r:r + 1], xt[r:r + 1], dev(np.int32([r])), *c)
    assert np.array_equal(c[2].cpu().numpy(), once[2])
    got, want = c[0].view(torch.uint8).cpu().numpy(), once[0]
    if fmt == "e4m3":
        assert np.array_equal(got, want)
    else:  # int8 codes halve as the scale doubles: at most one step off
        assert np.abs(got.view(np.int8).astype(int) - want.view(np.int8)).max() <= 1


def test_append_scale_of_another_producer(ctx):
    # an old scale that is no power of two stays while it is large enough
    rng = np.random.default_rng(8)
    kc, ks = random_cache(rng, 2, 1, 8, 32, "int8")
    ks[:] = 0.3
    x64, x = bf16(rng.standard_normal((3, 1, 32)))
    got = run_append(ctx, x, x, [4, 5, 6], kc, kc, ks, ks, "int8")
    wc, ws = ref.append(x64, [4, 5, 6], kc, ks, "int8")
    assert np.array_equal(got[0], wc) and np.array_equal(got[2], ws) and got[2][0, 0] == np.float32(0.3)


def test_append_takes_rows_out_of_a_wider_tensor(ctx):
    rng = np.random.default_rng(9)
    H, D, P = 2, 64, 8
    kc, ks = random_cache(rng, 4, H, P, D, "int8")
    x64, x = bf16(rng.standard_normal((10, 3 * H, D)))
    got = run_append(ctx, x[:, H:2 * H], x[:, 2 * H:], range(10), kc, kc, ks, ks, "int8")
    for i, part in ((0, x64[:, H:2 * H]), (1, x64[:, 2 * H:])):
        wc, ws = ref.append(part, range(10), kc, ks, "int8")
        assert np.array_equal(got[i], wc) and np.array_equal(got[2 + i], ws)


# ------------------------------------------------------------------ attention
def attn_case(seed, B, T, Q, H, D, P, N, fmt, counts, K=0, n_extra=3, poison=True, vexp=3):
    rng = np.random.default_rng(seed)
    n = B * N + n_extra
    kc, ks = random_cache(rng, n, H, P, D, fmt)
    vc, vs = random_cache(rng, n, H, P, D, fmt)
    # scores of a few units: codes are up to 448 or 127
    ks = (ks * 2.0 ** (-6 if fmt == "e4m3" else -5)).astype(np.float32)
    vs = (2.0 ** rng.integers(-vexp, vexp + 1, vs.shape)).astype(np.float32)
    table = rng.permutation(n)[:B * N].reshape(B, N).astype(np.int32)
    counts = np.asarray(counts, np.int32).reshape(B, T)
    if poison:  # rows that no token sees hold NaN codes (or the largest) under NaN scales
        for b in range(B):
            c = int(counts[b].max())
            for p in range(N):
                seen = min(max(c - p * P, 0), P)
                kc[table[b, p], :, seen:] = 127
                vc[table[b, p], :, seen:] = 127
                if seen == 0:
                    ks[table[b, p]] = np.nan
                    vs[table[b, p]] = np.nan
    page_idx = None
    if K:
        page_idx = np.full((B * T, K), -1, np.int32)
        for r in range(B * T):
            m = min(K, N)
            page_idx[r, :m] = rng.permutation(N)[:m]
    q64, q = bf16(rng.standard_normal((B, T, Q, D)))
    return dict(q64=q64, q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, counts=counts,
                page_idx=page_idx, scale=D ** -0.5, fmt=fmt)


def launch_attn(ctx, c, out=None, lse=None, stream=None, t=None):
    from page_scoring_top_b200 import binding
    B, T, Q, D = c["q64"].shape
    if out is None:
        out = torch.full((B, T, Q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, T, Q), float("nan"), device="cuda")
    t = t or upload(c)
    binding.kv_attention(ctx, c["q"], *t[:4], t[4], t[5], out, lse=lse, page_idx=t[6], scale=c["scale"],
                         stream=stream)
    return out, lse


def upload(c):
    return [dev(c["kc"]).view(CODE[c["fmt"]]), dev(c["vc"]).view(CODE[c["fmt"]]), dev(c["ks"]),
            dev(c["vs"]), dev(c["table"]), dev(c["counts"]),
            None if c["page_idx"] is None else dev(c["page_idx"])]


def check_attn(ctx, c, bits=0):
    out, lse = launch_attn(ctx, c)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    o, l, A, ds, top = ref.attention(c["q64"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["counts"],
                                     c["page_idx"], c["scale"], c["fmt"])
    keys = c["table"].shape[1] * c["kc"].shape[2] * (1 if c["page_idx"] is None else 2)
    tol = ref.tolerance(o, A, ds, top, keys)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), "%d of %d outside, worst %.3g of the bound" % (
        bad.sum(), bad.size, np.nanmax(np.abs(got - o) / tol))
    empty = np.isneginf(l)
    assert np.array_equal(empty, np.isneginf(gl))
    assert (got[empty] == 0).all()
    ltol = ds[..., 0] * 2 + 2.0 ** -22 * (np.abs(np.where(empty, 0, l)) + 4) + 2.0 ** -23 * (keys + 64)
    assert (np.abs(gl[~empty] - l[~empty]) <= ltol[~empty]).all()
    assert status(ctx) == bits


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [16, 48, 64, 96, 128, 192, 256])
def test_attention_dense_head_dims(ctx, fmt, D):
    counts = [[200], [1], [0], [64], [127]]
    check_attn(ctx, attn_case(D, 5, 1, 8, 2, D, 64, 4, fmt, counts))


@pytest.mark.parametrize("P", [1, 2, 4, 7, 8, 16, 24, 31, 32, 33, 48, 64, 100, 128, 256])
def test_attention_dense_page_sizes(ctx, P):
    N = -(-520 // P)
    counts = [[N * P], [P], [min(P + 1, N * P)], [3], [N * P - 1]]
    check_attn(ctx, attn_case(P, 5, 1, 4, 1, 64, P, N, "e4m3" if P % 2 else "int8", counts))


@pytest.mark.parametrize("Q,H", [(1, 1), (3, 3), (2, 1), (10, 2), (14, 2), (16, 1), (17, 1), (24, 1), (32, 1),
                                 (48, 1), (64, 1), (65, 1), (128, 1), (130, 1), (40, 8)])
def test_attention_head_layouts(ctx, Q, H):
    check_attn(ctx, attn_case(Q + H, 2, 1, Q, H, 128, 16, 9, "e4m3", [[131], [144]]))


@pytest.mark.parametrize("T,Q,H", [(2, 4, 1), (3, 10, 2), (4, 8, 2), (5, 3, 1), (16, 8, 1), (17, 16, 2), (33, 4, 2),
                                   (70, 2, 2), (9, 40, 1), (130, 1, 1)])
def test_attention_causal_tokens(ctx, T, Q, H):
    # token t sees pos0 + t + 1 keys; the last request is padded behind two tokens
    pos0 = np.array([0, 100, 37])
    counts = pos0[:, None] + np.arange(T) + 1
    counts[2, 2:] = 0
    N = -(-int(counts.max()) // 16)
    check_attn(ctx, attn_case(T + Q, 3, T, Q, H, 128, 16, N, "e4m3", counts))


@pytest.mark.parametrize("Q,P", [(16, 16), (12, 4), (4, 16), (16, 64), (40, 8)])
def test_attention_many_short_items_wide_heads(ctx, Q, P):
    # the ring of stages at its smallest beside the groups of warps, and items
    # that end within it: groups wait for one another while they hold stages
    rng = np.random.default_rng(Q + P)
    counts = rng.integers(1, 700, (90, 1))
    check_attn(ctx, attn_case(Q + P, 90, 1, Q * 2, 2, 256, P, -(-700 // P), "int8", counts))


@pytest.mark.parametrize("B,T,Q,H,D,P,pos0,fmt", [
    (1, 17, 4, 1, 64, 32, 0, "int8"), (1, 33, 4, 1, 128, 64, 0, "e4m3"), (2, 40, 8, 2, 128, 64, 900, "e4m3"),
    (2, 40, 8, 2, 128, 64, 900, "int8"), (1, 130, 4, 1, 64, 128, 257, "e4m3"), (1, 9, 16, 2, 128, 256, 1000, "int8"),
    (3, 20, 16, 2, 96, 48, 70, "e4m3"), (1, 33, 8, 1, 112, 7, 50, "int8"), (2, 70, 2, 1, 48, 100, 333, "e4m3"),
    (1, 20, 256, 1, 128, 32, 90, "e4m3"), (1, 3, 130, 1, 64, 16, 40, "int8"), (1, 16, 8, 1, 128, 1, 30, "e4m3"),
    (1, 70, 1, 1, 64, 7, 30, "e4m3"), (1, 16, 8, 1, 128, 64, 30000, "e4m3")])
def test_attention_prompts(ctx, B, T, Q, H, D, P, pos0, fmt):
    # more than 64 rows (tokens x heads) to a kv head; the last request starts empty
    counts = np.arange(T)[None] + 1 + np.array([pos0] * (B - 1) + [pos0 if B == 1 else 0])[:, None]
    N = -(-int(counts.max()) // P)
    check_attn(ctx, attn_case(T + D + P, B, T, Q, H, D, P, N, fmt, counts))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_prompt_many_tiles_per_sm(ctx, D):
    counts = np.array([32000, 31000, 32000, 777, 29000, 31999])[:, None] - 15 + np.arange(16)
    check_attn(ctx, attn_case(28, 6, 16, 8, 1, D, 64, 500, "e4m3", counts))


def test_attention_prompt_many_items_per_sm(ctx):
    rng = np.random.default_rng(29)
    counts = rng.integers(0, 300, (200, 1)) + np.arange(17)[None]
    counts[::7] = 0
    check_attn(ctx, attn_case(29, 200, 17, 4, 1, 64, 32, 10, "int8", counts))


def test_attention_prompt_padding_and_scales(ctx):
    # padded tokens between real ones, a negative softmax scale, value scales far
    # apart (as in test_attention_scales_far_apart), a block outside the pool
    rng = np.random.default_rng(30)
    counts = np.where(rng.random((2, 40)) < 0.3, 0, rng.integers(1, 600, (2, 40)))
    c = attn_case(30, 2, 40, 4, 1, 128, 64, 10, "e4m3", counts, vexp=30)
    check_attn(ctx, c)
    c["scale"] = -c["scale"]
    check_attn(ctx, c)
    c = attn_case(31, 1, 40, 4, 1, 64, 32, 10, "int8", 280 + np.arange(40)[None], poison=False)
    c["table"][0, 3] = -1
    c["table"][0, 6] = 99999
    check_attn(ctx, c, bits=4)


def test_attention_counts_in_any_order(ctx):
    # key counts are data: neither rising nor equal over a request's tokens
    rng = np.random.default_rng(2)
    for T, Q, H in ((6, 4, 2), (40, 8, 1)):
        check_attn(ctx, attn_case(T, 4, T, Q, H, 64, 32, 8, "int8", rng.integers(0, 257, (4, T))))


@pytest.mark.parametrize("D,H,Q", [(128, 1, 4), (64, 2, 16), (256, 1, 2), (96, 2, 6)])
@pytest.mark.parametrize("P,K", [(64, 7), (16, 40), (4, 33), (24, 5), (128, 1)])
def test_attention_selected_pages(ctx, D, H, Q, P, K):
    N = K + 9
    counts = [[N * P], [N * P // 2 + 1], [0], [P // 2 + 1]]
    check_attn(ctx, attn_case(P + K + D, 4, 1, Q, H, D, P, N, "e4m3" if K % 2 else "int8", counts, K=K))


def test_attention_selected_pages_per_token(ctx):
    counts = np.array([[300, 301, 302], [5, 6, 0]])
    check_attn(ctx, attn_case(1, 2, 3, 8, 2, 128, 16, 19, "int8", counts, K=12))


def test_attention_long_rows_few(ctx):
    # one row spread over the whole GPU, and rows of very unequal length beside it
    check_attn(ctx, attn_case(11, 1, 1, 8, 2, 64, 64, 300, "e4m3", [[300 * 64 - 5]]))
    check_attn(ctx, attn_case(12, 6, 1, 4, 1, 64, 16, 600, "int8", [[9600], [1], [0], [31], [5000], [33]]))


@pytest.mark.parametrize("D,K", [(16, 0), (128, 0), (128, 900)])
def test_attention_many_units_per_sm(ctx, D, K):
    # hundreds of 32-key units on every SM: the ring of stages goes round many times
    N = 960
    check_attn(ctx, attn_case(27, 10, 1, 1, 1, D, 64, N, "e4m3", [[N * 64 - 9 * b] for b in range(10)], K=K))


def test_attention_many_short_rows(ctx):
    rng = np.random.default_rng(13)
    check_attn(ctx, attn_case(13, 700, 1, 2, 1, 16, 8, 3, "e4m3", rng.integers(0, 25, (700, 1))))


def test_attention_page_listed_twice_counts_twice(ctx):
    c = attn_case(14, 1, 1, 4, 1, 64, 16, 6, "int8", [[90]], K=5)
    c["page_idx"][0] = [3, 1, 3, -1, 5]
    check_attn(ctx, c)


def test_attention_nothing_selected(ctx):
    c = attn_case(15, 2, 1, 4, 1, 64, 16, 6, "e4m3", [[90], [20]], K=3)
    c["page_idx"][0] = -1
    c["page_idx"][1] = [4, 5, -1]  # pages past the request's keys
    check_attn(ctx, c)


def test_attention_scales_far_apart(ctx):
    # pages whose value scales differ by 2^60: the far smaller ones still carry
    # the output where the weights are theirs
    c = attn_case(16, 3, 1, 4, 1, 64, 16, 8, "e4m3", [[128], [100], [33]], vexp=30)
    c["ks"] *= 4
    check_attn(ctx, c)
    c["vs"][:] = np.float32(2.0 ** -90)
    check_attn(ctx, c)


def test_attention_zero_scales_and_scores(ctx):
    c = attn_case(17, 2, 1, 4, 1, 64, 16, 4, "int8", [[60], [64]], poison=False)
    c["vs"][c["table"][0]] = 0.0  # the first request's values are all zero
    c["ks"][c["table"][1, 1]] = 0.0
    check_attn(ctx, c)


def test_attention_large_and_tiny_queries(ctx):
    for f in (1e30, 1e-30):
        c = attn_case(18, 2, 1, 4, 2, 128, 16, 4, "e4m3", [[60], [64]])
        c["q64"], c["q"] = bf16(c["q64"] * f)
        c["scale"] = float(np.float32(c["scale"] / f))
        check_attn(ctx, c)


def test_attention_later_nan_stays_out(ctx):
    # a NaN value or key that only the last token sees must not reach the others
    for T, Q, H, P in ((4, 4, 1, 16), (16, 8, 1, 16), (40, 4, 1, 16), (40, 4, 1, 32)):
        counts = 50 + np.arange(T)[None] + 1
        N = -(-(50 + T) // P)
        c = attn_case(19, 1, T, Q, H, 64, P, N, "e4m3", counts)
        clean = launch_attn(ctx, c)[0]
        for w in ("kc", "vc"):
            p, i = divmod(50 + T - 1, P)
            c[w][c["table"][0, p], :, i, 5] = 127
        out = launch_attn(ctx, c)[0]
        assert torch.isnan(out[0, T - 1]).any()
        assert torch.equal(out[0, :T - 1], clean[0, :T - 1])
    assert status(ctx) == 0


def test_attention_bad_values_are_reported(ctx):
    c = attn_case(20, 2, 1, 4, 1, 64, 16, 4, "int8", [[64], [64]], K=4, poison=False)
    c["page_idx"][0, 1] = 4
    c["page_idx"][0, 2] = -2
    check_attn(ctx, c, bits=4)
    c = attn_case(21, 2, 1, 4, 1, 64, 16, 4, "int8", [[64], [64]], poison=False)
    c["table"][0, 1] = 2 ** 31 - 1
    c["table"][1, 2] = -1
    check_attn(ctx, c, bits=4)
    c = attn_case(22, 2, 1, 4, 1, 64, 16, 4, "int8", [[65], [-3]], poison=False)
    check_attn(ctx, c, bits=1)


def test_attention_strided_queries_and_tables(ctx):
    c = attn_case(23, 3, 2, 4, 2, 64, 16, 5, "int8", [[80, 70], [3, 4], [0, 1]])
    wide = torch.randn((3, 2, 12, 64), device="cuda").to(torch.bfloat16)
    wide[:, :, 4:8] = c["q"]
    c["q"] = wide[:, :, 4:8]
    t = upload(c)
    big = torch.full((3, 9), 2 ** 30, dtype=torch.int32, device="cuda")
    big[:, :5] = t[4]
    t[4] = big[:, :5]
    out, lse = launch_attn(ctx, c, t=t)
    o, l, A, ds, top = ref.attention(c["q64"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["counts"],
                                     None, c["scale"], "int8")
    assert (np.abs(out.double().cpu().numpy() - o) <= ref.tolerance(o, A, ds, top, 80)).all()
    assert status(ctx) == 0


def test_attention_repeats_bit_for_bit(ctx):
    for counts, K in (([[9000]], 0), ([[9000]], 200)):
        c = attn_case(24, 1, 1, 8, 2, 128, 32, 282, "e4m3", counts, K=K)
        t = upload(c)
        a, la = launch_attn(ctx, c, t=t)
        for _ in range(3):
            b, lb = launch_attn(ctx, c, t=t)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_attention_on_another_stream_and_captured(ctx):
    c = attn_case(25, 2, 1, 8, 2, 128, 16, 200, "e4m3", [[3200], [777]])
    t = upload(c)
    want, wl = launch_attn(ctx, c, t=t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    launch_attn(ctx, c, out, lse, stream=s, t=t)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    outs = []
    for g in (g1, g2):  # two graphs on one context, replayed one after the other
        o, l = torch.zeros_like(want), torch.zeros_like(wl)
        with torch.cuda.graph(g):
            launch_attn(ctx, c, o, l, t=t)
        outs.append((o, l))
    for _ in range(3):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, wl)
    assert status(ctx) == 0


def test_binding_refuses(ctx):
    from page_scoring_top_b200 import binding
    c = attn_case(26, 2, 1, 4, 2, 64, 16, 4, "int8", [[64], [64]])
    t = upload(c)
    out = torch.empty((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")

    def call(q=c["q"], kc=t[0], vc=t[1], ks=t[2], vs=t[3], table=t[4], counts=t[5], o=out, **kw):
        binding.kv_attention(ctx, q, kc, vc, ks, vs, table, counts, o, **kw)

    call()
    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(q=c["q"].float()), dict(q=c["q"][0]), dict(kc=t[0].view(torch.uint8)),
               dict(vc=t[1][:1]), dict(vc=t[1].view(torch.float8_e4m3fn)), dict(ks=t[2].double()),
               dict(vs=t[3][:, :1]), dict(table=t[4].long()), dict(table=t[4][:1]),
               dict(counts=t[5][:1]), dict(o=out[:1]), dict(o=out.transpose(0, 1)),
               dict(lse=torch.empty((2, 4), device="cuda")), dict(q=c["q"].cpu()),
               dict(page_idx=torch.zeros((1, 3), **i32)), dict(page_idx=torch.zeros((2, 0), **i32)),
               dict(q=c["q"].transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    three = torch.empty((2, 1, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.IdxError):
        call(q=three, o=three.clone())
    with pytest.raises(binding.IdxError):
        call(scale=float("nan"))
    slots = torch.zeros(2, **i32)
    with pytest.raises(ValueError):
        binding.kv_append(ctx, c["q"][:, 0], c["q"][:, 0], slots, *t[:4])
    assert status(ctx) == 0


# -------------------------------------------------------------- the whole path
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_serving_steps(ctx, fmt):
    """A prompt, then decode steps: tables, append, pooled page centroids, the indexer's
    selection, attention over the selected pages -- against the references over the cache that
    the append itself is checked to have written."""
    from page_scoring_top_b200 import binding
    B, H, Q, D, P, N, K = 3, 2, 8, 128, 16, 24, 5
    n_blocks = B * N
    rng = np.random.default_rng(31)
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(n_blocks).astype(np.int32)).cuda()
    heads = [torch.zeros(1, **i32), torch.zeros(1, **i32)]
    table = torch.full((B, N), -1, **i32)
    cache = [torch.zeros((n_blocks, H, P, D), dtype=CODE[fmt], device="cuda") for _ in range(2)]
    scale = [torch.zeros((n_blocks, H), device="cuda") for _ in range(2)]
    cached = np.zeros(B, np.int32)
    all_keys = np.zeros((B, N * P, D))
    refk = [np.zeros((n_blocks, H, P, D), np.uint8) for _ in range(2)]
    refs = [np.zeros((n_blocks, H), np.float32) for _ in range(2)]
    with binding.Context(0, max_rows=B * 4, max_n=N, max_k=K) as ictx:
        for step, T in enumerate((150, 1, 4, 1)):
            fresh = np.minimum(np.int32([T, T, 77]), T)
            maps = [torch.empty((B, T), **i32) for _ in range(3)]
            binding.kv_block_tables(ctx, dev(cached), dev(fresh), P, n_blocks, table, free, heads[0],
                                    heads[1], *maps)
            heads.reverse()
            slots, counts, pages = maps
            (k64, k), (v64, v) = [bf16(rng.standard_normal((B, T, H, D))) for _ in range(2)]
            binding.kv_append(ctx, k.view(B * T, H, D), v.view(B * T, H, D), slots, *cache, *scale)
            for i, x in enumerate((k64, v64)):
                refk[i], refs[i] = ref.append(x.reshape(B * T, H, D), slots.cpu().numpy().reshape(-1),
                                              refk[i], refs[i], fmt)
                assert np.array_equal(cache[i].view(torch.uint8).cpu().numpy(), refk[i])
                assert np.array_equal(scale[i].cpu().numpy(), refs[i])
            for b in range(B):
                all_keys[b, cached[b]:cached[b] + fresh[b]] = k64[b, :fresh[b], 0]
            cached += fresh
            q64, q = bf16(rng.standard_normal((B, T, Q, D)))
            page_idx = None
            if T <= 4:  # decode: the indexer picks the pages
                keys = synth.f32_to_bf16_bits(all_keys.astype(np.float32)).view(np.int16)
                cent = torch.zeros((B, N, D), dtype=torch.int16, device="cuda")
                binding.centroid_pool(ictx, dev(keys), dev(cached), P, cent)
                page_idx = torch.empty((B * T, K), **i32)
                binding.score_topk_fused_tokens(ictx, q, cent, pages, K, page_idx)
                assert binding.idx_get_status(ictx)[1] == 0
            out = torch.empty((B, T, Q, D), dtype=torch.bfloat16, device="cuda")
            lse = torch.empty((B, T, Q), device="cuda")
            binding.kv_attention(ctx, q, *cache, *scale, table, counts, out, lse=lse, page_idx=page_idx)
            o, l, A, ds, top = ref.attention(
                q64, refk[0], refk[1], refs[0], refs[1], table.cpu().numpy(), counts.cpu().numpy(),
                None if page_idx is None else page_idx.cpu().numpy(), D ** -0.5, fmt)
            assert (np.abs(out.double().cpu().numpy() - o) <= ref.tolerance(o, A, ds, top, N * P)).all()
            assert np.array_equal(np.isneginf(l), np.isneginf(lse.cpu().numpy()))
    assert status(ctx) == 0
