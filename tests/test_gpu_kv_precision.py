"""What kv_attention's fp16 operands hold: outputs that rest on weights far below
the row's largest, value scales far apart, queries of a wide range.

The bound counts the roundings: bf16's half step 2^-8 of the result; fp16's half
step 2^-11 of a weight, and below its normal range FLOOR of the largest weight
(times its value scale); twice the scores' fp32 error; one fp32 step per 16 keys
that a tensor-core sum takes in, and a few of the joins'."""

import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv import bf16, ctx, launch_attn, status  # noqa: F401  (ctx: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

STREAMED, PROMPT = 2.0 ** -39, 2.0 ** -32


def make(fmt, T, Q, D, P, keys, K=0, seed=0):
    """One request whose T tokens see about `keys` keys: codes zero, scales one, q = (1, 0, ...)."""
    N = -(-keys // P)
    rng = np.random.default_rng(seed)
    q = np.zeros((1, T, Q, D))
    q[..., 0] = 1
    c = dict(fmt=fmt, scale=1.0, counts=(keys - T + 1 + np.arange(T, dtype=np.int32))[None],
             kc=np.zeros((N, 1, P, D), np.uint8), vc=np.zeros((N, 1, P, D), np.uint8),
             ks=np.ones((N, 1), np.float32), vs=np.ones((N, 1), np.float32),
             table=rng.permutation(N).astype(np.int32)[None], page_idx=None)
    c["q64"], c["q"] = bf16(q)
    if K:
        c["page_idx"] = np.stack([rng.permutation(N)[:K] for _ in range(T)]).astype(np.int32)
    return c, rng


def at(c, name):
    """The codes of the request's keys in the order of their positions (a copy), and back."""
    x = c[name][c["table"][0], 0]
    return x.reshape(-1, x.shape[-1])


def put(c, name, x):
    c[name][c["table"][0], 0] = x.reshape(c[name][c["table"][0], 0].shape)


def check(ctx, c, floor):
    """Against the formula in 64 bits, every output column for itself."""
    out, lse = launch_attn(ctx, c)
    got, gl = out.double().cpu().numpy()[0], lse.double().cpu().numpy()[0]
    P, D = c["kc"].shape[2:]
    pages = c["table"][0]
    k = ref.decode(at(c, "kc"), c["fmt"]) * c["ks"][pages, 0].astype(np.float64).repeat(P)[:, None]
    v8 = ref.decode(at(c, "vc"), c["fmt"])
    w = c["vs"][pages, 0].astype(np.float64).repeat(P)
    scale = float(np.float32(c["scale"]))
    for t in range(got.shape[0]):
        keep = np.arange(len(k)) < c["counts"][0, t]
        if c["page_idx"] is not None:
            keep &= np.isin(np.arange(len(k)) // P, c["page_idx"][t])
        s = (c["q64"][0, t] @ k[keep].T) * scale
        sabs = (np.abs(c["q64"][0, t]) @ np.abs(k[keep].T)) * abs(scale)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        p /= l
        want, A = p @ (w[keep][:, None] * v8[keep]), p @ (w[keep][:, None] * np.abs(v8[keep]))
        ds = 2.0 ** -24 * ((D + 8) * sabs.max(1) + 8 * np.abs(s).max(1) + 8)[:, None]
        sums = 2.0 ** -23 * (keep.sum() / 16 + 64)
        tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -11 + 2 * ds + sums) \
            + floor * (p * w[keep]).max(1)[:, None] * np.abs(v8[keep]).sum(0)
        off = np.abs(got[t] - want) / (tol + 1e-300)
        assert off.max() <= 1, "token %d: %.3g of the bound, %.3g relative to the result" % (
            t, off.max(), (np.abs(got[t] - want) / np.abs(want).clip(1e-300)).max())
        z = (m + np.log(l))[:, 0]
        ltol = 2 * ds[:, 0] + 2.0 ** -22 * (np.abs(z) + 4) + sums
        assert (np.abs(gl[t] - z) <= ltol).all()
    assert status(ctx) == 0


KERNELS = [(STREAMED, dict(T=1, Q=4, D=64, P=64)), (STREAMED, dict(T=2, Q=16, D=128, P=16)),
           (STREAMED, dict(T=1, Q=8, D=256, P=32)), (STREAMED, dict(T=1, Q=4, D=128, P=64, K=50)),
           (PROMPT, dict(T=40, Q=4, D=128, P=64)), (PROMPT, dict(T=20, Q=8, D=64, P=16))]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("below", [18.3, 20.4, 22.6, 23.6, 25.5])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_keys_far_below_the_largest_weight(ctx, fmt, below, floor, shape):
    # every 32nd key has 2^below times the weight of the others and no value in
    # half of the columns: those hold the others' values alone
    c, rng = make(fmt, keys=4096, seed=int(below * 10), **shape)
    n, D = at(c, "kc").shape
    sink = np.arange(n) % 32 == 7
    k, v = np.zeros((n, D)), rng.integers(40, 56, (n, D)).astype(float)
    k[sink, 0] = 64
    v[sink, :D // 2] = 0
    put(c, "kc", ref.encode(k, fmt))
    put(c, "vc", ref.encode(v, fmt))
    c["scale"] = float(np.float32(below * np.log(2) / 64))
    check(ctx, c, floor)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 1.3 * 2.0 ** 20, 1.7 * 2.0 ** 23])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_pages_far_below_the_largest_value_scale(ctx, fmt, ratio, floor, shape):
    # equal weights; a third of the pages has value scales `ratio` times the
    # others' and no value in half of the columns
    c, rng = make(fmt, keys=4096, seed=int(ratio), **shape)
    n, D = at(c, "kc").shape
    P = c["kc"].shape[2]
    big = np.arange(n) // P % 3 == 1
    v = rng.integers(40, 56, (n, D)).astype(float)
    v[big, :D // 2] = 0
    put(c, "vc", ref.encode(v, fmt))
    c["vs"][c["table"][0], 0] = np.where(big[::P], ratio, 0.77)
    check(ctx, c, floor)


@pytest.mark.parametrize("top", [10, 14, 20, 22, 24, 25, 26, 27, 28, 30, 60])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_scores_whose_fp32_steps_are_large(ctx, top, floor, shape):
    # the scores' own fp32 steps reach 2, 4, 8 ... : one key is far above the
    # others and the output is its value
    for sign in (1, -1):
        c, rng = make("int8", keys=300, seed=top, **dict(shape, **({"K": 4} if "K" in shape else {})))
        n, D = at(c, "kc").shape
        P = c["kc"].shape[2]
        best = [int(x) * P + 3 for x in (range(-(-n // P)) if c["page_idx"] is None else c["page_idx"][0])][1]
        k = np.zeros((n, D))
        k[:, 0] = sign * 64
        k[best, 0] = sign * 64 + 32
        v = rng.integers(-127, 128, (n, D)).astype(float)
        put(c, "kc", ref.encode(k, "int8"))
        put(c, "vc", ref.encode(v, "int8"))
        c["scale"] = float(2.0 ** (top - 6))
        out, lse = launch_attn(ctx, c)
        got = out.double().cpu().numpy()[0]
        tol = 2.0 ** -8 * np.abs(v[best]) + 2.0 ** -10 * 127
        assert (np.abs(got - v[best]) <= tol).all()
        assert torch.isfinite(lse).all()
    assert status(ctx) == 0


@pytest.mark.parametrize("vs", [2.0 ** -110, 2.0 ** -99, 2.0 ** -86, 1.5 * 2.0 ** -90, 2.0 ** 100, 3e36])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_value_scales_at_the_ends_of_their_range(ctx, vs, floor, shape):
    c, rng = make("int8", keys=2000, seed=3, **shape)
    n, D = at(c, "kc").shape
    k = rng.integers(-60, 61, (n, D)).astype(float)
    put(c, "kc", ref.encode(k, "int8"))
    put(c, "vc", ref.encode(rng.integers(1, 100, (n, D)).astype(float), "int8"))
    c["scale"] = 0.02
    c["vs"][:] = vs
    if vs < 2.0 ** -86:
        floor = 2.0 ** -24  # (counts as 2^-86: the weights keep 2^14 less)
    check(ctx, c, floor)


def test_many_keys_of_zero_scale(ctx):
    # the sum of the weights over the smallest scale stays finite
    for shape in (dict(T=1, Q=4, D=64, P=64), dict(T=20, Q=4, D=64, P=64)):
        c, _ = make("int8", keys=40000, **shape)
        c["vs"][:] = 0
        out, lse = launch_attn(ctx, c)
        assert not out.any()
        want = np.log(c["counts"][0].astype(float))
        assert np.abs(lse.double().cpu().numpy()[0] - want[:, None]).max() < 1e-4
    assert status(ctx) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("span", [0, 12, 18, 21, 24])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_queries_with_an_element_far_above_the_others(ctx, fmt, span, floor, shape):
    # one element 2^span above the others, where the keys are zero: the scores are
    # those of the other elements, which use all of bf16's digits
    c, rng = make(fmt, keys=700, seed=span, **dict(shape, **({"K": 8} if "K" in shape else {})))
    n, D = at(c, "kc").shape
    q = rng.uniform(0.25, 2, c["q64"].shape) * rng.choice([-1, 1], c["q64"].shape)
    q[..., 5] = 2.0 ** span
    c["q64"], c["q"] = bf16(q)
    k = rng.integers(-60, 61, (n, D)).astype(float)
    k[:, 5] = 0
    put(c, "kc", ref.encode(k, fmt))
    put(c, "vc", ref.encode(rng.integers(-100, 101, (n, D)).astype(float), fmt))
    c["scale"] = float(np.float32(3 / (40 * 1.2 * D ** 0.5)))
    check(ctx, c, floor)


@pytest.mark.parametrize("size", [1e-39, 2.0 ** -130, 1e-36, 2.0 ** -112, 1e-30, 1e30, 3e38])
@pytest.mark.parametrize("floor,shape", KERNELS)
def test_queries_at_the_ends_of_their_range(ctx, size, floor, shape):
    c, rng = make("int8", keys=500, seed=9, **dict(shape, **({"K": 8} if "K" in shape else {})))
    n, D = at(c, "kc").shape
    c["q64"], c["q"] = bf16(rng.choice([-1, 0.5, 1], c["q64"].shape) * size)
    k = rng.integers(-60, 61, (n, D)).astype(float)
    put(c, "kc", ref.encode(k, "int8"))
    put(c, "vc", ref.encode(rng.integers(-100, 101, (n, D)).astype(float), "int8"))
    c["scale"] = float(np.float32(min(3 / (40 * D ** 0.5) / size, 1e38)))
    check(ctx, c, floor)


@pytest.mark.parametrize("floor,shape", KERNELS)
def test_lse_of_a_few_equal_scores(ctx, floor, shape):
    # log(n): a base-2 logarithm below 4 to two fp32 steps of 2^-22, and two roundings
    shape = dict(shape)
    shape.pop("K", None)
    for n in range(1, 16):
        c, _ = make("int8", keys=64, **shape)
        c["counts"][:] = n
        lse = launch_attn(ctx, c)[1].double().cpu().numpy()
        assert np.abs(lse - np.log(n)).max() <= np.log(2) * 2.0 ** -21 + 2 * 2.0 ** -24 * np.log(n)
    assert status(ctx) == 0
