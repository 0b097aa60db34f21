"""What kv_attention's fp16 operands and fp32 scores hold."""

import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv import bf16, ctx, launch_attn, status  # noqa: F401  (ctx: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


KERNELS = [("streamed", dict(T=1, Q=4, D=64, P=64)), ("streamed", dict(T=2, Q=16, D=128, P=16)),
           ("streamed", dict(T=1, Q=8, D=256, P=32)), ("streamed", dict(T=1, Q=4, D=128, P=64, K=50)),
           ("prompt", dict(T=40, Q=4, D=128, P=64)), ("prompt", dict(T=20, Q=8, D=64, P=16))]


@pytest.mark.parametrize("top", [10, 14, 20, 22, 24, 25, 26, 27, 28, 30, 60])
@pytest.mark.parametrize("kernel,shape", KERNELS)
def test_scores_whose_fp32_steps_are_large(ctx, top, kernel, shape):
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
