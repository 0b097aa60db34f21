"""What the workspace of attention over the KV cache costs a context, and that the
calls that share its memory leave one another alone."""

import numpy as np
import pytest

from test_gpu_kv import attn_case, launch_attn, upload

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def taken(**limits):
    from page_scoring_top_b200 import binding
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    with binding.Context(0, **limits):
        return before - torch.cuda.mem_get_info()[0]


def test_a_context_with_large_limits_pays_no_more_for_it():
    # the attention's 19.7 MB lie within the scores' scratch, 67 MB here
    taken(max_rows=1, max_n=1, max_k=1)
    small = taken(max_rows=1, max_n=1, max_k=1)
    large = taken(max_rows=64, max_n=1 << 18, max_k=1)
    scratch = 64 * (1 << 18) * 4
    lists = large - scratch  # what a context of these limits has besides
    assert small <= 24 << 20
    assert lists < 12 << 20, "%.1f MB beside the scratch" % (lists / 1e6)


def test_calls_in_turn_on_one_context():
    from page_scoring_top_b200 import binding
    c = attn_case(50, 2, 1, 8, 2, 128, 16, 200, "e4m3", [[3200], [777]])
    t = upload(c)
    g = torch.Generator(device="cuda").manual_seed(1)
    B, T, N, Q, D, K = 4, 8, 5000, 3, 96, 300  # eight tokens: scores into the scratch, then the selection
    q = torch.randn((B, T, Q, D), generator=g, device="cuda").to(torch.bfloat16)
    cent = torch.randn((B, N, D), generator=g, device="cuda").to(torch.bfloat16)
    with binding.Context(0, max_rows=B * T, max_n=N, max_k=K) as ctx:
        def select():
            idx = torch.empty((B * T, K), dtype=torch.int32, device="cuda")
            val = torch.empty((B * T, K), device="cuda")
            binding.score_topk_fused(ctx, q, cent, None, K, idx, val)
            return idx, val
        want, wl = launch_attn(ctx, c, t=t)
        wi, wv = select()
        for _ in range(5):
            out, lse = launch_attn(ctx, c, t=t)
            idx, val = select()
            assert torch.equal(out, want) and torch.equal(lse, wl)
            assert torch.equal(idx, wi) and torch.equal(val, wv)
        assert binding.idx_get_status(ctx)[1] == 0
    assert np.isfinite(wv.cpu().numpy()).all()
