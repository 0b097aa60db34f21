"""CPU checks of what the 8-bit KV cache calls refuse at the ends of their ranges
(no GPU is touched: a refused call never reads its context)."""

import ctypes

import pytest

from test_kv_cpu import ATTN, ATTN_OK, EINVAL, EUNSUPPORTED, TABLES, TABLES_OK, _call, lib  # noqa: F401  (lib: the fixture)

pytest.importorskip("torch")

# buffers of their own for every argument (B = 2, T = 3; 8 entries in the free list)
PLACES = ctypes.create_string_buffer(4096)
AT = (ctypes.addressof(PLACES) + 255) & ~255
APART = dict(TABLES_OK, cached=AT, fresh=AT + 64, page_table=AT + 128, free_list=AT + 192, free_head=AT + 256,
             free_head_out=AT + 320, slots=AT + 384, key_counts=AT + 448, page_counts=AT + 512)


@pytest.mark.parametrize("out", ["slots", "key_counts", "page_counts", "free_head_out"])
@pytest.mark.parametrize("read,entries", [("cached", 2), ("fresh", 2), ("free_list", 8), ("free_head", 1)])
def test_block_tables_refuses_outputs_over_its_inputs(lib, out, read, entries):  # noqa: F811
    size = 1 if out == "free_head_out" else 6
    for off in (0, entries - 1, 1 - size):
        assert _call(lib.kv_block_tables, TABLES, APART, **{out: APART[read] + 4 * off}) == EINVAL
    for off in (entries, -size):  # side by side: not refused for that (nor launched here, without a GPU)
        import torch
        if not torch.cuda.is_available():
            assert _call(lib.kv_block_tables, TABLES, APART, **{out: APART[read] + 4 * off}) != EINVAL


NEAR = (2 ** 31 - 17) // 16  # pages of 16 that hold the most positions below 2^31 - 16


@pytest.mark.parametrize("change", [
    dict(N=NEAR, ld_pt=NEAR, page_idx=None, K=0), dict(N=NEAR, ld_pt=NEAR), dict(K=2 ** 31 - 20)])
def test_attention_refuses_positions_that_leave_31_bits(lib, change):  # noqa: F811
    assert _call(lib.kv_attention, ATTN, ATTN_OK, **change) == EUNSUPPORTED


def test_the_text_for_unsupported_shapes_covers_the_cache(lib):  # noqa: F811
    lib.idx_strerror.restype = ctypes.c_char_p
    text = lib.idx_strerror(EUNSUPPORTED)
    assert b"multiple of 8" in text and b"16 for the KV cache" in text and b"limit" in text
