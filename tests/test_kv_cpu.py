"""CPU checks of the 8-bit KV cache calls: what the host refuses before any
launch (no GPU is touched: the context is a block of zeros that a refused call
never reads), the binding's checks, and the references against hand-worked
values."""

import ctypes

import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")

EINVAL, EUNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from page_scoring_top_b200 import binding, build
    build.build()
    return binding.lib()


CTX = ctypes.create_string_buffer(4096)
MEM = ctypes.create_string_buffer(8192)
BASE = (ctypes.addressof(MEM) + 255) & ~255


def _call(fn, names, good, **change):
    args = dict(good, **change)
    return fn(*[args[n] for n in names])


TABLES = "ctx cached fresh B T P N page_table ld_pt n_blocks free_list n_free free_head " \
         "free_head_out slots key_counts page_counts stream".split()
TABLES_OK = dict(ctx=ctypes.addressof(CTX), cached=BASE, fresh=BASE, B=2, T=3, P=16, N=4,
                 page_table=BASE, ld_pt=4, n_blocks=8, free_list=BASE, n_free=8, free_head=BASE,
                 free_head_out=BASE + 4, slots=BASE, key_counts=BASE, page_counts=BASE, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), EINVAL), (dict(cached=None), EINVAL), (dict(page_table=None), EINVAL),
    (dict(slots=None), EINVAL), (dict(key_counts=None), EINVAL), (dict(page_counts=None), EINVAL),
    (dict(B=0), EINVAL), (dict(T=0), EINVAL), (dict(P=0), EINVAL), (dict(N=0), EINVAL),
    (dict(ld_pt=3), EINVAL), (dict(n_blocks=0), EINVAL), (dict(n_free=-1), EINVAL),
    (dict(free_list=None), EINVAL), (dict(free_head_out=BASE), EINVAL),
    (dict(P=1 << 20, N=1 << 12, ld_pt=1 << 12), EUNSUPPORTED),
    (dict(n_blocks=1 << 30), EUNSUPPORTED), (dict(B=1 << 20, T=1 << 12), EUNSUPPORTED)])
def test_block_tables_refuses(lib, change, code):
    assert _call(lib.kv_block_tables, TABLES, TABLES_OK, **change) == code


APPEND = "ctx k v ldk ldv slots R H D P n_blocks format k_cache v_cache k_scale v_scale stream".split()
APPEND_OK = dict(ctx=ctypes.addressof(CTX), k=BASE, v=BASE, ldk=256, ldv=256, slots=BASE, R=2, H=2,
                 D=128, P=16, n_blocks=4, format=0, k_cache=BASE, v_cache=BASE, k_scale=BASE,
                 v_scale=BASE, stream=None)


CACHE_BAD = [
    (dict(k_cache=None), EINVAL), (dict(v_cache=None), EINVAL), (dict(k_scale=None), EINVAL),
    (dict(v_scale=None), EINVAL), (dict(k_cache=BASE + 8), EINVAL), (dict(v_cache=BASE + 1), EINVAL),
    (dict(k_scale=BASE + 2), EINVAL), (dict(n_blocks=0), EINVAL), (dict(H=0), EINVAL),
    (dict(P=0), EINVAL), (dict(format=2), EINVAL), (dict(format=-1), EINVAL),
    (dict(D=0), EINVAL), (dict(D=72), EUNSUPPORTED), (dict(D=272), EUNSUPPORTED),
    (dict(n_blocks=1 << 27), EUNSUPPORTED), (dict(P=1 << 17), EUNSUPPORTED)]


@pytest.mark.parametrize("change,code", CACHE_BAD + [
    (dict(ctx=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
    (dict(slots=None), EINVAL), (dict(R=0), EINVAL), (dict(k=BASE + 8), EINVAL),
    (dict(v=BASE + 2), EINVAL), (dict(ldk=260), EINVAL), (dict(ldv=248), EINVAL), (dict(ldk=0), EINVAL)])
def test_append_refuses(lib, change, code):
    assert _call(lib.kv_append, APPEND, APPEND_OK, **change) == code


ATTN = "ctx q ldq k_cache v_cache k_scale v_scale n_blocks format page_table ld_pt N key_counts " \
       "page_idx K B T Q H D P scale out lse stream".split()
ATTN_OK = dict(ctx=ctypes.addressof(CTX), q=BASE, ldq=512, k_cache=BASE, v_cache=BASE, k_scale=BASE,
               v_scale=BASE, n_blocks=4, format=0, page_table=BASE, ld_pt=4, N=4, key_counts=BASE,
               page_idx=BASE, K=2, B=1, T=1, Q=4, H=2, D=128, P=16, scale=0.1, out=BASE, lse=None,
               stream=None)


@pytest.mark.parametrize("change,code", CACHE_BAD + [
    (dict(ctx=None), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL),
    (dict(page_table=None), EINVAL), (dict(key_counts=None), EINVAL), (dict(B=0), EINVAL),
    (dict(T=0), EINVAL), (dict(Q=0), EINVAL), (dict(Q=5), EINVAL), (dict(N=0), EINVAL),
    (dict(ld_pt=3), EINVAL), (dict(K=0), EINVAL), (dict(page_idx=None), EINVAL),
    (dict(q=BASE + 8), EINVAL), (dict(out=BASE + 8), EINVAL), (dict(ldq=516), EINVAL),
    (dict(ldq=504), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(N=1 << 28, ld_pt=1 << 28), EUNSUPPORTED), (dict(B=1 << 20, T=1 << 10), EUNSUPPORTED)])
def test_attention_refuses(lib, change, code):
    assert _call(lib.kv_attention, ATTN, ATTN_OK, **change) == code


class _Ctx:
    device, handle = 0, None


def test_binding_refuses_tensors_off_the_device():
    from page_scoring_top_b200 import binding
    z = torch.zeros
    kc = z((2, 1, 16, 64), dtype=torch.int8)
    sc = z((2, 1))
    with pytest.raises(ValueError):
        binding.kv_append(_Ctx, z((1, 1, 64), dtype=torch.bfloat16), z((1, 1, 64), dtype=torch.bfloat16),
                          z(1, dtype=torch.int32), kc, kc, sc, sc)
    with pytest.raises(ValueError):
        binding.kv_attention(_Ctx, z((1, 1, 1, 64), dtype=torch.bfloat16), kc, kc, sc, sc,
                             z((1, 2), dtype=torch.int32), z((1, 1), dtype=torch.int32),
                             z((1, 1, 1, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        binding.kv_block_tables(_Ctx, z(1, dtype=torch.int32), None, 16, 2, z((1, 2), dtype=torch.int32),
                                z(2, dtype=torch.int32), None, None, z((1, 1), dtype=torch.int32),
                                z((1, 1), dtype=torch.int32), z((1, 1), dtype=torch.int32))


def test_binding_row_strides():
    from page_scoring_top_b200.binding import _kv_rows
    x = torch.zeros((6, 5, 8))
    assert _kv_rows("x", x, 1) == 40
    assert _kv_rows("x", x[:, 1:3], 1) == 40
    assert _kv_rows("x", x[::2, 1:3], 1) == 80
    assert _kv_rows("x", x[:1, 1:3], 1) == 16
    assert _kv_rows("x", x[:1].expand(6, 5, 8), 1) == 0  # the C call refuses it
    y = x.view(2, 3, 5, 8)
    assert _kv_rows("y", y[:, :, :2], 2) == 40
    assert _kv_rows("y", y[:, :1, :2], 2) == 120
    assert _kv_rows("y", y[:1, :, :2], 2) == 40
    for bad in (y[:, :2], y.transpose(0, 1), x.transpose(1, 2).unsqueeze(0)):
        with pytest.raises(ValueError):
            _kv_rows("y", bad, 2)


# ------------------------------------------------------------- the references
def test_reference_codes():
    assert ref.E4M3[0x7E] == 448 and ref.E4M3[0x08] == 2.0 ** -6 and ref.E4M3[0x01] == 2.0 ** -9
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.E4M3, t, equal_nan=True)
    x = np.array([0.0, 447.0, 448, 1000, -1000, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -11, np.inf, np.nan])
    want = [0x00, 0x7E, 0x7E, 0x7E, 0xFE, 0x38, 0x3A, 0x00, 0x01, 0x7E, 0x7F]
    assert ref.encode(x, "e4m3").tolist() == want
    x = np.linspace(-460, 460, 9001)
    got = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(ref.encode(np.float32(x).astype(np.float64), "e4m3"), got.numpy())
    assert ref.encode(np.array([0.5, 1.5, -2.5, 300.0, -300.0]), "int8").view(np.int8).tolist() == [0, 2, -2, 127, -127]


def test_reference_scales():
    assert ref.scale_for(448.0, "e4m3") == 1 and ref.scale_for(449.0, "e4m3") == 2
    assert ref.scale_for(127.0, "int8") == 1 and ref.scale_for(127.5, "int8") == 2
    assert ref.scale_for(0.0, "int8") == 2.0 ** -100


def test_reference_tables_by_hand():
    table = np.array([[7, -9], [-9, -9]], np.int32)
    out = ref.block_tables([3, 0], [2, 1], 2, 4, 2, table, 10, [5, 6, 2], 1)
    assert out[0].tolist() == [[7, 6], [2, -9]]
    assert out[1].tolist() == [[31, 24], [8, -1]]
    assert out[2].tolist() == [[4, 5], [1, 0]] and out[3].tolist() == [[1, 2], [1, 0]] and out[4] == 3


def test_reference_attention_by_hand():
    # one page, two keys, one of them past the count: the output is the first value row
    k = np.zeros((1, 1, 2, 16), np.uint8)
    v = np.full((1, 1, 2, 16), 4, np.uint8)
    v[0, 0, 1] = 100
    o = ref.attention(np.ones((1, 1, 1, 16)), k, v, np.ones((1, 1)), np.full((1, 1), 0.5),
                      np.zeros((1, 1), int), np.array([[1]]), None, 1.0, "int8")
    assert (o[0] == 2).all() and o[1].item() == 0.0
