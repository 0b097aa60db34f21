// kv_attn.cu -- what kv_attention launches (the kernels are in kv_attn.cuh).
#include "kv_attn.cuh"

namespace idx {

size_t kv_attn_ws_floats(int num_sms) { return (size_t)num_sms * 2 * kKvSlot; }

bool encode_cache_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const KvAttnArgs& a,
                      const uint8_t* cache, int dp, int rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)a.D, (cuuint64_t)a.n_blocks * a.H * a.P};
  const cuuint64_t strides[1] = {(cuuint64_t)a.D};
  const cuuint32_t box[2] = {(cuuint32_t)(dp < 128 ? dp : 128), (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(cache), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                dp == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv_attn(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  if (kv_attn_tc_supported(a)) return launch_kv_attn_tc(a, num_sms, stream);
  auto encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const int G = a.Q / a.H;
  const int dp = a.D <= 64 ? 64 : (a.D <= 128 ? 128 : 256);
  KvPlan pl{};
  // As few 8-row blocks as hold the tile's query rows.  Tokens share a tile only
  // where they share the keys.
  pl.GG = G < 64 ? G : 64;
  pl.ng = (G + pl.GG - 1) / pl.GG;
  const int64_t rows = a.page_idx ? G : (int64_t)G * a.T;
  const int nt = rows <= 8 ? 1 : 2, rg = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  const int fit = 8 * nt * rg / pl.GG;
  pl.TT = a.page_idx || fit < 1 ? 1 : (fit < a.T ? fit : a.T);
  pl.ntb = (a.T + pl.TT - 1) / pl.TT;
  // A copy must start on 128 bytes of shared memory: 64-byte rows go in pairs.
  pl.pitch = dp == 64 ? (a.P + 1) & ~1 : a.P;
  pl.ppt = pl.pitch <= kKvUnit / 2 ? kKvUnit / pl.pitch : 1;
  pl.tpp = (a.P + kKvUnit - 1) / kKvUnit;
  pl.box = a.P < kKvUnit ? a.P : kKvUnit;
  pl.ws = a.ws;
  pl.arrive = a.arrive;
  CUtensorMap mk, mv;
  if (!encode_cache_map(encode, &mk, a, a.k_cache, dp, pl.box) ||
      !encode_cache_map(encode, &mv, a, a.v_cache, dp, pl.box))
    return cudaErrorInvalidValue;
  if (dp == 64) return launch_kv_attn_dp<64>(mk, mv, a, pl, nt, rg, num_sms, stream);
  if (dp == 128) return launch_kv_attn_dp<128>(mk, mv, a, pl, nt, rg, num_sms, stream);
  return launch_kv_attn_dp<256>(mk, mv, a, pl, nt, rg, num_sms, stream);
}

}  // namespace idx
