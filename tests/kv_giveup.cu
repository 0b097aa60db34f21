// kv_giveup.cu -- the attention kernels in a build for tests, in which one CTA
// of a launch may run as if one of its bounded waits had expired: it abandons
// its work in the middle, with copies in flight, and has to leave everything
// that later launches use as a CTA that ends does.
#include <cstdint>
#include <cuda_runtime.h>

__device__ int g_give_up = -1;
__device__ __forceinline__ bool give_up(int* status) {
  if ((int)blockIdx.x != g_give_up) return false;
  atomicOr(status, 2);  // what an expired wait raises
  return true;
}
#define IDX_KV_GIVE_UP give_up(a.status)

#include "kv_attn.cuh"

namespace idx {

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

// Of the streamed kernel: one row block of D <= 64 codes, large and small pages.
template <>
cudaError_t launch_kv_attn_dp<64>(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& a, KvPlan pl,
                                  int nt, int rg, int grid, cudaStream_t stream) {
  if (nt != 1 || rg != 1 || a.format != kKvE4m3) return cudaErrorNotSupported;
  return pl.ppt > 1 ? launch_one<kKvE4m3, 64, 1, 1, true>(mk, mv, a, pl, grid, stream)
                    : launch_one<kKvE4m3, 64, 1, 1, false>(mk, mv, a, pl, grid, stream);
}
template <>
cudaError_t launch_kv_attn_dp<128>(const CUtensorMap&, const CUtensorMap&, const KvAttnArgs&, KvPlan, int, int,
                                   int, cudaStream_t) {
  return cudaErrorNotSupported;
}
template <>
cudaError_t launch_kv_attn_dp<256>(const CUtensorMap&, const CUtensorMap&, const KvAttnArgs&, KvPlan, int, int,
                                   int, cudaStream_t) {
  return cudaErrorNotSupported;
}

}  // namespace idx

#include "kv_attn.cu"
#include "kv_attn_tc.cu"

#define EXPORT extern "C" __attribute__((visibility("default")))

EXPORT int64_t giveup_ws_floats(int num_sms) { return (int64_t)idx::kv_attn_ws_floats(num_sms); }

// kv_attention of a contiguous e4m3 batch without page lists, on the current
// device and the default stream, with CTA `cta` giving up (-1: none).
EXPORT int giveup_attention(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, int n_blocks, const int32_t* page_table, int N,
                            const int32_t* key_counts, int B, int T, int Q, int H, int D, int P, float scale,
                            void* out, float* lse, float* ws, int32_t* arrive, int* status, int num_sms, int cta) {
  if (cudaMemcpyToSymbol(g_give_up, &cta, sizeof(int)) != cudaSuccess) return -1;
  idx::KvAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.ldq = (int64_t)Q * D;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.n_blocks = n_blocks;
  a.format = idx::kKvE4m3;
  a.page_table = page_table;
  a.ld_pt = N;
  a.N = N;
  a.key_counts = key_counts;
  a.B = B;
  a.T = T;
  a.Q = Q;
  a.H = H;
  a.D = D;
  a.P = P;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.ws = ws;
  a.arrive = arrive;
  a.status = status;
  if (idx::launch_kv_attn(a, num_sms, nullptr) != cudaSuccess) return -2;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : -3;
}
