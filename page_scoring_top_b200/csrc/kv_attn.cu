// kv_attn.cu -- attention over the pages of the 8-bit KV cache.
//
// Row (b, t), query head h, kv head g = h / (Q / H): over the keys i of the
// row's pages with position < key_counts[b][t],
//     s_i = scale * (q . k8_i) * k_scale[page, g],
//     out = sum_i softmax(s)_i * v8_i * v_scale[page, g],  lse = log sum_i exp(s_i)
// with the running maximum and sum of a softmax kept in fp32.  One warp per
// (row, query head); lane l holds elements 8 l .. 8 l + 7.
#include "kv.cuh"

namespace idx {

namespace {

constexpr int kWarps = 4;

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) kv_attn_simple(const KvAttnArgs a) {
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.B * a.T * a.Q) return;
  const int64_t r = w / a.Q;
  const int h = (int)(w - r * a.Q), g = h / (a.Q / a.H);
  const int b = (int)(r / a.T);
  const bool on = lane * 8 < a.D;
  int bits = 0;
  int count = a.key_counts[r];
  if (count < 0 || count > a.N * a.P) {
    bits |= kErrLengthClamped;
    count = count < 0 ? 0 : a.N * a.P;
  }
  float q[8], o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = on ? __uint_as_float((uint32_t)a.q[r * a.ldq + (int64_t)h * a.D + lane * 8 + e] << 16)
              : 0.f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int np = a.page_idx ? a.K : (count + a.P - 1) / a.P;
  for (int n = 0; n < np; ++n) {
    const int p = a.page_idx ? a.page_idx[r * a.K + n] : n;
    if (p < 0 || p >= a.N) {
      if (p != -1) bits |= kErrPageClamped;
      continue;
    }
    if ((int64_t)p * a.P >= count) continue;
    const int id = a.page_table[(int64_t)b * a.ld_pt + p];
    if (id < 0 || id >= a.n_blocks) {
      bits |= kErrPageClamped;
      continue;
    }
    const int64_t cell = (int64_t)id * a.H + g;
    const float ks = a.k_scale[cell] * a.scale, vs = a.v_scale[cell];
    const int keys = count - p * a.P < a.P ? count - p * a.P : a.P;
    for (int i = 0; i < keys; ++i) {
      const int64_t off = (cell * a.P + i) * a.D + lane * 8;
      float dot = 0.f;
      if (on) {
        const uint2 k = *reinterpret_cast<const uint2*>(a.k_cache + off);
        const uint32_t c[4] = {k.x, k.x >> 16, k.y, k.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = decode2<FMT>(c[e]);
          dot += q[2 * e] * x.x;
          dot += q[2 * e + 1] * x.y;
        }
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
      const float s = dot * ks;
      const float m2 = fmaxf(m, s), m2s = m2 == -INFINITY ? 0.f : m2;
      const float alpha = __expf(m - m2s), pr = __expf(s - m2s);
      m = m2;
      l = l * alpha + pr;
      if (on) {
        const uint2 v = *reinterpret_cast<const uint2*>(a.v_cache + off);
        const uint32_t c[4] = {v.x, v.x >> 16, v.y, v.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = decode2<FMT>(c[e]);
          o[2 * e] = o[2 * e] * alpha + pr * vs * x.x;
          o[2 * e + 1] = o[2 * e + 1] * alpha + pr * vs * x.y;
        }
      }
    }
  }
  if (on) {
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no keys: 0; NaN stays
#pragma unroll
    for (int e = 0; e < 8; ++e)
      a.out[(r * a.Q + h) * a.D + lane * 8 + e] =
          __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
  }
  if (lane == 0) {
    if (a.lse) a.lse[r * a.Q + h] = l == 0.f ? -INFINITY : m + __logf(l);
    if (bits) atomicOr(a.status, bits);
  }
}

}  // namespace

cudaError_t launch_kv_attn(const KvAttnArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.B * a.T * a.Q;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  if (a.format == kKvE4m3)
    kv_attn_simple<kKvE4m3><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    kv_attn_simple<kKvInt8><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace idx
