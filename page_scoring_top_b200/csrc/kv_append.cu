// kv_append.cu -- new keys and values into the 8-bit paged cache.
//
// A page (of one kv head, K and V apart) has one scale s, a power of two with
// QMAX * s >= every |x| stored under it.  Appending rows takes the rows'
// largest finite magnitude a, s' = 2^e with the least e that fits a, and, when
// the page holds older rows, s' = max(s, s'); if that raises the scale, the
// older rows' codes become rne(code * s / s'); the new rows' codes are
// rne(x / s').  The scales are powers of two because pages grow a token at a
// time: x / s' is then exact before its one rounding, and a growing scale
// moves e4m3 codes without a rounding (down to the code's subnormals), so the
// cache does not depend on how the tokens were cut into calls.  The price is
// at most one binade of the codes' range, which costs e4m3 (a float) nothing
// in relative precision and int8 at most one bit.
//
// A run is the rows of one call that continue one another in one page; its
// first row leads it.  CTA (window of rows, kv head, K or V) handles the runs
// that start in its window, one after the other, reading each row once: the
// rows stay in registers between the maximum and the rounding (up to kKeep
// passes of the CTA; longer runs read the rest again, from the L2).
//
// What bounds it: HBM for prompts (2 D bytes in, D out per row and head),
// latency for single tokens.
#include "kv.cuh"

namespace idx {

namespace {

constexpr int kAppThreads = 128;
constexpr int kAppWindow = 16;
constexpr int kKeep = 8;  // 16-byte pieces of the run that a thread keeps

// The larger of two bf16 magnitudes (sign removed, inf and NaN counted as 0), per half.
__device__ __forceinline__ uint32_t finite_max2(uint32_t m, uint32_t w) {
  w &= 0x7FFF7FFFu;
  if ((w & 0xFFFFu) >= 0x7F80u) w &= 0xFFFF0000u;
  if ((w >> 16) >= 0x7F80u) w &= 0xFFFFu;
  return __vmaxu2(m, w);
}

__device__ __forceinline__ uint32_t piece_max(uint32_t m, const uint4& v) {
  m = finite_max2(m, v.x);
  m = finite_max2(m, v.y);
  m = finite_max2(m, v.z);
  return finite_max2(m, v.w);
}

// Eight bf16 values over the scale sc as codes.  A scale of another producer
// need not be a power of two (inv then has a rounding of its own): divide.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& v, float sc, float inv, bool pow2) {
  auto two = [&](uint32_t w) {
    const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
    return pow2 ? encode2<FMT>(lo * inv, hi * inv)
                : encode2<FMT>(__fdiv_rn(lo, sc), __fdiv_rn(hi, sc));
  };
  return make_uint2(two(v.x) | (two(v.y) << 16), two(v.z) | (two(v.w) << 16));
}

template <int FMT>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const KvAppendArgs a, int window) {
  __shared__ uint32_t s_max[2][kAppThreads / 32];
  __shared__ int s_len[2];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const uint16_t* x = (is_v ? a.v : a.k) + (int64_t)h * a.D;
  const int64_t ldx = is_v ? a.ldv : a.ldk;
  uint8_t* cache = is_v ? a.v_cache : a.k_cache;
  float* scales = is_v ? a.v_scale : a.k_scale;
  const int nch = a.D / 8;                  // 8-element pieces of a row
  const int rpp = kAppThreads / nch;        // rows per pass of the CTA
  const int row = tid / nch, ch = tid - row * nch;
  const bool active = row < rpp;
  const int n_slots = a.n_blocks * a.P;
  const int t0 = blockIdx.x * window;
  const int t1 = t0 + window < a.R ? t0 + window : a.R;
  int prev = t0 > 0 ? __ldg(a.slots + t0 - 1) : -1;
  int buf = 0;
  for (int t = t0; t < t1; ++t) {
    const int s = __ldg(a.slots + t);
    const int before = prev;
    prev = s;
    if (s < 0 || s >= n_slots) {
      if ((s < -1 || s >= n_slots) && tid == 0 && h == 0 && !is_v)
        atomicOr(a.status, kErrPageClamped);
      continue;
    }
    const int page = s / a.P, off = s - page * a.P;
    if (off != 0 && before == s - 1) continue;  // not the first row of its run
    // the run: rows t .. t+n-1 at slots s .. s+n-1 of this page
    const int most = a.P - off < a.R - t ? a.P - off : a.R - t;
    if (tid == 0) s_len[buf] = most;
    __syncthreads();
    for (int i = tid; i < most; i += kAppThreads)
      if (__ldg(a.slots + t + i) != s + i) {
        atomicMin(&s_len[buf], i);
        break;
      }
    const int64_t cell = (int64_t)page * a.H + h;
    const float s_old = off ? scales[cell] : 0.f;
    __syncthreads();
    const int n = s_len[buf];
    const uint16_t* src = x + (int64_t)t * ldx + ch * 8;
    uint4 keep[kKeep];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int i = k * rpp + row;
      keep[k] = (active && i < n) ? __ldg(reinterpret_cast<const uint4*>(src + i * ldx))
                                  : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k) m = piece_max(m, keep[k]);
    if (active)
      for (int i = kKeep * rpp + row; i < n; i += rpp)
        m = piece_max(m, __ldg(reinterpret_cast<const uint4*>(src + i * ldx)));
    m = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) s_max[buf][wid] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppThreads / 32; ++w) m = m > s_max[buf][w] ? m : s_max[buf][w];
    const int e = scale_exp<FMT>(m);
    float sc = pow2f(e), inv = pow2f(-e);
    if (off) {
      if (s_old >= sc) {
        sc = s_old;
        inv = __fdiv_rn(1.f, sc);
      } else {  // the page's scale grows: its older rows move under it
        const float f = __fdiv_rn(s_old, sc);
        uint4* old = reinterpret_cast<uint4*>(cache + cell * a.P * a.D);
        for (int i = tid; i < off * (a.D / 16); i += kAppThreads) {
          uint4 w = old[i];
          auto move = [&](uint32_t c) {
            const float2 lo = decode2<FMT>(c), hi = decode2<FMT>(c >> 16);
            return encode2<FMT>(lo.x * f, lo.y * f) | (encode2<FMT>(hi.x * f, hi.y * f) << 16);
          };
          old[i] = make_uint4(move(w.x), move(w.y), move(w.z), move(w.w));
        }
      }
    }
    if (tid == 0) scales[cell] = sc;
    const bool pow2 = (__float_as_uint(sc) & 0x7FFFFFu) == 0;
    uint8_t* dst = cache + (cell * a.P + off) * a.D + ch * 8;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int i = k * rpp + row;
      if (active && i < n)
        *reinterpret_cast<uint2*>(dst + (int64_t)i * a.D) = encode8<FMT>(keep[k], sc, inv, pow2);
    }
    if (active)
      for (int i = kKeep * rpp + row; i < n; i += rpp)
        *reinterpret_cast<uint2*>(dst + (int64_t)i * a.D) =
            encode8<FMT>(__ldg(reinterpret_cast<const uint4*>(src + i * ldx)), sc, inv, pow2);
    buf ^= 1;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  // One row per CTA while that is not many CTAs (single tokens: each row leads
  // its own run); windows of rows beyond, where most rows continue a run.
  const int64_t per_row = (int64_t)a.R * a.H * 2;
  const int window = per_row <= 16384 ? 1 : kAppWindow;
  const dim3 grid((a.R + window - 1) / window, a.H, 2);
  if (a.format == kKvE4m3)
    kv_append_kernel<kKvE4m3><<<grid, kAppThreads, 0, stream>>>(a, window);
  else
    kv_append_kernel<kKvInt8><<<grid, kAppThreads, 0, stream>>>(a, window);
  return cudaGetLastError();
}

}  // namespace idx
