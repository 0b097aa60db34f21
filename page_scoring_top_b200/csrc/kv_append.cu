// kv_append.cu -- new keys and values into the 8-bit paged cache.
//
// A page (of one kv head, K and V apart) has one scale s, a power of two with
// QMAX * s >= every |x| stored under it.  Appending rows takes the rows'
// largest finite magnitude a, s' = 2^e with the least e that fits a, and, when
// the page holds older rows, s' = max(s, s'); if that raises the scale, the
// older rows' codes become rne(code * s / s'); the new rows' codes are
// rne(x / s').  The scales are powers of two because pages grow a token at a
// time: x / s' is then exact before its one rounding, and a growing scale
// moves e4m3 codes without a rounding while they stay in the code's normal
// range: those do not depend on how the tokens were cut into calls.  int8 codes,
// and e4m3 codes that become subnormal, are rounded again at each growth; as a
// growth at least halves the error before it, an int8 code stays less than one
// step from x / s' (1/2 + 1/4 + ...), and within one step of the code that one
// call would have written.  The price of the powers of two is at most one binade
// of the codes' range, which costs e4m3 (a float) nothing in relative precision
// and int8 at most one bit.
//
// A run is the rows of one call that continue one another in one page; its
// first row leads it.  A CTA (window of rows, kv head, K or V) handles the runs
// that start in its window, which its warps find from two loads per row and a
// ballot.  A warp takes a short run alone (single tokens: the warps of the CTA
// work on different rows and never wait for each other); the CTA takes a long
// one together.  The rows stay in registers between the maximum and the
// rounding (up to kKeep pieces a thread; more are read again, from the L2).
//
// What bounds it: HBM for prompts (2 D bytes in, D out per row and head; 16384
// tokens of 8 heads x 128: int8 24 us, 4.2 TB/s, e4m3 27 us), latency for single
// tokens (256 tokens: 8 us, replayed in a graph).
#include "kv.cuh"

namespace idx {

namespace {

constexpr int kAppWarps = 4;
constexpr int kAppThreads = kAppWarps * 32;
constexpr int kKeep = 8;       // 16-byte pieces of a run that a thread keeps
constexpr int kAppShort = 4;   // rows of a run that a warp takes alone

// The largest of the magnitudes of eight bf16 values and of m, as two 16-bit
// halves of their bits (sign removed: bit order is magnitude order, and what is
// not finite comes last).
__device__ __forceinline__ uint32_t piece_max(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// The same with what is not finite left out.
__device__ __forceinline__ uint32_t piece_max_finite(uint32_t m, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
    m = __vmaxu2(m, (lo < 0x7F80u ? lo : 0u) | (hi < 0x7F80u ? hi << 16 : 0u));
  }
  return m;
}

// Eight bf16 values over the scale sc as codes.  A scale of another producer
// need not be a power of two (inv then has a rounding of its own): divide.
// int8 in the common case (finite values, a power of two): adding 1.5 * 2^23
// rounds x / sc to the nearest integer, ties to even, in the sum's low byte.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const uint4& v, float sc, float inv, bool pow2, bool finite) {
  if (FMT == kKvInt8 && pow2 && finite) {
    auto at = [&](uint32_t w, bool high) {
      const float x = __uint_as_float(high ? w & 0xFFFF0000u : w << 16);
      return __float_as_uint(fmaf(x, inv, 12582912.f));
    };
    auto four = [&](uint32_t a, uint32_t b) {
      return __byte_perm(__byte_perm(at(a, false), at(a, true), 0x0040),
                         __byte_perm(at(b, false), at(b, true), 0x0040), 0x5410);
    };
    return make_uint2(four(v.x, v.y), four(v.z, v.w));
  }
  auto two = [&](uint32_t w) {
    const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
    return pow2 ? encode2<FMT>(lo * inv, hi * inv)
                : encode2<FMT>(__fdiv_rn(lo, sc), __fdiv_rn(hi, sc));
  };
  return make_uint2(two(v.x) | (two(v.y) << 16), two(v.z) | (two(v.w) << 16));
}

// One side (K or V) of one head of the cache.
struct Side {
  const uint16_t* x;  // the head's columns of row 0
  int64_t ldx;
  uint8_t* cache;
  float* scales;
};

// The n rows from t on into page `page` from row off on, by the CTA or a warp.
template <int FMT, bool CTA>
__device__ __forceinline__ void append_run(const KvAppendArgs& a, const Side& sd, int h, int t, int page,
                                           int off, int n, uint32_t* s_max) {
  const int idx = CTA ? threadIdx.x : (threadIdx.x & 31);
  constexpr int kThreads = CTA ? kAppThreads : 32;
  const int nch = a.D / 8;            // 8-element pieces of a row
  const int rpp = kThreads / nch;     // rows per pass
  const int row = idx / nch, ch = idx - row * nch;
  const bool active = row < rpp;
  const int64_t cell = (int64_t)page * a.H + h;
  const float s_old = off ? sd.scales[cell] : 0.f;
  const uint16_t* src = sd.x + (int64_t)t * sd.ldx + ch * 8;
  uint4 keep[kKeep];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = k * rpp + row;
    keep[k] = (active && i < n) ? __ldg(reinterpret_cast<const uint4*>(src + i * sd.ldx))
                                : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kKeep; ++k) m = piece_max(m, keep[k]);
  if (active)
    for (int i = kKeep * rpp + row; i < n; i += rpp)
      m = piece_max(m, __ldg(reinterpret_cast<const uint4*>(src + i * sd.ldx)));
  auto all = [&](uint32_t v, uint32_t* s) {  // over the halves and the threads
    v = (v & 0xFFFFu) > (v >> 16) ? (v & 0xFFFFu) : (v >> 16);
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (CTA) {
      if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kAppWarps; ++w) v = v > s[w] ? v : s[w];
    }
    return v;
  };
  m = all(m, s_max);
  const bool finite = m < 0x7F80u;
  if (!finite) {  // rare: again without infinities and NaN
    m = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) m = piece_max_finite(m, keep[k]);
    if (active)
      for (int i = kKeep * rpp + row; i < n; i += rpp)
        m = piece_max_finite(m, __ldg(reinterpret_cast<const uint4*>(src + i * sd.ldx)));
    m = all(m, s_max + 2 * kAppWarps);
  }
  const int e = scale_exp<FMT>(m);
  float sc = pow2f(e), inv = pow2f(-e);
  if (off) {
    if (s_old >= sc) {
      sc = s_old;
      inv = __fdiv_rn(1.f, sc);
    } else {  // the page's scale grows: its older rows move under it
      const float f = __fdiv_rn(s_old, sc);
      uint4* old = reinterpret_cast<uint4*>(sd.cache + cell * a.P * a.D);
      for (int i = idx; i < off * (a.D / 16); i += kThreads) {
        const uint4 w = old[i];
        auto move = [&](uint32_t c) {
          const float2 lo = decode2<FMT>(c), hi = decode2<FMT>(c >> 16);
          return encode2<FMT>(lo.x * f, lo.y * f) | (encode2<FMT>(hi.x * f, hi.y * f) << 16);
        };
        old[i] = make_uint4(move(w.x), move(w.y), move(w.z), move(w.w));
      }
    }
  }
  if (idx == 0) sd.scales[cell] = sc;  // every thread has read the old one: the maximum came between
  const bool pow2 = (__float_as_uint(sc) & 0x7FFFFFu) == 0;
  uint8_t* dst = sd.cache + (cell * a.P + off) * a.D + ch * 8;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = k * rpp + row;
    if (active && i < n)
      *reinterpret_cast<uint2*>(dst + (int64_t)i * a.D) = encode8<FMT>(keep[k], sc, inv, pow2, finite);
  }
  if (active)
    for (int i = kKeep * rpp + row; i < n; i += rpp)
      *reinterpret_cast<uint2*>(dst + (int64_t)i * a.D) =
          encode8<FMT>(__ldg(reinterpret_cast<const uint4*>(src + i * sd.ldx)), sc, inv, pow2, finite);
}

template <int FMT>
__global__ void __launch_bounds__(kAppThreads, 7) kv_append_kernel(const KvAppendArgs a, int window) {
  __shared__ uint32_t s_max[4][kAppWarps];  // two runs' maxima, all and finite
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const Side sd = {(is_v ? a.v : a.k) + (int64_t)h * a.D, is_v ? a.ldv : a.ldk,
                   is_v ? a.v_cache : a.k_cache, is_v ? a.v_scale : a.k_scale};
  const int n_slots = a.n_blocks * a.P;
  const int t0 = blockIdx.x * window;
  // every warp looks at the whole window, a row a lane
  const int t = t0 + lane;
  const bool in = lane < window && t < a.R;
  const int s = in ? __ldg(a.slots + t) : -1;
  const int before = in && t > 0 ? __ldg(a.slots + t - 1) : -1;
  const bool valid = s >= 0 && s < n_slots;
  if (!valid && s != -1 && wid == 0 && h == 0 && !is_v) atomicOr(a.status, kErrPageClamped);
  const int page = valid ? s / a.P : 0, off = valid ? s - page * a.P : 0;
  const bool goes_on = valid && off != 0 && before == s - 1;
  const uint32_t on = __ballot_sync(0xFFFFFFFFu, goes_on);
  uint32_t lead = __ballot_sync(0xFFFFFFFFu, valid && !goes_on);
  int shorts = 0, longs = 0;
  while (lead) {
    const int j = __ffs(lead) - 1;
    lead &= lead - 1;
    const int rs = __shfl_sync(0xFFFFFFFFu, s, j), rp = __shfl_sync(0xFFFFFFFFu, page, j);
    const int ro = __shfl_sync(0xFFFFFFFFu, off, j);
    // the run's rows in the window, then behind it
    const uint32_t rest = j < 31 ? ~(on >> (j + 1)) : 0xFFFFFFFFu;
    int n = rest ? __ffs(rest) : 32 - j;
    if (j + n == window) {
      const int most = a.P - ro < a.R - t0 - j ? a.P - ro : a.R - t0 - j;
      while (n < most) {
        const bool same = n + lane < most && __ldg(a.slots + t0 + j + n + lane) == rs + n + lane;
        const uint32_t miss = ~__ballot_sync(0xFFFFFFFFu, same);
        n += miss ? __ffs(miss) - 1 : 32;
        if (miss) break;
      }
    }
    if (n <= kAppShort) {
      if (shorts++ % kAppWarps == wid) append_run<FMT, false>(a, sd, h, t0 + j, rp, ro, n, nullptr);
    } else {  // (the other buffer: a warp may still read the last run's)
      append_run<FMT, true>(a, sd, h, t0 + j, rp, ro, n, s_max[longs++ & 1]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  // The window is as long as leaves enough CTAs to fill the GPU, from a row per
  // warp (a batch of single tokens) to a row per lane.
  int window = kAppWarps;
  while (window < 32 && (int64_t)a.R * a.H * 2 / (2 * window) >= 2368) window *= 2;
  const dim3 grid((a.R + window - 1) / window, a.H, 2);
  if (a.format == kKvE4m3)
    kv_append_kernel<kKvE4m3><<<grid, kAppThreads, 0, stream>>>(a, window);
  else
    kv_append_kernel<kKvInt8><<<grid, kAppThreads, 0, stream>>>(a, window);
  return cudaGetLastError();
}

}  // namespace idx
