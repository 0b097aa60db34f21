// kv_attn_tc.cu -- attention over the 8-bit KV cache for many query rows per
// key: tokens of one request that share its keys (prompts, chunks of tokens).
//
// The formulas are those of kv_attn.cuh: x_i = s_i log2(e) + log2(vs_i),
// weights p_i = 2^(x_i - m), O = sum p_i v8_i, l = sum p_i / vs_i, out = O / l.
// With 128 query rows (tokens x heads of one kv head) a key's codes are used
// for 128 rows, which is work for the tcgen05 tensor cores: per tile of 128
// keys S = Q K^T and O += P V, both M = 128, fp16 operands (codes are exact in
// fp16, bf16 queries down to 2^-31 of a row's largest, under a power of two per
// row), fp32 accumulators in TMEM.
//
// What bounds it: at one key head and 128 rows a tile costs 1024 cycles of the
// tensor cores, 1024 of the exponent unit (128 x 128 at 16 a cycle) and, when
// its keys come from HBM, 1400 of the memory; so the kernel is built to keep
// all of them busy at once:
//  * three producer warps: block table look-ups, TMA copies of the codes into a
//    ring of five 64-key stages for K and one for V, scales of the tile's keys;
//  * two converter warpgroups, one for K and one for V: codes -> fp16 operands
//    (128-byte swizzled; K as K-major, one buffer; V as it lies, keys by rows: the
//    B operand in its MN-major form, so nothing is transposed, two buffers);
//    the first also writes the queries at an item's start;
//  * one MMA warp: S of tile n into one of two TMEM buffers, then O += P V of
//    tile n - 1;
//  * two softmax warpgroups take alternate tiles, a thread per query row, with
//    a running maximum, a sum and an accumulator of their own (joined at the
//    item's end), so that neither waits for the other's rescaling; the weights
//    go back to TMEM as the A operand, over the scores they come from.  The
//    reference m is the maximum less 7, and moved (and the accumulator rescaled)
//    only when that exceeds it by 8: weights are at most 2^15, within fp16, and
//    the largest at least 2^7, so that those down to 2^-21 of it are held to
//    2^-11 of their own size and smaller ones to 2^-32 of the largest.
//
// Measured: 4 requests x 16 tokens x 64 heads over 24-32 k keys 190 us, 2 x 1024
// tokens x 32 heads over up to 8192 keys 438 us (0.31 PFLOP/s): bound by the chain
// scores, maximum, weights, product of the two streams (a tile takes an SM 4.1 us,
// with two under way) and, in it, by instruction fetch: the same loops with their
// roles in another order measured 406 to 472 us.
//
// TMEM, 512 columns: S0 S1 O0 O1, 128 each; weights in the first half of S.
// The split over the SMs and the joining of cut items are those of kv_attn.cuh,
// in tiles of 128 keys.  Keys lie in the order of their positions here (no page
// lists), so a row sees a prefix of them.  Values that no row sees are zeroed on
// conversion; a NaN value that only some rows see is zeroed too and noted by
// column with the first position it is at: a row gets NaN where that is below
// its own count.
#include <cudaTypedefs.h>

#include "kv_attn.cuh"

namespace idx {

namespace {

constexpr int kTkThreads = 640;
constexpr int kTkSoft = 256;       // softmax threads
constexpr int kTkKeys = 128;       // keys per tile
constexpr int kTkRows = 128;
constexpr int kTkHalf = 64;        // keys of a copied stage
constexpr int kTkStages = 5;       // stages of the rings of K and of V
constexpr int kTkCharge = 4;       // tiles that an item's start and end count for
constexpr int kTkMeta = 6;         // tiles whose scales are held: up to five are in the pipeline
constexpr float kTkLift = 7.f;     // log2 of the largest weight when the reference is moved
constexpr float kTkSlack = 8.f;    // log2 by which a row may exceed that before it is moved again
constexpr float kTkLarge = 8388608.f;  // exponents from here on take the long way

template <int DP, bool PERKEY>
struct TkLayout {
  static constexpr int kOp = kTkKeys * DP * 2;        // bytes of a 128-row operand
  static constexpr int kRaw = kTkHalf * DP;           // bytes of half a tile's codes
  static constexpr int kPer = PERKEY ? kTkKeys : 4;   // scale entries of a tile
  static constexpr size_t bars = 0;                   // 38 barriers
  static constexpr size_t misc = 384;                 // 64 ints
  static constexpr size_t rows = misc + 256;          // factor, limit (two items'); m, l of two streams
  static constexpr size_t nanpos = rows + 2 * 128 * 8 + 512 * 4;  // first position of a NaN per column
  static constexpr size_t meta = nanpos + 2 * 128 * 4;
  static constexpr size_t q = (meta + (size_t)kTkMeta * kPer * sizeof(KvPage) + 1023) & ~(size_t)1023;
  static constexpr size_t k16 = q + kOp;
  static constexpr size_t v16 = k16 + kOp;
  static constexpr size_t raw = v16 + 2 * kOp;
  static constexpr size_t total = raw + (size_t)2 * kTkStages * kRaw + 1024;
  static_assert(total <= kKvSmem, "shared memory");
};

struct TkPlan {
  int TT, ntb, GG, ng;
  int hb;            // rows of a copy: all in one page
  float* ws;
  int32_t* arrive;
};

__device__ __forceinline__ void tk_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// kind::f16, f16 x f16 -> f32, M = 128; the B operand K-major or MN-major.
constexpr uint32_t tk_idesc(int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// MN-major, 128-byte swizzle: 64-column blocks `lbo` bytes apart, 8-key groups 1024.
__device__ __forceinline__ uint64_t tk_desc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

__device__ __forceinline__ void tk_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
      "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tk_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tk_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One CTA's part of an item.
struct TkSeg {
  int64_t unit0;
  int nt, t0, t1;      // the item's tiles; this part's
  int b, tk, nrow, h0, nh, g;
  int max_count, min_count;
};

// A whole warp's walk over the CTA's parts (every role walks by itself).
struct TkWalk {
  const KvAttnArgs& a;
  const TkPlan& pl;
  int64_t rt, base, u, u_end;
  int items, nt, mx, mn;
  bool have;
  __device__ TkWalk(const KvAttnArgs& a_, const TkPlan& pl_, const int64_t* where, int64_t u0, int64_t u1)
      : a(a_), pl(pl_), rt(where[0]), base(where[1]), u(u0), u_end(u1), items(a_.H * pl_.ng), have(false) {}
  __device__ bool next(TkSeg& s, int& bits) {
    while (u < u_end) {
      const int b = (int)(rt / pl.ntb), tk = (int)(rt - (int64_t)b * pl.ntb) * pl.TT;
      const int ntok = a.T - tk < pl.TT ? a.T - tk : pl.TT;
      if (!have) {
        int x = 0, n = INT32_MAX;
        for (int t = threadIdx.x & 31; t < ntok; t += 32) {
          const int c = kv_count(a, (int64_t)b * a.T + tk + t, bits);
          x = c > x ? c : x;
          if (c > 0 && c < n) n = c;
        }
        mx = __reduce_max_sync(0xFFFFFFFFu, x);
        mn = __reduce_min_sync(0xFFFFFFFFu, n);
        nt = mx > kTkKeys ? (mx + kTkKeys - 1) / kTkKeys : 1;
        have = true;
      }
      const int64_t n = nt + kTkCharge, end = base + n * items;
      if (u >= end) {
        base = end;
        ++rt;
        have = false;
        continue;
      }
      const int it = (int)((u - base) / n);
      const int64_t x0 = (u - base) - it * n;
      const int64_t x1 = n - x0 < u_end - u ? n : x0 + (u_end - u);
      u += x1 - x0;
      s.t0 = x0 <= kTkCharge ? 0 : (int)(x0 - kTkCharge);
      s.t1 = x1 <= kTkCharge ? 0 : (int)(x1 - kTkCharge);
      if (s.t1 == s.t0) continue;
      s.unit0 = base + it * n + kTkCharge;
      s.nt = nt;
      s.b = b;
      s.tk = tk;
      s.g = it / pl.ng;
      const int G = a.Q / a.H, hg = it - s.g * pl.ng;
      s.nh = G - hg * pl.GG < pl.GG ? G - hg * pl.GG : pl.GG;
      s.nrow = ntok * s.nh;
      s.h0 = s.g * G + hg * pl.GG;
      s.max_count = mx;
      s.min_count = mn;
      return true;
    }
    return false;
  }
};

template <int FMT, int DP, bool PERKEY>
__global__ void __launch_bounds__(kTkThreads, 1)
    kv_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const KvAttnArgs a, const TkPlan pl) {
  using L = TkLayout<DP, PERKEY>;
  constexpr int NS = kTkStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  // rings of K and V: [2][NS]; buffers and streams: [2]
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t *raw_empty = raw_full + 2 * NS, *k_full = raw_empty + 2 * NS, *k_empty = k_full + 1,
           *v_full = k_empty + 1, *v_empty = v_full + 2, *s_full = v_empty + 2, *p_full = s_full + 2,
           *o_done = p_full + 2, *q_full = o_done + 2, *q_empty = q_full + 2, *o_free = q_empty + 1,
           *m_done = o_free + 2;
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* s_abort = misc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
  int* s_flag = misc + 2;
  volatile uint32_t* s_turn = reinterpret_cast<volatile uint32_t*>(misc + 4);  // next tile to be fetched
  int64_t* s_where = reinterpret_cast<int64_t*>(misc + 8);  // row tile, units before it
  int* s_part = misc + 12;  // copied stages of the first tile that was not fetched whole
  long long* s_warp = reinterpret_cast<long long*>(misc + 24);
  float* s_qf = reinterpret_cast<float*>(smem + L::rows);
  int* s_lim = reinterpret_cast<int*>(s_qf + 256);
  float* s_ml = reinterpret_cast<float*>(s_lim + 256);  // m of streams 0, 1, then l
  int* s_nan = reinterpret_cast<int*>(smem + L::nanpos);
  KvPage* pages = reinterpret_cast<KvPage*>(smem + L::meta);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.H * pl.ng;
  const int64_t nrt = (int64_t)a.B * pl.ntb;
  int bits = 0;

  // ---- the split (as in kv_attn.cuh, in tiles)
  auto tiles = [&](int64_t rt) {
    const int b = (int)(rt / pl.ntb), t0 = (int)(rt - (int64_t)b * pl.ntb) * pl.TT;
    const int n = a.T - t0 < pl.TT ? a.T - t0 : pl.TT;
    int mx = 0;
    for (int t = 0; t < n; ++t) {
      const int c = kv_count(a, (int64_t)b * a.T + t0 + t, bits);
      mx = c > mx ? c : mx;
    }
    return (mx > kTkKeys ? (mx + kTkKeys - 1) / kTkKeys : 1) + kTkCharge;
  };
  const int64_t per = (nrt + kTkThreads - 1) / kTkThreads;
  const int64_t rt0 = tid * per < nrt ? tid * per : nrt;
  const int64_t rt1 = rt0 + per < nrt ? rt0 + per : nrt;
  if (tid == 0) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  long long mine = 0;
  for (int64_t rt = rt0; rt < rt1; ++rt) mine += tiles(rt);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid < 256) s_nan[tid] = INT32_MAX;
  if (tid == 0) {
    *s_abort = IDX_KV_GIVE_UP;
    *s_turn = 0;
    *s_part = 0;
    for (int i = 0; i < 2 * NS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    mbar_init(k_full, 4);
    mbar_init(k_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&o_free[i], 8);
    }
    mbar_init(q_empty, 1);
    mbar_init(m_done, 1);
    fence_mbar_init();
  }
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kTkThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  before += incl - mine;
  const int64_t W = total * items;
  int64_t nc = W / (2 + kTkCharge);
  nc = nc < 1 ? 1 : (nc < (int64_t)gridDim.x ? nc : (int64_t)gridDim.x);
  if ((int64_t)blockIdx.x >= nc) return;
  const int64_t u_begin = W * blockIdx.x / nc, u_end = W * (blockIdx.x + 1) / nc;
  {
    long long base = before * items;
    if (u_begin < base + mine * items && u_end > base)
      for (int64_t rt = rt0; rt < rt1; ++rt) {
        const int64_t n = tiles(rt);
        if (u_begin >= base && u_begin < base + n * items) {
          s_where[0] = rt;
          s_where[1] = base;
        }
        base += n * items;
      }
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TkWalk walk(a, pl, s_where, u_begin, u_end);
  TkSeg sg;

  // The launch's 96 registers a thread: 256 x 136 + 256 x 64 + 128 x 72 <= 640 x 96.
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp != 17) {
      // ================================================================ producers
      // Three warps take the tiles in turns, so that three chains of look-ups
      // are under way; the copies are issued in the order of the tiles.
      const uint32_t pw = warp == 16 ? 0 : warp - 17;
      const int copies = kTkKeys / pl.hb;
      const int oob = a.n_blocks * a.H * a.P;  // a row past the cache: reads zeros
      constexpr int NE = PERKEY ? 4 : 1;       // scale entries a lane looks up
      constexpr int KE = kTkKeys / L::kPer;    // keys of an entry
      uint32_t n = 0;                          // tiles so far
      bool ok = true;
      while (ok && walk.next(sg, bits)) {
        for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
          if (n % 3 != pw) continue;
          // the block of a position, -1 where there is no key to see
          auto block_of = [&](int pos) {
            if (pos >= sg.max_count) return -1;
            const int id = __ldg(a.page_table + (int64_t)sg.b * a.ld_pt + pos / a.P);
            if (id >= 0 && id < a.n_blocks) return id;
            bits |= kErrPageClamped;
            return -1;
          };
          int row[NE];
          KvPage x[NE];
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const int c = i * 32 + lane;
            row[i] = oob;
            if (c < copies) {
              const int pos = t * kTkKeys + c * pl.hb, id = block_of(pos);
              if (id >= 0) row[i] = (int)(((int64_t)id * a.H + sg.g) * a.P) + pos % a.P;
            }
            x[i] = KvPage{0.f, -INFINITY, 0.f, 1.f};
            if (c < L::kPer) {
              const int id = block_of(t * kTkKeys + c * KE);
              if (id >= 0) {
                const int64_t cell = (int64_t)id * a.H + sg.g;
                x[i] = kv_scales(__ldg(a.k_scale + cell), __ldg(a.v_scale + cell));
              }
            }
          }
          bool got = false;
          for (uint32_t i = 0; i < kMaxWaitIters && !got && !*s_abort; ++i) {
            got = *s_turn == n;
            if (!got) __nanosleep(40);
          }
          ok = __all_sync(0xFFFFFFFFu, got);
          if (!ok) {
            if (!*s_abort && lane == 0) {
              *s_abort = 1;
              atomicOr(a.status, kErrWaitTimeout);
            }
            break;
          }
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) {  // halves of K, halves of V
            const int kv = i2 >> 1, half = i2 & 1;
            const uint32_t r = 2 * n + half, st = kv * NS + r % NS, ph = (r / NS) & 1;
            ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&raw_empty[st], ph ^ 1, s_abort, a.status));
            if (!ok) {
              if (lane == 0) *s_part = i2;
              break;
            }
            if (i2 == 0) {
#pragma unroll
              for (int i = 0; i < NE; ++i)
                if (i * 32 + lane < L::kPer) pages[(size_t)(n % kTkMeta) * L::kPer + i * 32 + lane] = x[i];
              __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], L::kRaw);
            __syncwarp();
            unsigned char* dst = smem + L::raw + (size_t)st * L::kRaw;
            const int first = half * (copies / 2);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
              const int c = i * 32 + lane - first;
              if (c >= 0 && c < copies / 2)
                tma_load_2d(dst + c * pl.hb * DP, kv ? &map_v : &map_k, 0, row[i], &raw_full[st]);
            }
            __syncwarp();
          }
          __threadfence_block();
          if (ok && lane == 0) *s_turn = n + 1;
        }
      }
      // The copies end before the CTA does, whether or not they are still
      // waited for: of each stage the latest, its earlier ones ended before it.
      asm volatile("bar.sync %0, 96;" ::"n"(kKvProducerBarrier) : "memory");
      if (pw == 0 && lane < 2 * NS) {
        const int kv = lane / NS, st = lane - kv * NS, part = *s_part;
        const int used = 2 * (int)*s_turn + (kv ? (part > 2 ? part - 2 : 0) : (part < 2 ? part : 2));
        if (used > st) mbar_wait_drain(&raw_full[lane], (uint32_t)((used - 1 - st) / NS) & 1);
      }
      if (bits) atomicOr(a.status, bits);
    } else if (warp == 17) {
      // ================================================================ MMA
      const uint32_t q_s = smem_u32(smem + L::q), k_s = smem_u32(smem + L::k16), v_s = smem_u32(smem + L::v16);
      constexpr uint32_t kBlk = kTkKeys * 128;  // bytes of a 64-column block
      uint32_t n = 0;
      int seg = 0;
      bool ok = true;
      auto await = [&](uint64_t* bar, uint32_t ph) {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_spin(bar, ph, s_abort, a.status));
        return ok;
      };
      auto pv = [&](uint32_t i, bool acc) {
        const uint32_t b = i & 1, ph = (i >> 1) & 1;
        if (!await(&v_full[b], ph) || !await(&p_full[b], ph)) return;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < kTkKeys / 16; ++k)
            tk_mma_ts(tmem + 256 + b * 128, tmem + b * 128 + k * 8,
                      tk_desc_mn(v_s + b * L::kOp + k * 2048, kBlk), tk_idesc(DP, true), acc || k > 0);
          umma_commit(&v_empty[b]);
          umma_commit(&o_done[b]);
        }
        __syncwarp();
      };
      while (ok && walk.next(sg, bits)) {
        if (!await(&q_full[seg & 1], (seg >> 1) & 1)) break;
        const uint32_t n0 = n, n1 = n + (sg.t1 - sg.t0);
        for (; n < n1 && ok; ++n) {
          const uint32_t b = n & 1;
          if (!await(k_full, n & 1)) break;
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              umma_bf16(tmem + b * 128, umma_desc_sw128(q_s + (k >> 2) * kBlk + (k & 3) * 32),
                        umma_desc_sw128(k_s + (k >> 2) * kBlk + (k & 3) * 32), tk_idesc(128, false),
                        k > 0);
            umma_commit(k_empty);
            umma_commit(&s_full[b]);
            if (n + 1 == n1) umma_commit(q_empty);
          }
          __syncwarp();
          if (n > n0) {
            if (n == n0 + 1 && seg > 0 && !await(&o_free[(seg - 1) & 1], ((seg - 1) >> 1) & 1)) break;
            pv(n - 1, n - 1 >= n0 + 2);
          }
        }
        if (!ok) break;
        if (n1 == n0 + 1 && seg > 0 && !await(&o_free[(seg - 1) & 1], ((seg - 1) >> 1) & 1)) break;
        pv(n1 - 1, n1 - 1 >= n0 + 2);
        ++seg;
      }
      // the products end before the TMEM that they write is freed, whether or
      // not their readers still wait for them
      if (lane == 0) umma_commit(m_done);
      __syncwarp();
      mbar_wait_drain(m_done, 0);
    }
  } else if (warp >= 8) {
    // ================================================================== converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int ct = tid & 127;       // within the warpgroup
    const int kv = (warp >> 2) - 2;  // the keys' or the values'
    uint32_t n = 0;
    int seg = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t ph) {
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, ph, s_abort, a.status));
      return ok;
    };
    while (ok && walk.next(sg, bits)) {
      // ---- queries: a thread per row, once the last item's scores are done;
      // factors, limits and NaN positions have the places of the item before
      if (kv == 0 && seg > 0 && !await(q_empty, (seg - 1) & 1)) break;
      if (seg > 1 && !await(&o_free[seg & 1], ((seg - 2) >> 1) & 1)) break;
      const int sb = (seg & 1) * 128;
      if (!kv) {
        const int m = ct;
        const bool use = m < sg.nrow;
        const int tt = use ? m / sg.nh : 0;
        const int64_t r = (int64_t)sg.b * a.T + sg.tk + tt;
        const uint16_t* src = a.q + r * a.ldq + (int64_t)(sg.h0 + m - tt * sg.nh) * a.D;
        auto piece = [&](int i) {
          return use && i * 8 < a.D ? __ldg(reinterpret_cast<const uint4*>(src + i * 8)) : make_uint4(0u, 0u, 0u, 0u);
        };
        uint32_t top = 0;
#pragma unroll 4
        for (int i = 0; i < DP / 8; ++i) {
          const uint4 v = piece(i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
            top = lo < 0x7F80u && lo > top ? lo : top;
            top = hi < 0x7F80u && hi > top ? hi : top;
          }
        }
        float f, inverse;
        query_factors((int)(top >> 7), f, inverse);
        unsigned char* row = smem + L::q + m * 128;
#pragma unroll 4
        for (int i = 0; i < DP / 8; ++i) {  // (again, from the L1)
          const uint4 v = piece(i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_f16(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
          *reinterpret_cast<uint4*>(row + (i >> 3) * (kTkRows * 128) + ((i & 7) ^ (m & 7)) * 16) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        s_qf[sb + m] = a.scale * 1.44269504088896340736f * inverse;
        s_lim[sb + m] = use ? kv_count(a, r, bits) : 0;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[seg & 1]);
      }
      for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
        const uint32_t b = n & 1;
        const int left = sg.max_count - t * kTkKeys;  // keys that some row sees
        // not all rows see all of the keys: values to be zeroed or noted
        const bool mixed = kv && (t + 1) * kTkKeys > sg.min_count;
        unsigned char* dst = smem + (kv ? L::v16 + b * L::kOp : L::k16);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t r = 2 * n + half, st = kv * NS + r % NS;
          if (!await(&raw_full[st], (r / NS) & 1)) break;
          if (half == 0 && !(kv ? await(&v_empty[b], ((n >> 1) & 1) ^ 1) : await(k_empty, (n & 1) ^ 1))) break;
          const unsigned char* src = smem + L::raw + (size_t)st * L::kRaw;
          // 16 codes a step, eight rows of a piece column side by side; a warp
          // takes 16 rows
          constexpr int PC = DP / 16;  // pieces of a row
          auto place = [&](int i, int& row, int& pc) {
            row = (warp & 3) * 16 + (i * 4 / PC) * 8 + (lane & 7);
            pc = ((i * 4) % PC + (lane >> 3)) % PC;
            const int at = DP == 64 ? (pc ^ ((row >> 1) & 3)) : (pc ^ (row & 7));
            const uint4 w = *reinterpret_cast<const uint4*>(src + row * DP + at * 16);
            row += half * kTkHalf;
            return w;
          };
          auto store = [&](const uint4& w, int row, int pc) {
            uint32_t o[8];
            codes4<FMT, false>(w.x, o[0], o[1]);
            codes4<FMT, false>(w.y, o[2], o[3]);
            codes4<FMT, false>(w.z, o[4], o[5]);
            codes4<FMT, false>(w.w, o[6], o[7]);
            unsigned char* d = dst + (pc >> 2) * (kTkKeys * 128) + row * 128;
            const int c2 = (pc & 3) * 2;
            *reinterpret_cast<uint4*>(d + ((c2 ^ (row & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(d + (((c2 + 1) ^ (row & 7)) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
          };
          if (!mixed) {  // (rolled: the roles' loops share the instruction cache)
#pragma unroll 1
            for (int i = 0; i < PC / 2; ++i) {
              int row, pc;
              const uint4 w = place(i, row, pc);
              store(w, row, pc);
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < PC / 2; ++i) {
              int row, pc;
              uint4 w = place(i, row, pc);
              if (row >= left) w = make_uint4(0u, 0u, 0u, 0u);
              if (FMT == kKvE4m3) {
                auto clean = [&](uint32_t c, int k) {
                  uint32_t hit = ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                  while (hit) {
                    const int y = (__ffs(hit) - 1) >> 3;
                    hit &= hit - 1;
                    atomicMin(&s_nan[sb + pc * 16 + k * 4 + y], t * kTkKeys + row);
                    c &= ~(0xFFu << (8 * y));
                  }
                  return c;
                };
                w = make_uint4(clean(w.x, 0), clean(w.y, 1), clean(w.z, 2), clean(w.w, 3));
              }
              store(w, row, pc);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[st]);
            if (half) mbar_arrive(kv ? &v_full[b] : k_full);
          }
        }
      }
      ++seg;
    }
  } else {
    // ===================================================================== softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    const int wg = warp >> 2, row = tid & 127;  // stream; query row
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 TMEM lanes
    const uint32_t s_t = lanes + wg * 128;
    uint32_t n = 0;
    int seg = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t ph) {
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, ph, s_abort, a.status));
      return ok;
    };
    while (walk.next(sg, bits)) {
      const uint32_t n0 = n, n1 = n + (sg.t1 - sg.t0);
      await(&q_full[seg & 1], (seg >> 1) & 1);
      const int sb = (seg & 1) * 128;
      const float qf = s_qf[sb + row];
      const int lim = s_lim[sb + row];
      float m = -INFINITY, l = 0.f;
      bool large = false;  // some row of the warp has a reference of 2^23 or more
      for (; n < n1 && ok; ++n) {
        if ((int)(n & 1) != wg) continue;
        const int t = sg.t0 + (int)(n - n0);
        if (!await(&s_full[wg], (n >> 1) & 1)) break;
        tc_fence_after();
        const KvPage* pg = pages + (size_t)(n % kTkMeta) * L::kPer;
        // every row sees every key (a negative softmax scale goes the long way)
        const bool all = (t + 1) * kTkKeys <= sg.min_count && a.scale >= 0.f;
        const int seen = lim - t * kTkKeys;  // keys that this row sees
        // the row's maximum; one scale and no mask: of the scores as they are
        float top = -INFINITY;
        auto maxima = [&](auto all_tag) {
          constexpr bool ALL = decltype(all_tag)::value;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32_nowait(s_t + c * 32, x);
            const KvPage e = pg[PERKEY ? 0 : c];
            tmem_ld_wait();
            float m0 = -INFINITY, m1 = -INFINITY;
            if (PERKEY || !ALL) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const KvPage k = PERKEY ? pg[PERKEY ? c * 32 + j : 0] : e;
                float v = fmaf(__uint_as_float(x[j]), k.ks * qf, k.lv);
                if (!ALL && c * 32 + j >= seen) v = -INFINITY;
                if (j & 1) m1 = fmaxf(m1, v);
                else m0 = fmaxf(m0, v);
              }
              top = max3(top, m0, m1);
            } else {  // the factor is not negative: the maximum of the scores as they are
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                m0 = max3(m0, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                m1 = max3(m1, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
              }
              top = fmaxf(top, fmaf(fmaxf(m0, m1), e.ks * qf, e.lv));
            }
          }
        };
        if (all) maxima(std::true_type());
        else maxima(std::false_type());
        top -= kTkLift;
        const bool move = top > m + kTkSlack || (m == -INFINITY && top > m);
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float m2 = move ? top : m;
          const float f = m2 == -INFINITY ? 1.f : ex2(m - m2);
          m = m2;
          l *= f;
          large = __any_sync(0xFFFFFFFFu, m2 != -INFINITY && fabsf(m2) >= kTkLarge);
          if (n >= n0 + 2) {  // the stream has an accumulator already
            if (!await(&o_done[wg], ((n >> 1) - 1) & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_nowait(lanes + 256 + wg * 128 + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tk_st32(lanes + 256 + wg * 128 + c * 32, o);
            }
          }
        }
        const float z = m == -INFINITY ? 0.f : m;
        // the weights, 16 columns for 32 scores, behind the scores still to read.
        // One addition for x - z leaves the rounding of x in the exponent; where
        // that may be large (2^23: half a step is 1/2), x is rounded as z was.
        auto weights = [&](auto all_tag) {
          constexpr bool ALL = decltype(all_tag)::value;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32], w[16];
            tmem_ld32_nowait(s_t + c * 32, x);
            const KvPage e = pg[PERKEY ? 0 : c];
            const float f = e.ks * qf, d = e.lv - z;
            tmem_ld_wait();
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float p[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float v = __uint_as_float(x[j + k]);
                if (PERKEY) {
                  const KvPage g = pg[PERKEY ? c * 32 + j + k : 0];
                  p[k] = ALL ? ex2(fmaf(v, g.ks * qf, g.lv - z)) : ex2(fmaf(v, g.ks * qf, g.lv) - z);
                  if (!ALL && c * 32 + j + k >= seen) p[k] = 0.f;
                  l = fmaf(p[k], g.iv, l);
                  p[k] *= g.rest;
                } else {
                  p[k] = ALL ? ex2(fmaf(v, f, d)) : ex2(fmaf(v, f, e.lv) - z);
                  if (!ALL && c * 32 + j + k >= seen) p[k] = 0.f;
                  (k ? s1 : s0) += p[k];
                }
              }
              if (!PERKEY && e.rest != 1.f) {
                p[0] *= e.rest;
                p[1] *= e.rest;
              }
              w[j >> 1] = pack_weights(p[0], p[1]);
            }
            if (!PERKEY) l = fmaf(s0 + s1, e.iv, l);
            tk_st16(s_t + c * 16, w);
          }
        };
        if (all && !large) weights(std::true_type());
        else weights(std::false_type());
        tk_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg]);
      }
      n = n1;
      // ---- the item's end: the two streams joined, each warpgroup half the columns
      s_ml[wg * 128 + row] = m;
      s_ml[256 + wg * 128 + row] = l;
      // the last products of both streams, in their order (only then is a
      // barrier's one phase bit clear about which of its passes it means)
      const bool two = n1 - n0 > 1;
      if (two) await(&o_done[n1 & 1], ((n1 - 2) >> 1) & 1);
      await(&o_done[(n1 - 1) & 1], ((n1 - 1) >> 1) & 1);
      tc_fence_after();
      if (tid == 0) s_flag[0] = *s_abort;
      group_sync(kTkSoft);
      const bool aborted = s_flag[0] != 0;
      const uint32_t sa = n0 & 1;  // the stream of the first tile
      const float ma = s_ml[sa * 128 + row], la = s_ml[256 + sa * 128 + row];
      const float mb = two ? s_ml[(sa ^ 1) * 128 + row] : -INFINITY, lb = two ? s_ml[256 + (sa ^ 1) * 128 + row] : 0.f;
      float rm = fmaxf(ma, mb);
      auto factor = [&](float mk, float lk) { return mk == -INFINITY ? (lk == lk ? 0.f : lk) : ex2(mk - rm); };
      const float fa = factor(ma, la), fb = factor(mb, lb);
      float rl = (ma == -INFINITY && la == la ? 0.f : la * fa) + (mb == -INFINITY && lb == lb ? 0.f : lb * fb);
      if (lim == 0) {
        rm = -INFINITY;
        rl = 0.f;
      }
      const bool part = !(sg.t0 == 0 && sg.t1 == sg.nt);
      float* wslot = pl.ws + (int64_t)(2 * blockIdx.x + (sg.t0 == 0 ? 1 : 0)) * kKvSlot;
      const int tt = row / sg.nh;
      const int64_t rq = ((int64_t)sg.b * a.T + sg.tk + tt) * a.Q + sg.h0 + row - tt * sg.nh;
      const bool write = row < sg.nrow && !aborted;
      const bool zero = rl == 0.f;
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const int col0 = wg * (DP / 2) + c * 32;
        uint32_t oa[32], ob[32];
        tmem_ld32_nowait(lanes + 256 + sa * 128 + col0, oa);
        if (two) tmem_ld32_nowait(lanes + 256 + (sa ^ 1) * 128 + col0, ob);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float v = __uint_as_float(oa[j]) * fa;
          if (two) v = fmaf(__uint_as_float(ob[j]), fb, v);
          if (FMT == kKvE4m3 && s_nan[sb + col0 + j] < lim) v = __int_as_float(0x7FC00000);
          oa[j] = __float_as_uint(v);
        }
        if (write) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (col0 + j >= a.D) break;
            if (part) {
              float* d = wslot + row * 128 + col0 + j;
              *reinterpret_cast<uint4*>(d) = make_uint4(oa[j], oa[j + 1], oa[j + 2], oa[j + 3]);
              *reinterpret_cast<uint4*>(d + 4) = make_uint4(oa[j + 4], oa[j + 5], oa[j + 6], oa[j + 7]);
            } else {
              uint32_t p[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                p[k] = zero ? 0u
                            : (uint32_t)__bfloat16_as_ushort(
                                  __float2bfloat16_rn(__fdiv_rn(__uint_as_float(oa[j + 2 * k]), rl))) |
                                  ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(
                                       __fdiv_rn(__uint_as_float(oa[j + 2 * k + 1]), rl)))
                                   << 16);
              *reinterpret_cast<uint4*>(a.out + rq * a.D + col0 + j) = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
        }
      }
      if (write && wg == 0) {
        if (part) {
          wslot[128 * 128 + row] = rm;
          wslot[128 * 128 + 128 + row] = rl;
        } else if (a.lse) {
          a.lse[rq] = zero ? -INFINITY : kv_lse<(int)kTkLift>(rm, rl);
        }
      }
      tc_fence_before();
      if (part) __threadfence();
      group_sync(kTkSoft);  // limits, NaN positions and accumulators have been read
      if (wg == 0) s_nan[sb + row] = INT32_MAX;  // for the item after the next
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[seg & 1]);
      if (part) {
        int64_t c0;
        const int np = kv_parts(sg.unit0, sg.nt, W, nc, c0);
        if (tid == 0) s_flag[1] = kv_arrive(pl.arrive, c0, np) && !aborted;
        group_sync(kTkSoft);
        if (s_flag[1]) {
          __threadfence();
          // a warp per row, four columns a lane; the parts in the order of the keys
          const float* ws0 = pl.ws + 2 * c0 * kKvSlot;
          const int col = lane * 4;
          for (int r = warp; r < sg.nrow; r += 8) {
            float m_ = -INFINITY, l_ = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < np; k0 += 4) {
              float mk[4], lk[4];
              float4 w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if (k0 + x >= np) break;
                const float* p = ws0 + (int64_t)(2 * (k0 + x) + (k0 + x == 0 ? 1 : 0)) * kKvSlot;
                mk[x] = __ldcg(p + 128 * 128 + r);
                lk[x] = __ldcg(p + 128 * 128 + 128 + r);
                w[x] = col < a.D ? __ldcg(reinterpret_cast<const float4*>(p + r * 128 + col))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if (k0 + x >= np) break;
                const float mn = fmaxf(m_, mk[x]);
                const float f0 = m_ == -INFINITY ? (l_ == l_ ? 0.f : l_) : ex2(m_ - mn);
                const float f1 = mk[x] == -INFINITY ? (lk[x] == lk[x] ? 0.f : lk[x]) : ex2(mk[x] - mn);
                m_ = mn;
                l_ = fmaf(l_, f0, lk[x] * f1);
                o.x = fmaf(o.x, f0, w[x].x * f1);
                o.y = fmaf(o.y, f0, w[x].y * f1);
                o.z = fmaf(o.z, f0, w[x].z * f1);
                o.w = fmaf(o.w, f0, w[x].w * f1);
              }
            }
            const int t2 = r / sg.nh;
            const int64_t q2 = ((int64_t)sg.b * a.T + sg.tk + t2) * a.Q + sg.h0 + r - t2 * sg.nh;
            const bool z2 = l_ == 0.f;
            auto pair = [&](float x, float y) {
              return z2 ? 0u
                        : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(x, l_))) |
                              ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(y, l_))) << 16);
            };
            if (col < a.D)
              *reinterpret_cast<uint2*>(a.out + q2 * a.D + col) = make_uint2(pair(o.x, o.y), pair(o.z, o.w));
            if (lane == 0 && a.lse)
              a.lse[q2] = z2 ? -INFINITY : kv_lse<(int)kTkLift>(m_, l_);
          }
        }
        group_sync(kTkSoft);  // s_flag is read
      }
      ++seg;
    }
  }
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int FMT, int DP, bool PERKEY>
cudaError_t launch_tk(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& a, const TkPlan& pl, int grid,
                      cudaStream_t stream) {
  using L = TkLayout<DP, PERKEY>;
  auto kern = kv_attn_tc_kernel<FMT, DP, PERKEY>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::total);
  if (e != cudaSuccess) return e;
  kern<<<grid, kTkThreads, L::total, stream>>>(mk, mv, a, pl);
  return cudaGetLastError();
}

}  // namespace

bool kv_attn_tc_supported(const KvAttnArgs& a) {
  // More rows to a key head than the other kernel's tile has, keys in the order
  // of their positions, copies that start on 128 bytes of shared memory.
  return !a.page_idx && a.D <= 128 && (int64_t)a.T * (a.Q / a.H) > 64 && (a.D > 64 || a.P % 2 == 0);
}

cudaError_t launch_kv_attn_tc(const KvAttnArgs& a, int num_sms, cudaStream_t stream) {
  auto encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const int G = a.Q / a.H, dp = a.D <= 64 ? 64 : 128;
  TkPlan pl{};
  pl.GG = G < kTkRows ? G : kTkRows;
  pl.ng = (G + pl.GG - 1) / pl.GG;
  const int fit = kTkRows / pl.GG;
  pl.TT = fit < a.T ? fit : a.T;
  pl.ntb = (a.T + pl.TT - 1) / pl.TT;
  const int low = a.P & -a.P;  // the largest power of two in P
  pl.hb = low < kTkHalf ? low : kTkHalf;
  pl.ws = a.ws;
  pl.arrive = a.arrive;
  CUtensorMap mk, mv;
  if (!encode_cache_map(encode, &mk, a, a.k_cache, dp, pl.hb) ||
      !encode_cache_map(encode, &mv, a, a.v_cache, dp, pl.hb))
    return cudaErrorInvalidValue;
  const bool perkey = pl.hb < 32;
#define IDX_TK_GO(F)                                                                        \
  (dp == 64 ? (perkey ? launch_tk<F, 64, true>(mk, mv, a, pl, num_sms, stream)              \
                      : launch_tk<F, 64, false>(mk, mv, a, pl, num_sms, stream))            \
            : (perkey ? launch_tk<F, 128, true>(mk, mv, a, pl, num_sms, stream)             \
                      : launch_tk<F, 128, false>(mk, mv, a, pl, num_sms, stream)))
  return a.format == kKvE4m3 ? IDX_TK_GO(kKvE4m3) : IDX_TK_GO(kKvInt8);
#undef IDX_TK_GO
}

}  // namespace idx
