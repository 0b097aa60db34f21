// kv_attn.cuh -- attention over the pages of the 8-bit KV cache, streamed.
//
// Row (b, t), query head h, kv head g = h / G (G = Q / H): over the keys i that
// the row sees,
//     s_i = scale * (q . k8_i) * ks_i,   out = sum_i softmax(s)_i * v8_i * vs_i,
// k8, v8 the codes and ks, vs their page's scales.  One pass over the keys with
// the running maximum and sum of the softmax.
//
// The value scale goes into the exponent: with x_i = s_i log2(e) + log2(vs_i)
// and m the running maximum of x less 14,
//     p_i = 2^(x_i - m) <= 2^14,  O += p_i v8_i,  l += p_i / vs_i,
//     out = O / l,  lse = (m + log2 l) ln 2.
// So the weights that meet the codes in the tensor cores end at the top of
// fp16's range whatever the scales are: those down to 2^-28 of the largest are
// held to 2^-11 of their own size, smaller ones to 2^-39 of the largest (a key
// with most of the weight and no value, over a long context, leaves the output
// to them).  e4m3 and int8 codes are exact in fp16, products are exact and sums
// are fp32.  bf16 queries become fp16 under a power of two per row that brings the
// largest element to fp16's top binade (its inverse goes into the score's
// factor): exact for elements down to 2^-31 of the largest, to 2^-39 of it below.
// A value scale below 2^-86 counts as 2^-86 in the exponent (the sum l stays
// finite), and its weights are multiplied by what is left.
//
// Work: a row tile is TT tokens of one request (1 with page lists, which differ
// by token) and up to 16*MT query rows (tokens x heads of one kv head), an item
// is a row tile and a kv head, a unit is 32 keys of it.  The units of all items
// are laid end to end, with a charge for each item's start and end, and cut
// evenly over the CTAs (one per SM).  An item that
// is cut leaves partial results (O, m, l) in the workspace; the last of its
// CTAs to arrive joins them in the order of the keys.
//
// A CTA has four producer warps and twelve (or eight) consumer warps.  A producer
// looks up 32 units at a time (page list, block table, scales; one per lane),
// skips those without keys, and has the TMA engine copy the keys and values of
// each into a ring of stages.  The producers take the look-ups in turns, so that
// four chains of dependent loads are under way; they fill the stages in order,
// each passing the number used so far to the next.  A consumer warp takes every
// 12th stage for up to 16 query rows (up to four warps share a stage when there are
// more rows) with an accumulator of its own, so no two
// warps meet before the item's end; there they join their maxima, sums and
// accumulators.
// One unit is 32 keys x D codes of K and of V: 8 KB at D = 128.
//
// The matrix instruction is the warp-wide m16n8k16, with the keys (of the
// scores) and the value columns (of the outputs) as its 16 rows and the query
// rows as its 8 columns: the 4 or 8 heads of a kv head fill them, and a code is
// decoded once for all rows of a warp.  With so few query rows a key is used for
// 4 flops a row and code, far below what the tcgen05 tiles of 128 rows are for,
// and the codes have to pass through registers to become fp16 anyway: they go
// from there into the instruction without a second trip through shared memory.
// The order of the head dim within a product is free, so a lane takes 16
// consecutive codes of a key as four steps' operands; the keys of the product
// with V come transposed out of ldmatrix as pairs of codes, which one byte
// permute turns into two operands (even and odd dims).
//
// What bounds it: HBM by its bytes (2 D per key and kv head); measured at 32
// requests x 256 pages of 64 keys, 8 kv heads: D = 128 e4m3 167 us (5.2 TB/s), D =
// 256 287 us (6.0), D = 64 129 us (3.4): with fewer bytes a unit the
// consumers' decoding and softmax are what the memory waits for (570 warp
// instructions a unit in all roles, 910 at D = 256 and 390 at D = 64).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kv.cuh"
#include "tc.cuh"

// A test build defines this as a condition under which a CTA runs as if one of
// its waits had expired.
#ifndef IDX_KV_GIVE_UP
#define IDX_KV_GIVE_UP 0
#endif

namespace idx {

constexpr int kKvProducers = 4;
constexpr int kKvProducerBarrier = 2;  // the named barrier of the producer warps
constexpr int kKvUnit = 32;        // keys per unit
constexpr int kKvMaxStages = 32;
constexpr int kKvMaxBatch = 8;     // units the producer issues at once, at most
// Units that an item's start and end count for in the split (8: 179 us, 14: 176, 20:
// 173, 28: 167 for 32 x 256 pages of 64; 512 rows of 64-key pages 107, 95, 89, 88).
constexpr int kKvCharge = 28;
constexpr int kKvSegs = 64;        // descriptor ring: more than the stages and a group of warps
constexpr int kKvSmem = 227 * 1024;
constexpr float kKvMinScale = 1.2924697071141057e-26f;  // 2^-86
constexpr float kKvLift = 14.f;            // log2 of the largest weight

// What the host settles for a launch.
struct KvPlan {
  int TT;           // tokens per row tile
  int ntb;          // row tiles per request
  int GG;           // query heads per item
  int ng;           // items per kv head
  int ppt, tpp;     // pages per unit (P < 32) or units per page
  int pitch;        // rows from page to page in a unit of several pages
  int box;          // rows of a copy
  int nstage;
  float* ws;        // 2 slots per CTA: O [64][256], m, l
  int32_t* arrive;  // one counter per CTA, zero between launches
};
constexpr int kKvSlot = 64 * 256 + 256;  // floats of a workspace slot (also O [128][128], m, l)

struct KvSeg {
  int64_t unit0;    // the item's first unit, as the split counts
  int nt;           // its units
  int b, t0, nrow;  // request, first token, query rows (tokens x heads)
  int h0;           // first query head
  int first, last;  // whether this segment has the item's first and last unit
  int max_count;    // keys that the tile's rows see: the most
};

// Scales of a stage's keys (one entry, or one per key where a unit has several
// pages): the score's, log2 and inverse of the value's, and what is left of a
// value scale below 2^-86.  Beside them the position of the (first) key, and
// per stage its segment, kKvFull, the number of its keys and the parity of its
// latest pass (-1: never filled).
struct KvPage {
  float ks, lv, iv, rest;
};
constexpr int kKvFull = 1;  // every row that sees any key sees all 32

// NT: 8-row blocks of query rows that a warp holds; RG: groups of warps over the
// query rows (8 * NT * RG rows in all).
template <int DP, int NT, int RG, bool MULTI>
struct KvLayout {
  static constexpr int RB = DP < 128 ? DP : 128;      // bytes of a row in a block
  static constexpr int NB = DP / RB;                  // column blocks
  static constexpr int NC = DP == 256 ? 8 : 12;       // consumer warps
  static constexpr int kThreads = (NC + kKvProducers) * 32;
  static constexpr int KG = NC / RG;                  // groups of warps taking turns
  // The launch's registers (128 or 168 a thread), moved from the producers to
  // the consumers: 4 x 80 + 12 x 144 = 16 x 128, 4 x 80 + 8 x 208 <= 12 x 168.
  static constexpr int kProducerRegs = 80;
  static constexpr int kConsumerRegs = NC == 8 ? 208 : 144;
  static constexpr int WR = 8 * NT;                   // rows of a warp
  static constexpr int M = WR * RG;                   // rows of a tile
  static constexpr int kStage = 2 * kKvUnit * DP;     // K then V
  static constexpr int kJoin = NC * (WR < 16 ? 16 : WR) * 36;  // floats to join accumulators in
  static constexpr int kQPitch = DP * 2 + 16;
  static constexpr int kPages = MULTI ? kKvUnit : 1;  // scale entries: per key or one
  static constexpr size_t bars = 0;                                    // full, empty
  static constexpr size_t misc = bars + 2 * kKvMaxStages * 8;          // 64 ints
  static constexpr size_t seg = misc + 256;
  static constexpr size_t meta = seg + kKvSegs * sizeof(KvSeg);        // int[4] per stage
  static constexpr size_t page = meta + kKvMaxStages * 16;
  static constexpr size_t pos = page + (size_t)kKvMaxStages * kPages * sizeof(KvPage);
  static constexpr size_t ml = (pos + (size_t)kKvMaxStages * kPages * 4 + 15) & ~(size_t)15;
  static constexpr size_t rows = ml + NC * WR * 8;                     // factor, limits, m, l per row
  static constexpr size_t q = rows + 64 * 20;
  static constexpr size_t join = q + (size_t)M * kQPitch;
  static constexpr size_t ring = (join + (size_t)kJoin * 4 + 1023) & ~(size_t)1023;
  static constexpr int stages() {
    const int n = (int)((kKvSmem - 1024 - ring) / kStage);
    return n < kKvMaxStages ? n : kKvMaxStages;
  }
  // A batch waits for all of its stages.  At an item's end every group but the
  // last may hold a stage of the next item (that is how it learns of the end)
  // until the last one has met them: what is left must hold a batch.
  static constexpr int batch() {
    return stages() - KG + 1 < kKvMaxBatch ? stages() - KG + 1 : kKvMaxBatch;
  }
  static constexpr size_t total() { return ring + (size_t)stages() * kStage + 1024; }
  static_assert(NC % RG == 0 && stages() >= KG, "each group of warps needs a stage");
  static_assert(kKvSegs > kKvMaxStages + KG, "descriptors must outlive their stages");
  static_assert(kJoin >= kThreads * 6, "the partial results are joined there too");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The weights' pair.  Saturated: where a step of the scores is 8 or more, the
// reference may round down by it, and a weight reach 2^16.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// int8 to fp16: 0x6400 + (code ^ 0x80) is 1024 + 128 + code, exactly.
__device__ __forceinline__ uint32_t minus_1152(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0x64806480u));
  return r;
}

// A transposed 8x8 block of fp16: lane 4 r + c holds (r, 2 c), (r, 2 c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

// The power of two that a row of queries is multiplied by, from the exponent field
// of its largest finite element (which it brings to [2^14, 2^15), or as near as
// its own range allows), and its inverse.
__device__ __forceinline__ void query_factors(int field, float& f, float& inverse) {
  const int e = field < 15 ? 15 : field;  // at most 254
  f = __int_as_float((268 - e) << 23);
  inverse = __int_as_float((e - 14) << 23);
}

// Four codes of a word as fp16 pairs: (0, 1), (2, 3), or, ACROSS, (0, 2), (1, 3).
template <int FMT, bool ACROSS>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& x, uint32_t& y) {
  if (FMT == kKvE4m3) {
    if (ACROSS) w = __byte_perm(w, 0, 0x3120);
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(w));
  } else {
    w ^= 0x80808080u;
    x = minus_1152(__byte_perm(w, 0x64646464u, ACROSS ? 0x4240 : 0x4140));
    y = minus_1152(__byte_perm(w, 0x64646464u, ACROSS ? 0x4341 : 0x4342));
  }
}

// A page's entry from its scales.
__device__ __forceinline__ KvPage kv_scales(float ks, float vs) {
  const float v1 = fmaxf(vs, kKvMinScale);
  const uint32_t vb = __float_as_uint(v1);
  KvPage e;
  e.ks = ks;
  // 2^lv must give a power of two back exactly
  e.lv = (vb & 0x7FFFFFu) ? __log2f(v1) : (float)((int)(vb >> 23) - 127);
  e.iv = __fdiv_rn(1.f, v1);
  e.rest = vs < kKvMinScale ? vs * (1.f / kKvMinScale) : (vs == vs ? 1.f : vs);
  return e;
}

// Units of row tile rt (at least one: a tile without keys still has an output),
// and the most and fewest keys that its rows with keys see.
struct KvTile {
  int nt, max_count, min_count;
};

__device__ __forceinline__ int kv_count(const KvAttnArgs& a, int64_t r, int& bits) {
  int c = __ldg(a.key_counts + r);
  if (c < 0 || c > a.N * a.P) {
    bits |= kErrLengthClamped;
    c = c < 0 ? 0 : a.N * a.P;
  }
  return c;
}

__device__ __forceinline__ int kv_units(const KvAttnArgs& a, const KvPlan& pl, int max_count) {
  int np = (max_count + a.P - 1) / a.P;
  int64_t nt;
  if (a.page_idx) {
    np = np < a.K ? np : a.K;  // a list of distinct pages has no more with keys
    nt = pl.ppt > 1 ? (np + pl.ppt - 1) / pl.ppt : (int64_t)np * pl.tpp;
  } else if (pl.ppt > 1) {
    nt = (np + pl.ppt - 1) / pl.ppt;
  } else {
    nt = np ? (int64_t)(np - 1) * pl.tpp + (max_count - (np - 1) * a.P + kKvUnit - 1) / kKvUnit : 0;
  }
  return nt < 1 ? 1 : (int)nt;
}

// One thread's walk over the tile's tokens.
__device__ __forceinline__ KvTile kv_tile(const KvAttnArgs& a, const KvPlan& pl, int64_t rt,
                                          int& bits) {
  const int b = (int)(rt / pl.ntb), t0 = (int)(rt - (int64_t)b * pl.ntb) * pl.TT;
  const int n = a.T - t0 < pl.TT ? a.T - t0 : pl.TT;
  KvTile k;
  k.max_count = 0;
  k.min_count = INT32_MAX;
  for (int t = 0; t < n; ++t) {
    const int c = kv_count(a, (int64_t)b * a.T + t0 + t, bits);
    k.max_count = c > k.max_count ? c : k.max_count;
    if (c > 0 && c < k.min_count) k.min_count = c;
  }
  k.nt = kv_units(a, pl, k.max_count);
  return k;
}

// An item of nt units from unit0 on, cut over CTAs of which nc share W units:
// the first of them and how many they are.
__device__ __forceinline__ int kv_parts(int64_t unit0, int nt, int64_t W, int64_t nc, int64_t& c0) {
  c0 = ((unit0 + 1) * nc + W - 1) / W - 1;
  return (int)(((unit0 + nt) * nc + W - 1) / W - 1 - c0) + 1;
}

// log(sum_i exp(s_i)) of a row from its reference and sum, whose weights carry
// 2^LIFT: taken off first, so that the logarithm is of the size of the count.
template <int LIFT>
__device__ __forceinline__ float kv_lse(float m, float l) {
  return (m + (float)LIFT + __log2f(l * (1.f / (1 << LIFT)))) * 0.69314718055994530942f;
}

// One thread of a CTA is through with its part of such an item, written or not
// (every CTA arrives, so that the counter is zero again when the call ends).
// True for the last to arrive.
__device__ __forceinline__ bool kv_arrive(int32_t* arrive, int64_t c0, int np) {
  const bool last = atomicAdd(arrive + c0, 1) == np - 1;
  if (last) arrive[c0] = 0;
  return last;
}

template <int FMT, int DP, int NT, int RG, bool MULTI>
__global__ void __launch_bounds__(KvLayout<DP, NT, RG, MULTI>::kThreads, 1)
    kv_attn_kernel(const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const KvAttnArgs a,
                   const KvPlan pl) {
  using L = KvLayout<DP, NT, RG, MULTI>;
  constexpr int KG = L::KG, NC = L::NC, M = L::M;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* empty = full + kKvMaxStages;
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* s_abort = misc;        // misc[0]
  int* s_flag = misc + 2;              // per segment: aborted, last to arrive
  int* s_done = misc + 4;              // segments ended before the CTA gave up
  int64_t* s_where = reinterpret_cast<int64_t*>(misc + 8);  // row tile, units before, both ends
  long long* s_warp = reinterpret_cast<long long*>(misc + 24);  // warp sums
  volatile unsigned long long* s_tot =  // per look-up: its number, stages before it
      reinterpret_cast<volatile unsigned long long*>(misc + 56);
  KvSeg* segs = reinterpret_cast<KvSeg*>(smem + L::seg);
  int* meta = reinterpret_cast<int*>(smem + L::meta);
  KvPage* pages = reinterpret_cast<KvPage*>(smem + L::page);
  int* poss = reinterpret_cast<int*>(smem + L::pos);
  unsigned char* ring = smem + L::ring;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ns = pl.nstage;
  const int items = a.H * pl.ng;  // items per row tile
  const int64_t nrt = (int64_t)a.B * pl.ntb;
  int bits = 0;

  // ---- the split: units before each thread's row tiles, then this CTA's share
  const int64_t per = (nrt + L::kThreads - 1) / L::kThreads;
  const int64_t rt0 = tid * per < nrt ? tid * per : nrt;
  const int64_t rt1 = rt0 + per < nrt ? rt0 + per : nrt;
  long long mine = 0;
  if (tid == 0) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  int nt_first = 0;
  for (int64_t rt = rt0; rt < rt1; ++rt) {
    const int nt = kv_tile(a, pl, rt, bits).nt;
    if (rt == rt0) nt_first = nt;
    mine += nt + kKvCharge;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid < ns) {
    mbar_init(&full[tid], 1);
    mbar_init(&empty[tid], RG);
    fence_mbar_init();
    meta[tid * 4 + 3] = -1;
  }
  if (tid == 0) {
    *s_abort = IDX_KV_GIVE_UP;
    *s_done = 0;
  }
  if (tid < kKvProducers) s_tot[tid] = tid ? ~0ull : 0ull;
  if (MULTI)  // rows between and behind a unit's pages hold no key
    for (int i = tid; i < kKvMaxStages * L::kPages; i += L::kThreads) {
      pages[i] = KvPage{0.f, 0.f, 0.f, 0.f};
      poss[i] = INT32_MAX;
    }
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < L::kThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  before += incl - mine;
  const int64_t W = total * items;
  // at least a unit for each group of warps, so that a short batch is not cut
  // into more parts than joining them is worth
  int64_t nc = (W + KG) / (KG + 8);
  nc = nc < 1 ? 1 : (nc < (int64_t)gridDim.x ? nc : (int64_t)gridDim.x);
  if ((int64_t)blockIdx.x >= nc) return;
  if (tid == 0) {
    s_where[2] = W;
    s_where[3] = nc;
  }
  const int64_t u_begin = W * blockIdx.x / nc, u_end = W * (blockIdx.x + 1) / nc;
  {
    long long base = before * items;
    if (u_begin < base + mine * items && u_end > base)
      for (int64_t rt = rt0; rt < rt1; ++rt) {
        const int64_t n = (rt == rt0 ? nt_first : kv_tile(a, pl, rt, bits).nt) + kKvCharge;
        if (u_begin >= base && u_begin < base + n * items) {
          s_where[0] = rt;
          s_where[1] = base;
          s_where[4] = rt * items + (u_begin - base) / n;
        }
        if (u_end - 1 >= base && u_end - 1 < base + n * items) {
          // a last item of which only charged units fall here is not this CTA's
          const int64_t it = (u_end - 1 - base) / n;
          s_where[5] = rt * items + it - (u_end - base - it * n <= kKvCharge ? 1 : 0);
        }
        base += n * items;
      }
  }
  __syncthreads();
  const int nseg = (int)(s_where[5] - s_where[4] + 1);
  if (nseg <= 0) return;

  if (warp >= NC) {
    // =================================================================== producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kProducerRegs));
    const int pw = warp - NC;
    int64_t rt = s_where[0], base = s_where[1], u = u_begin;
    uint32_t look = 0;            // look-ups so far, of all producers
    int sidx = 0;
    bool ok = true;
    // The stages used before look-up `look`, once its predecessor has filled its own.
    auto stages_before = [&](uint32_t& n) {
      for (uint32_t it = 0; it < kMaxWaitIters; ++it) {
        const unsigned long long v = s_tot[look % kKvProducers];
        if ((uint32_t)(v >> 32) == look) {
          __threadfence_block();
          n = (uint32_t)v;
          return true;
        }
        if (*s_abort) return false;
        __nanosleep(100);  // leaves the issue slots to the consumers
      }
      *s_abort = 1;
      atomicOr(a.status, kErrWaitTimeout);
      return false;
    };
    auto tell = [&](uint32_t n) {  // whole warp: its shared-memory writes come first
      __threadfence_block();
      __syncwarp();
      if (lane == 0)
        s_tot[(look + 1) % kKvProducers] = ((unsigned long long)(look + 1) << 32) | n;
    };
    while (ok && u < u_end) {
      // the row tile: counts of its tokens, a lane each
      const int b = (int)(rt / pl.ntb), tk = (int)(rt - (int64_t)b * pl.ntb) * pl.TT;
      const int ntok = a.T - tk < pl.TT ? a.T - tk : pl.TT;
      int mx = 0, mn = INT32_MAX;
      for (int t = lane; t < ntok; t += 32) {
        const int c = kv_count(a, (int64_t)b * a.T + tk + t, bits);
        mx = c > mx ? c : mx;
        if (c > 0 && c < mn) mn = c;
      }
      mx = __reduce_max_sync(0xFFFFFFFFu, mx);
      mn = __reduce_min_sync(0xFFFFFFFFu, mn);
      const int nt = kv_units(a, pl, mx);
      const int64_t n = nt + kKvCharge;
      const int64_t rt_end = base + n * items;
      while (ok && u < u_end && u < rt_end) {
        const int it = (int)((u - base) / n);
        const int64_t x0 = (u - base) - it * n;
        const int64_t x1 = n - x0 < u_end - u ? n : x0 + (u_end - u);
        u += x1 - x0;
        // the charged units come first: a cut among them is a cut before the item
        const int t0 = x0 <= kKvCharge ? 0 : (int)(x0 - kKvCharge);
        const int t1 = x1 <= kKvCharge ? 0 : (int)(x1 - kKvCharge);
        if (t1 == t0) continue;
        const int g = it / pl.ng, hg = it - g * pl.ng;
        const int G = a.Q / a.H;
        const int heads = G - hg * pl.GG < pl.GG ? G - hg * pl.GG : pl.GG;
        // units of the list: past the expected ones too in the item's last
        // segment (lists with gaps or repeated pages)
        const int64_t r = (int64_t)b * a.T + tk;
        const int np = a.page_idx ? a.K : (mx + a.P - 1) / a.P;
        int64_t stop = t1;
        if (mx == 0) stop = t0;
        else if (a.page_idx && t1 == nt)
          stop = MULTI ? (np + pl.ppt - 1) / pl.ppt : (int64_t)np * pl.tpp;
        const int tpc = MULTI ? 32 / pl.ppt : 32;  // units per look-up
        int64_t c = t0;
        do {  // a segment without units has a look-up too: its stage without keys
          if (look % kKvProducers != (uint32_t)pw) {
            ++look;
            c += tpc;
            continue;
          }
          int e, sub = 0;
          bool valid;
          if (MULTI) {
            const int64_t e64 = c * pl.ppt + lane;
            valid = lane < tpc * pl.ppt && e64 < np && c + lane / pl.ppt < stop;
            e = (int)e64;
          } else {
            const int64_t t = c + lane;
            valid = t < stop;
            e = (int)(t / pl.tpp);
            sub = (int)(t - (int64_t)e * pl.tpp) * kKvUnit;
          }
          int p = 0, id = 0;
          if (valid) {
            p = a.page_idx ? __ldg(a.page_idx + r * a.K + e) : e;
            if (p < 0 || p >= a.N) {
              if (p != -1) bits |= kErrPageClamped;
              valid = false;
            }
          }
          valid = valid && (int64_t)p * a.P + sub < mx;
          if (valid) {
            id = __ldg(a.page_table + (int64_t)b * a.ld_pt + p);
            if (id < 0 || id >= a.n_blocks) {
              bits |= kErrPageClamped;
              valid = false;
            }
          }
          float ks = 0.f, vs = 0.f;
          int pos = INT32_MAX, row = 0, nk = 0;
          if (valid) {
            const int64_t cell = (int64_t)id * a.H + g;
            ks = __ldg(a.k_scale + cell);  // (not waited for before the copies are issued)
            vs = __ldg(a.v_scale + cell);
            pos = p * a.P + sub;
            row = (int)(cell * a.P) + sub;
            nk = a.P - sub < kKvUnit ? a.P - sub : kKvUnit;
            nk = mx - pos < nk ? mx - pos : nk;
          }
          const bool whole = valid && nk == (MULTI ? a.P : kKvUnit) && pos + nk <= mn;
          const uint32_t vmask = __ballot_sync(0xFFFFFFFFu, valid);
          const uint32_t fmask = __ballot_sync(0xFFFFFFFFu, whole);
          // this lane's unit: its lanes, its first lane, its place among the
          // look-up's units with keys
          const int unit = MULTI ? lane / pl.ppt : lane;
          const uint32_t who =
              MULTI ? (pl.ppt == 32 ? 0xFFFFFFFFu : ((1u << pl.ppt) - 1u) << ((unit * pl.ppt) & 31))
                    : 1u << lane;
          const bool busy = (vmask & who) != 0 && unit < tpc;
          const bool leads = busy && (!MULTI || lane == unit * pl.ppt);
          const uint32_t lead = __ballot_sync(0xFFFFFFFFu, leads);
          const int found = __popc(lead);
          const bool none = found == 0 && c == t0;
          const int fill = none ? 1 : found;
          uint32_t used = 0;
          ok = __all_sync(0xFFFFFFFFu, stages_before(used));
          if (!ok) break;
          if (c == t0 && lane == 0) {
            KvSeg& s = segs[sidx % kKvSegs];
            s.unit0 = base + it * n + kKvCharge;
            s.nt = nt;
            s.b = b;
            s.t0 = tk;
            s.nrow = ntok * heads;
            s.h0 = g * G + hg * pl.GG;
            s.first = t0 == 0;
            s.last = t1 == nt;
            s.max_count = mx;
          }
          int slot = (int)(used % (uint32_t)ns), phase = (int)((used / (uint32_t)ns) & 1) ^ 1;
          const int place = __popc(lead & ((MULTI ? 1u << ((unit * pl.ppt) & 31) : 1u << lane) - 1u));
          int my = slot + place, my_phase = phase;  // the stage and its phase
          while (my >= ns) {
            my -= ns;
            my_phase ^= 1;
          }
          // batch() units at a time, every lane for itself: a stage is filled
          // as soon as the batch's last one is free
          for (int b0 = 0; b0 < found && ok; b0 += L::batch()) {
            const bool go = busy && place >= b0 && place < b0 + L::batch();
            bool got = true;
            if (go) got = mbar_wait_bounded(&empty[my], my_phase, s_abort, a.status);
            ok = __all_sync(0xFFFFFFFFu, got);
            if (!ok) break;
            // The copies first: their bytes may arrive before they are expected,
            // the phase still waits for the arrival that expects them.
            if (go && valid) {
              unsigned char* dst = ring + (size_t)my * L::kStage +
                                   (MULTI ? (lane - unit * pl.ppt) * pl.pitch : 0) * L::RB;
#pragma unroll
              for (int cb = 0; cb < L::NB; ++cb) {
                tma_load_2d(dst + cb * kKvUnit * L::RB, &map_k, cb * L::RB, row, &full[my]);
                tma_load_2d(dst + (L::NB + cb) * kKvUnit * L::RB, &map_v, cb * L::RB, row, &full[my]);
              }
            }
            if (go) {
              const KvPage pg = valid ? kv_scales(ks, vs) : KvPage{0.f, 0.f, 0.f, 0.f};
              if (MULTI) {  // entries of the page's keys
                const int k = lane - unit * pl.ppt;
                for (int i = 0; i < a.P; ++i) {
                  pages[my * L::kPages + k * pl.pitch + i] = pg;
                  poss[my * L::kPages + k * pl.pitch + i] = valid ? pos + i : INT32_MAX;
                }
              } else {
                pages[my] = pg;
                poss[my] = pos;
              }
              if (leads) {
                const bool f = (fmask & who) == who && (!MULTI || pl.ppt * a.P == kKvUnit);
                meta[my * 4] = sidx;
                meta[my * 4 + 1] = f ? kKvFull : 0;
                meta[my * 4 + 2] = nk;
                meta[my * 4 + 3] = my_phase ^ 1;
              }
            }
            if (MULTI) __syncwarp();
            if (go && leads)
              mbar_arrive_expect_tx(&full[my], (uint32_t)__popc(vmask & who) * 2u * L::NB * L::RB *
                                                   (uint32_t)pl.box);
            __syncwarp();
          }
          if (ok && none) {
            ok = __all_sync(0xFFFFFFFFu,
                            mbar_wait_bounded(&empty[slot], phase, s_abort, a.status));
            if (!ok) break;
            if (lane < L::kPages) {
              pages[slot * L::kPages + lane] = KvPage{0.f, 0.f, 0.f, 0.f};
              poss[slot * L::kPages + lane] = INT32_MAX;
            }
            if (lane == 0) {
              meta[slot * 4] = sidx;
              meta[slot * 4 + 1] = 0;
              meta[slot * 4 + 2] = 0;
              meta[slot * 4 + 3] = phase ^ 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[slot]);
            __syncwarp();
          }
          // Only now the next look-up may issue: the one bit of a barrier's
          // phase tells neighbouring passes over the ring apart, so stages are
          // filled strictly in order.
          if (ok) tell(used + fill);
          ++look;
          c += tpc;
        } while (c < stop && ok);
        ++sidx;
      }
      base = rt_end;
      ++rt;
    }
    // a last stage for each group of warps
    if (ok && look % kKvProducers == (uint32_t)pw) {
      uint32_t used = 0;
      ok = __all_sync(0xFFFFFFFFu, stages_before(used));
      for (int i = 0; i < KG && ok; ++i, ++used) {
        const int slot = (int)(used % (uint32_t)ns), phase = (int)((used / (uint32_t)ns) & 1) ^ 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[slot], phase, s_abort, a.status));
        if (ok && lane == 0) {
          meta[slot * 4] = INT32_MAX;
          meta[slot * 4 + 3] = phase ^ 1;
          mbar_arrive(&full[slot]);
        }
        __syncwarp();
      }
    }
    // The copies end before the CTA does, whether or not they are still waited
    // for: of each stage the latest, its earlier ones ended before it.
    asm volatile("bar.sync %0, %1;" ::"n"(kKvProducerBarrier), "n"(kKvProducers * 32) : "memory");
    if (pw == 0 && lane < ns && meta[lane * 4 + 3] >= 0) mbar_wait_drain(&full[lane], (uint32_t)meta[lane * 4 + 3]);
    if (bits) atomicOr(a.status, bits);
    return;
  }

  // ===================================================================== consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kConsumerRegs));
  const int rg = warp % RG, kg = warp / RG;
  const int g8 = lane >> 2, c4 = lane & 3;  // row and column pair of a fragment
  // Row i of an 8-key block is this key (with 128-byte rows, such that the two
  // rows of a quarter warp's load differ in the swizzle's high bit).
  constexpr bool PERM = DP >= 128;
  auto key_of = [](int i) { return PERM ? (i >> 1) + 4 * (i & 1) : i; };
  const int krow = key_of(g8);
  const int r0 = rg * L::WR;  // the warp's first query row
  float* s_m = reinterpret_cast<float*>(smem + L::ml);
  float* s_l = s_m + NC * L::WR;
  float* s_qf = reinterpret_cast<float*>(smem + L::rows);
  int* s_lims = reinterpret_cast<int*>(s_qf + 64);
  float* s_rowm = reinterpret_cast<float*>(s_lims + 128);  // the joined rows' m and l
  float* s_rowl = s_rowm + 64;
  unsigned char* s_q = smem + L::q;
  float* s_join = reinterpret_cast<float*>(smem + L::join);
  int slot = kg, phase = 0;
  // Waits for this group's next stage.  A stage goes to another group on the
  // next pass when the stages are no multiple of the groups, and copies land
  // out of order: the pass before must have been used up (its stage released)
  // before the one bit of the full barrier's phase can mean this pass.
  auto await = [&]() {
    const bool got = mbar_wait_bounded(&empty[slot], phase ^ 1, s_abort, a.status) &&
                     mbar_wait_bounded(&full[slot], phase, s_abort, a.status);
    return __all_sync(0xFFFFFFFFu, got) != 0;
  };
  bool ok = await();
  int cur = ok ? meta[slot * 4] : INT32_MAX;

  // queries of a segment: a warp per row, loaded while the one before it is
  // joined, then normalised to a power of two and written as fp16
  constexpr int QR = (M + NC - 1) / NC;
  const int G = a.Q / a.H;
  uint4 qv[QR];
  int qlim[QR];
  auto load_q = [&](const KvSeg& sg) {
    const int nh = G - sg.h0 % G < pl.GG ? G - sg.h0 % G : pl.GG;  // heads of the item
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int m = warp + i * NC;
      qv[i] = make_uint4(0u, 0u, 0u, 0u);
      qlim[i] = 0;
      if (m < sg.nrow) {
        const int tt = m / nh;
        const int64_t r = (int64_t)sg.b * a.T + sg.t0 + tt;
        qlim[i] = kv_count(a, r, bits);
        if (lane * 8 < a.D)
          qv[i] = __ldg(reinterpret_cast<const uint4*>(
              a.q + r * a.ldq + (int64_t)(sg.h0 + m - tt * nh) * a.D + lane * 8));
      }
    }
  };
  auto store_q = [&](int* s_lim) {
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int m = warp + i * NC;
      if (m >= M) break;
      const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
        top = lo < 0x7F80u && lo > top ? lo : top;
        top = hi < 0x7F80u && hi > top ? hi : top;
      }
      float f, inverse;
      query_factors((int)(__reduce_max_sync(0xFFFFFFFFu, top) >> 7), f, inverse);
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = pack_f16(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
      if (lane * 8 < DP)
        *reinterpret_cast<uint4*>(s_q + m * L::kQPitch + lane * 16) =
            make_uint4(o[0], o[1], o[2], o[3]);
      if (lane == 0) {
        s_qf[m] = a.scale * 1.44269504088896340736f * inverse;
        s_lim[m] = qlim[i];
      }
    }
  };
  if (ok) load_q(segs[0]);

  for (int s = 0; s < nseg; ++s) {
    // On an expired wait (cur is then "past every segment") the descriptors may
    // be missing: the warps still meet at every barrier, and write nothing.
    const KvSeg& sg = segs[s % kKvSegs];
    int* s_lim = s_lims + (s & 1) * 64;  // still read when the next item's is written
    store_q(s_lim);
    group_sync(NC * 32);
    float oacc[DP / 16][NT][4];
#pragma unroll
    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) oacc[j][n][x] = 0.f;
    float m[NT][2], l[NT][2];  // of rows r0 + 8 n + 2 c4 + e; l over this lane's keys
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    // One stage; FULL: no row that sees any key misses one of these.
    auto unit = [&](auto full_tag) {
      constexpr bool is_full = decltype(full_tag)::value;
      const unsigned char* kb_ = ring + (size_t)slot * L::kStage;
      const uint32_t vb_ = smem_u32(kb_) + kKvUnit * DP;
      const int nk = is_full ? kKvUnit : meta[slot * 4 + 2];
      // Position of key j of the unit, INT32_MAX if it is none.
      auto pos_of = [&](int j) {
        return MULTI ? poss[slot * L::kPages + (MULTI ? j : 0)] : (j < nk ? poss[slot] + j : INT32_MAX);
      };
      // ---- scores, keys x rows: block t holds keys 16 t + krow (x = 0, 1) and
      // 8 further on (x = 2, 3), rows 8 n + 2 c4 + (x & 1).  One row block is
      // two chains of products for each key block.
      constexpr int CH = NT == 1 ? 2 : 1;
      float sc[CH][2][NT][4];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[c][t][n][x] = 0.f;
#pragma unroll 1
      for (int h = 0; h < DP / 64; ++h) {
        uint4 w[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = t * 16 + e * 8 + krow;
            const int chunk = DP == 64 ? (c4 ^ ((row >> 1) & 3)) : (((h & 1) * 4 + c4) ^ (row & 7));
            w[t][e] = *reinterpret_cast<const uint4*>(
                kb_ + (DP == 256 ? (h >> 1) * kKvUnit * 128 : 0) + row * L::RB + chunk * 16);
          }
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          // dims 64 h + 16 c4 + 8 i2 .. + 7 of the rows: two steps' operands
          uint4 qb[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            qb[n] = *reinterpret_cast<const uint4*>(s_q + (r0 + n * 8 + g8) * L::kQPitch + h * 128 +
                                                    c4 * 32 + i2 * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              uint32_t ka[4];
              codes4<FMT, false>(i2 ? (i ? w[t][0].w : w[t][0].z) : (i ? w[t][0].y : w[t][0].x), ka[0], ka[2]);
              codes4<FMT, false>(i2 ? (i ? w[t][1].w : w[t][1].z) : (i ? w[t][1].y : w[t][1].x), ka[1], ka[3]);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(sc[CH == 2 ? i : 0][t][n], ka, i ? qb[n].z : qb[n].x, i ? qb[n].w : qb[n].y);
            }
        }
      }
      if (CH == 2) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[0][t][0][x] += sc[CH - 1][t][0][x];
      }
      // ---- scales, masks, running maximum
      KvPage pg[MULTI ? 4 : 1];  // of keys 16 t + 8 e + krow
#pragma unroll
      for (int i = 0; i < (MULTI ? 4 : 1); ++i)
        pg[i] = pages[slot * L::kPages + (MULTI ? i * 8 + krow : 0)];
      bool up = false;
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 qf = *reinterpret_cast<const float2*>(s_qf + r0 + n * 8 + 2 * c4);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const KvPage& e = pg[MULTI ? t * 2 + (x >> 1) : 0];
            sc[0][t][n][x] = fmaf(sc[0][t][n][x], e.ks * ((x & 1) ? qf.y : qf.x), e.lv);
          }
        if constexpr (!is_full) {
          const int2 lim = *reinterpret_cast<const int2*>(s_lim + r0 + n * 8 + 2 * c4);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (pos_of(t * 16 + (x >> 1) * 8 + krow) >= ((x & 1) ? lim.y : lim.x))
                sc[0][t][n][x] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(fmaxf(sc[0][0][n][e], sc[0][0][n][2 + e]),
                          fmaxf(sc[0][1][n][e], sc[0][1][n][2 + e]));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16)) - kKvLift;
          top[n][e] = v;
          up |= v > m[n][e];
        }
      }
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float v = fmaxf(m[n][e], top[n][e]);
            f[e] = v == -INFINITY ? 1.f : ex2(m[n][e] - v);
            m[n][e] = v;
            l[n][e] *= f[e];
          }
#pragma unroll
          for (int j = 0; j < DP / 16; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) oacc[j][n][x] *= f[x & 1];
        }
      }
      // ---- weights, transposed into the second product's operand
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float z0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
        const float z1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const KvPage& g = pg[MULTI ? t * 2 + e : 0];
            float p0 = ex2(sc[0][t][n][2 * e] - z0), p1 = ex2(sc[0][t][n][2 * e + 1] - z1);
            l[n][0] = fmaf(p0, g.iv, l[n][0]);
            l[n][1] = fmaf(p1, g.iv, l[n][1]);
            if (MULTI || g.rest != 1.f) {
              p0 *= g.rest;
              p1 *= g.rest;
            }
            pb[t][n][e] = transpose8(pack_weights(p0, p1));
          }
      }
      // ---- O += V^T P: dims 16 j + 2 g8 (x = 0, 1) and one further (x = 2, 3)
      const int vrow = key_of(lane & 7);  // lane i of 8 gives the address of row i's key
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t keep[2];  // bytes of this lane's keys (2 c4 and the next) that some row sees
        if constexpr (!is_full) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            keep[e] = 0;
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (pos_of(t * 16 + e * 8 + key_of(2 * c4 + y)) < sg.max_count)
                keep[e] |= 0xFFFFu << (16 * y);
          }
        }
        const int row = t * 16 + ((lane >> 3) & 1) * 8 + vrow;
#pragma unroll
        for (int j2 = 0; j2 < DP / 32; ++j2) {
          const int ch = j2 * 2 + (lane >> 4);
          const int chunk = DP == 64 ? (ch ^ ((row >> 1) & 3)) : ((ch & 7) ^ (row & 7));
          uint32_t r[4];
          ldsm4_t(r, vb_ + (DP == 256 ? (ch >> 3) * kKvUnit * 128 : 0) + row * L::RB + chunk * 16);
          if constexpr (!is_full) {
            r[0] &= keep[0];
            r[1] &= keep[1];
            r[2] &= keep[0];
            r[3] &= keep[1];
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = j2 * 2 + x;
            uint32_t va[4];
            codes4<FMT, true>(r[2 * x], va[0], va[1]);
            codes4<FMT, true>(r[2 * x + 1], va[2], va[3]);
            if (FMT == kKvE4m3 && !is_full && pl.TT > 1) {
              // Rows of several tokens, and keys that not all of them see: a
              // NaN among those must reach the rows that do, and only them
              // (zero weights do not stop it).
              uint32_t bad[4];
              bool any = false;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                bad[y] = (((va[y] & 0x7FFFu) > 0x7C00u) ? 0xFFFFu : 0u) |
                         (((va[y] & 0x7FFF0000u) > 0x7C000000u) ? 0xFFFF0000u : 0u);
                any |= bad[y] != 0;
              }
              if (__any_sync(0xFFFFFFFFu, any)) {
                uint32_t ones[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  ones[y] = bad[y] & 0x3C003C00u;
                  va[y] &= ~bad[y];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const int lim = s_lim[r0 + n * 8 + g8];
                  uint32_t see[2] = {0u, 0u};  // 1 where the row sees the key
#pragma unroll
                  for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                      if (pos_of(t * 16 + e * 8 + key_of(2 * c4 + y)) < lim) see[e] |= 0x3C00u << (16 * y);
                  float hit[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(hit, ones, see[0], see[1]);
#pragma unroll
                  for (int y = 0; y < 4; ++y)
                    if (hit[y] > 0.f) oacc[j][n][y] = __int_as_float(0x7FC00000);
                }
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(oacc[j][n], va, pb[t][n][0], pb[t][n][1]);
          }
        }
      }
    };
    while (cur == s) {
      if (meta[slot * 4 + 1] & kKvFull) unit(std::true_type());
      else unit(std::false_type());
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      slot += KG;
      if (slot >= ns) {
        slot -= ns;
        phase ^= 1;
      }
      ok = await();
      cur = ok ? meta[slot * 4] : INT32_MAX;
    }

    // ---- the item's end: join the groups of warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 16);
        if (g8 == 0) {
          s_m[warp * L::WR + n * 8 + 2 * c4 + e] = m[n][e];
          s_l[warp * L::WR + n * 8 + 2 * c4 + e] = l[n][e];
        }
      }
    if (tid == 0) s_flag[0] = *s_abort;
    group_sync(NC * 32);
    const bool aborted = s_flag[0] != 0;
    if (tid == 0 && !aborted) *s_done = s + 1;
    const bool part = !(sg.first && sg.last);  // the item is in several CTAs
    float* wslot = pl.ws + (int64_t)(2 * blockIdx.x + (sg.first ? 1 : 0)) * kKvSlot;
    const int nh = G - sg.h0 % G < pl.GG ? G - sg.h0 % G : pl.GG;
    // four columns of a row, joined, to their places
    auto finish = [&](int row, int oc, float m, float l, const float4& o) {
      const int tt = row / nh;
      const int64_t rq = ((int64_t)sg.b * a.T + sg.t0 + tt) * a.Q + sg.h0 + row - tt * nh;
      const bool zero = l == 0.f;
      auto two = [&](float x, float y) {
        return zero ? 0u
                    : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(x, l))) |
                          ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(y, l))) << 16);
      };
      *reinterpret_cast<uint2*>(a.out + rq * a.D + oc) = make_uint2(two(o.x, o.y), two(o.z, o.w));
      if (oc == 0 && a.lse)
        a.lse[rq] = zero ? -INFINITY : kv_lse<(int)kKvLift>(m, l);
    };
    auto own_factor = [&](float mk, float lk, float m) {  // 0 for no keys, NaN stays
      return mk == -INFINITY ? (lk == lk ? 0.f : lk) : ex2(mk - m);
    };
    auto entry = [&](int k, int row) {  // the row's place in group k
      return (k * RG + row / L::WR) * L::WR + row % L::WR;
    };
    if (tid < sg.nrow && !aborted) {
      float rm = -INFINITY, rl = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) rm = fmaxf(rm, s_m[entry(k, tid)]);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float mk = s_m[entry(k, tid)], lk = s_l[entry(k, tid)];
        rl = fmaf(mk == -INFINITY ? (lk == lk ? 0.f : 1.f) : lk, own_factor(mk, lk, rm), rl);
      }
      const bool none = s_lim[tid] == 0;  // padding: whatever its query gave
      s_rowm[tid] = none ? -INFINITY : rm;
      s_rowl[tid] = none ? 0.f : rl;
    }
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < KG; ++k) mm = fmaxf(mm, s_m[entry(k, r0 + n * 8 + 2 * c4 + e)]);
        f[n][e] = own_factor(m[n][e], l[n][e], mm);
      }
    // The accumulators go through shared memory, as many columns at a time as
    // its room holds of the rows in use.
    const int rr = sg.nrow < L::WR ? sg.nrow : L::WR;
    int per = 1;
    while (per * 2 <= DP / 32 && NC * rr * (per * 64 + 4) <= L::kJoin) per *= 2;
    const int jp = per * 32 + 4;
#pragma unroll
    for (int cb = 0; cb < DP / 32; ++cb) {
      const int sub = cb & (per - 1);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const auto& o = oacc[cb * 2 + j][n];
          const int row = n * 8 + 2 * c4;
          float* d = s_join + (warp * rr + row) * jp + sub * 32 + j * 16 + 2 * g8;
          if (row < rr) *reinterpret_cast<float2*>(d) = make_float2(o[0] * f[n][0], o[2] * f[n][0]);
          if (row + 1 < rr)
            *reinterpret_cast<float2*>(d + jp) = make_float2(o[1] * f[n][1], o[3] * f[n][1]);
        }
      if (sub != per - 1) continue;
      group_sync(NC * 32);
      const int pieces = per * 8;  // of four columns
      for (int i = tid; i < sg.nrow * pieces && !aborted; i += NC * 32) {
        const int row = i / pieces, pc = i - row * pieces;
        const int oc = (cb - sub) * 32 + pc * 4;  // the output column
        if (oc >= a.D) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const int w = k * RG + row / L::WR;
          const float4 u =
              *reinterpret_cast<const float4*>(s_join + (w * rr + row % L::WR) * jp + pc * 4);
          o.x += u.x;
          o.y += u.y;
          o.z += u.z;
          o.w += u.w;
        }
        if (part) {
          *reinterpret_cast<float4*>(wslot + row * 256 + oc) = o;
          if (oc == 0) {
            wslot[64 * 256 + row] = s_rowm[row];
            wslot[64 * 256 + 64 + row] = s_rowl[row];
          }
        } else {
          finish(row, oc, s_rowm[row], s_rowl[row], o);
        }
      }
      if (cb != DP / 32 - 1) group_sync(NC * 32);
    }
    if (ok && s + 1 < nseg) load_q(segs[(s + 1) % kKvSegs]);
    if (part && !aborted) {
      // the item's CTAs: c0 holds its first unit, c1 its last
      int64_t c0;
      const int np = kv_parts(sg.unit0, sg.nt, s_where[2], s_where[3], c0);
      __threadfence();
      group_sync(NC * 32);
      if (tid == 0) s_flag[1] = kv_arrive(pl.arrive, c0, np);
      group_sync(NC * 32);
      if (s_flag[1]) {
        __threadfence();
        // Part 0 is in the second slot of its CTA, the others in the first of
        // theirs.  Threads that the pieces leave over share the parts of a piece.
        const float* ws0 = pl.ws + 2 * c0 * kKvSlot;
        const int cpr = a.D / 4, np4 = sg.nrow * cpr;
        int share = NC * 32 / np4;
        share = share < 1 ? 1 : (share < np ? share : np);
        for (int i0 = 0; i0 < np4; i0 += NC * 32) {
          const int piece = share > 1 ? tid % np4 : i0 + tid, sh = share > 1 ? tid / np4 : 0;
          const bool on = piece < np4 && sh < share;
          const int row = piece / cpr, oc = (piece - row * cpr) * 4;
          float m = -INFINITY, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          auto add = [&](float mk, float lk, const float4& u) {
            const float mn = fmaxf(m, mk);
            const float fa = own_factor(m, l, mn), fb = own_factor(mk, lk, mn);
            m = mn;
            l = fmaf(l, fa, lk * fb);
            o.x = fmaf(o.x, fa, u.x * fb);
            o.y = fmaf(o.y, fa, u.y * fb);
            o.z = fmaf(o.z, fa, u.z * fb);
            o.w = fmaf(o.w, fa, u.w * fb);
          };
          constexpr int UP = 4;  // parts in flight
          for (int k0 = sh; on && k0 < np; k0 += UP * share) {
            float mk[UP], lk[UP];
            float4 u[UP];
#pragma unroll
            for (int x = 0; x < UP; ++x) {
              const int k = k0 + x * share;
              if (k >= np) break;
              const float* p = ws0 + (int64_t)(2 * k + (k == 0 ? 1 : 0)) * kKvSlot;
              mk[x] = __ldcg(p + 64 * 256 + row);
              lk[x] = __ldcg(p + 64 * 256 + 64 + row);
              u[x] = __ldcg(reinterpret_cast<const float4*>(p + row * 256 + oc));
            }
#pragma unroll
            for (int x = 0; x < UP; ++x)
              if (k0 + x * share < np) add(mk[x], lk[x], u[x]);
          }
          if (share > 1) {  // np4 * share <= the threads: one round
            float* d = s_join + tid * 6;
            group_sync(NC * 32);
            if (on && sh > 0) {
              d[0] = m;
              d[1] = l;
              d[2] = o.x;
              d[3] = o.y;
              d[4] = o.z;
              d[5] = o.w;
            }
            group_sync(NC * 32);
            for (int x = 1; on && sh == 0 && x < share; ++x) {
              const float* p = s_join + (x * np4 + piece) * 6;
              add(p[0], p[1], make_float4(p[2], p[3], p[4], p[5]));
            }
          }
          if (on && sh == 0) finish(row, oc, m, l, o);
        }
        group_sync(NC * 32);  // s_join is free again
      }
    }
  }
  // A CTA that gave up arrives at the items that it did not come to.  Their
  // descriptors may be missing: the walk of the producers again.
  if (tid == 0 && *s_done < nseg) {
    const int64_t W = s_where[2], nc = s_where[3], u1 = W * (blockIdx.x + 1) / nc;
    int64_t rt = s_where[0], base = s_where[1], u = W * blockIdx.x / nc;
    for (int s = 0; u < u1; ++rt) {
      const int nt = kv_tile(a, pl, rt, bits).nt;
      const int64_t n = nt + kKvCharge, rt_end = base + n * items;
      while (u < u1 && u < rt_end) {
        const int64_t it = (u - base) / n, x0 = (u - base) - it * n;
        const int64_t x1 = n - x0 < u1 - u ? n : x0 + (u1 - u);
        u += x1 - x0;
        if (x1 <= kKvCharge) continue;  // charged units only: not this CTA's
        int64_t c0;
        const int np = kv_parts(base + it * n + kKvCharge, nt, W, nc, c0);
        if (s++ >= *s_done && np > 1) kv_arrive(pl.arrive, c0, np);
      }
      base = rt_end;
    }
  }
}

// nt, rg: 1, 1 / 2, 1 / 2, 2 / 2, 4.
PFN_cuTensorMapEncodeTiled_v12000 get_encode();
// The cache as rows of D codes; boxes of `rows` rows and at most 128 codes,
// 16-byte pieces swizzled within 128 (dp == 64: 64) bytes; codes past D read as 0.
bool encode_cache_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const KvAttnArgs& a,
                      const uint8_t* cache, int dp, int rows);
bool kv_attn_tc_supported(const KvAttnArgs& a);
cudaError_t launch_kv_attn_tc(const KvAttnArgs& a, int num_sms, cudaStream_t stream);

template <int DP>
cudaError_t launch_kv_attn_dp(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& a,
                              KvPlan pl, int nt, int rg, int grid, cudaStream_t stream);

template <int FMT, int DP, int NT, int RG, bool MULTI>
static cudaError_t launch_one(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& a,
                              KvPlan& pl, int grid, cudaStream_t stream) {
  using L = KvLayout<DP, NT, RG, MULTI>;
  pl.nstage = L::stages();
  const size_t smem = L::total();
  auto kern = kv_attn_kernel<FMT, DP, NT, RG, MULTI>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, L::kThreads, smem, stream>>>(mk, mv, a, pl);
  return cudaGetLastError();
}

#ifdef IDX_KV_ATTN_DP
template <>
cudaError_t launch_kv_attn_dp<IDX_KV_ATTN_DP>(const CUtensorMap& mk, const CUtensorMap& mv,
                                              const KvAttnArgs& a, KvPlan pl, int nt, int rg,
                                              int grid, cudaStream_t stream) {
  constexpr int DP = IDX_KV_ATTN_DP;
  const bool multi = pl.ppt > 1;
#define IDX_KV_GO(F, N, R)                                                         \
  (multi ? launch_one<F, DP, N, R, true>(mk, mv, a, pl, grid, stream)              \
         : launch_one<F, DP, N, R, false>(mk, mv, a, pl, grid, stream))
#define IDX_KV_ROWS(F)                                                             \
  (nt == 1 ? IDX_KV_GO(F, 1, 1)                                                    \
           : rg == 1 ? IDX_KV_GO(F, 2, 1) : rg == 2 ? IDX_KV_GO(F, 2, 2) : IDX_KV_GO(F, 2, 4))
  return a.format == kKvE4m3 ? IDX_KV_ROWS(kKvE4m3) : IDX_KV_ROWS(kKvInt8);
#undef IDX_KV_ROWS
#undef IDX_KV_GO
}
#endif

}  // namespace idx
