// kv_tables.cu -- block tables and slot maps from request lengths.
//
// Request b holds cached[b] keys and gets fresh[b] more.  Its pages
// have .. want-1 (have = ceil(cached / P), want = ceil((cached + fresh) / P))
// come from the free list, requests in order: a prefix sum over want - have
// gives each request its place in the list.  From the pages follow the slot of
// every new token and the key and page counts of its attention row.
//
// What bounds it: latency (a few kilobytes of lengths, 12 bytes out per
// token; 6 us for 256 single tokens and for 64 x 1024, replayed in a graph).
// So it is one kernel, without a second pass for the prefix sum: every CTA sums
// the needs of all requests before its own group (two coalesced loads per
// request, from the L2) and scans its group in shared memory.  The slots of new
// pages are read from the free list itself, not from the table entries that the
// same launch writes.
#include "common.cuh"
#include "kernels.h"

namespace idx {

namespace {

constexpr int kTabThreads = 256;
constexpr int kTabTokens = 1024;  // tokens a CTA maps

struct Req {
  int cached, fresh, have, need;
  bool clamped;
};

__device__ __forceinline__ Req load_req(const KvTablesArgs& a, int b) {
  Req r;
  const int room = a.N * a.P;
  const int c = __ldg(a.cached + b);
  r.cached = c < 0 ? 0 : (c > room ? room : c);
  const int f = a.fresh ? __ldg(a.fresh + b) : a.T;
  const int most = a.T < room - r.cached ? a.T : room - r.cached;
  r.fresh = f < 0 ? 0 : (f > most ? most : f);
  r.clamped = r.cached != c || r.fresh != f;
  r.have = (r.cached + a.P - 1) / a.P;
  r.need = (r.cached + r.fresh + a.P - 1) / a.P - r.have;
  return r;
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const KvTablesArgs a, int group,
                                                                int tchunk) {
  __shared__ int s_cached[kTabThreads], s_fresh[kTabThreads], s_have[kTabThreads],
      s_need[kTabThreads];
  __shared__ long long s_start[kTabThreads];
  __shared__ long long s_warp[kTabThreads / 32], s_before[kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int b0 = blockIdx.x * group;
  const int nb = a.B - b0 < group ? a.B - b0 : group;
  int bits = 0;

  // pages needed by the requests before this group
  long long before = 0;
  for (int b = tid; b < b0; b += kTabThreads) before += load_req(a, b).need;
  Req r{};
  if (tid < nb) {
    r = load_req(a, b0 + tid);
    if (r.clamped) bits |= kErrLengthClamped;
  }
  long long incl = r.need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
  }
  if (lane == 31) s_warp[wid] = incl;
  if (lane == 0) s_before[wid] = before;
  __syncthreads();
  int head = a.free_head ? __ldg(a.free_head) : 0;
  if (head < 0 || head > a.n_free) {
    bits |= kErrLengthClamped;
    head = head < 0 ? 0 : a.n_free;
  }
  long long start = head;
  for (int w = 0; w < kTabThreads / 32; ++w) {
    start += s_before[w];
    if (w < wid) start += s_warp[w];
  }
  start += incl - r.need;
  if (tid < nb) {
    s_cached[tid] = r.cached;
    s_fresh[tid] = r.fresh;
    s_have[tid] = r.have;
    s_need[tid] = r.need;
    s_start[tid] = start;
    if (b0 + tid == a.B - 1 && blockIdx.y == 0 && a.free_head_out) {
      const long long end = start + r.need;
      *a.free_head_out = end < a.n_free ? (int)end : a.n_free;
    }
  }
  __syncthreads();

  // The block of page j >= have of the group's request i, or -1.
  auto fresh_block = [&](int i, int j) {
    const long long src = s_start[i] + (j - s_have[i]);
    if (src >= a.n_free) {
      bits |= kErrNoFreePage;
      return -1;
    }
    const int id = __ldg(a.free_list + src);
    if (id < 0 || id >= a.n_blocks) {
      bits |= kErrPageClamped;
      return -1;
    }
    return id;
  };

  // new table entries: a warp per request, the CTAs of a group in turns
  for (int i = wid; i < nb; i += kTabThreads / 32)
    for (int n = blockIdx.y * 32 + lane; n < s_need[i]; n += gridDim.y * 32)
      a.page_table[(int64_t)(b0 + i) * a.ld_pt + s_have[i] + n] = fresh_block(i, s_have[i] + n);

  const int t0 = blockIdx.y * tchunk;
  const int tn = a.T - t0 < tchunk ? a.T - t0 : tchunk;
  for (int w = tid; w < nb * tn; w += kTabThreads) {
    const int i = w / tn, t = t0 + (w - i * tn);
    int slot = -1, keys = 0;
    if (t < s_fresh[i]) {
      const int pos = s_cached[i] + t, j = pos / a.P;
      int id;
      if (j < s_have[i]) {
        id = __ldg(a.page_table + (int64_t)(b0 + i) * a.ld_pt + j);
        if (id < 0 || id >= a.n_blocks) {
          bits |= kErrPageClamped;
          id = -1;
        }
      } else {
        id = fresh_block(i, j);
      }
      if (id >= 0) {
        slot = id * a.P + (pos - j * a.P);
        keys = pos + 1;
      }
    }
    const int64_t o = (int64_t)(b0 + i) * a.T + t;
    a.slots[o] = slot;
    a.key_counts[o] = keys;
    a.page_counts[o] = (keys + a.P - 1) / a.P;
  }
  if (bits) atomicOr(a.status, bits);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesArgs& a, cudaStream_t stream) {
  // a group of requests per CTA while it maps about kTabTokens tokens; a
  // longer chunk of one request is cut over the grid's y
  const int fit = kTabTokens / a.T;
  const int group = fit < 1 ? 1 : (fit < kTabThreads ? fit : kTabThreads);
  const int tchunk = a.T < kTabTokens ? a.T : kTabTokens;
  const int gy = (a.T + tchunk - 1) / tchunk;
  const dim3 grid((a.B + group - 1) / group, gy < 65535 ? gy : 65535);
  const int chunk = (a.T + (int)grid.y - 1) / (int)grid.y;
  kv_tables_kernel<<<grid, kTabThreads, 0, stream>>>(a, group, chunk);
  return cudaGetLastError();
}

}  // namespace idx
