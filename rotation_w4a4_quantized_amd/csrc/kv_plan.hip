// kv_plan: page tables, slots and positions of a step's tokens from the
// requests' lengths.
//
// The pages of ended requests are pushed on the stack of free pages in the
// order of the requests, then every request pops what it needs, in order. With
// the running sums of pages given back and of pages needed, entry i of the
// stack after the pushes is known without building it: free[i] below the old
// top, else a page of an ended request. So each workgroup makes the sums for
// itself (B <= 4096 requests, 256 threads), fills its share of the tables and
// of the tokens, and none waits for another: one launch. Reads and writes never
// meet: pushes go above the old top, popped pages into table entries past a
// live request's pages, and both are read only below those.
//
// Bound by latency: the loads of the lengths, two block scans and a search in
// LDS of log2(B) steps before the first table entry can be asked for: 3 requests
// 5.5 us by graph, 256 requests with tables of 2048 pages 9.3 us (90 KB), 4096
// requests 26 us; 64 prompts of up to 4096 tokens 9.4 us (2.0 MB, 0.2 TB/s).
#include <algorithm>

#include "kv_common.hpp"
#include "launch.hpp"

namespace rw4 {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kSat = 1 << 30;  // sums saturate here (every size is below it, so a sum of rows there is past T)

__device__ __forceinline__ int sat_add(int a, int b) {   // a, b in [0, kSat]
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(kSat)));
}

// saturating sum of the values of the threads before this one
__device__ __forceinline__ int block_scan(int v, int* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v = sat_add(v, u);
  }
  if (lane == 63) part[wave] = v;
  __syncthreads();
  v = __shfl_up(v, 1, 64);
  if (lane == 0) v = 0;
  for (int w = 0; w < wave; ++w) v = sat_add(v, part[w]);
  __syncthreads();
  return v;
}

// first index in [0, n) whose running sum exceeds i (n if none)
__device__ __forceinline__ int upper(const int* end, int n, int i) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(KvPlanArgs p) {
  extern __shared__ int lds[];
  int* cu = lds;                 // [B + 1]: row offsets
  int* back = cu + p.B + 1;      // [B]: running sum of pages given back
  int* need = back + p.B;        // [B]: running sum of pages needed
  __shared__ int part[kPlanThreads / 64];
  const int B = static_cast<int>(p.B), T = static_cast<int>(p.T), lg = p.lg_page;
  const int tid = threadIdx.x, per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  const int64_t most = p.max_pages << lg;   // tokens that a table row can hold

  int sum = 0;
  for (int b = b0; b < b1; ++b) sum = sat_add(sum, min(max(p.new_len[b], 0), kSat));
  int at = block_scan(sum, part);
  if (tid == 0) cu[0] = 0;
  for (int b = b0; b < b1; ++b) {
    at = sat_add(at, min(max(p.new_len[b], 0), kSat));
    cu[b + 1] = at;                         // not yet cut to T: a request past T is refused
  }
  __syncthreads();

  auto lengths = [&](int b, int64_t& ctx, int64_t& cnt, bool& ended, bool& bad) {
    ctx = p.ctx_len[b];
    const int64_t n = p.new_len[b];
    cnt = n > 0 ? n : 0;
    ended = n == -1;
    bad = ctx < 0 || ctx > most || n < -1 || ctx + cnt > most || cu[b + 1] > T;
  };
  auto pages = [&](int64_t tokens) { return static_cast<int>((tokens + (int64_t(1) << lg) - 1) >> lg); };
  int sb = 0, sn = 0;
  for (int b = b0; b < b1; ++b) {
    int64_t ctx, cnt;
    bool ended, bad;
    lengths(b, ctx, cnt, ended, bad);
    if (!bad) {
      if (ended) sb = sat_add(sb, pages(ctx));
      else sn = sat_add(sn, pages(ctx + cnt) - pages(ctx));
    }
    back[b] = sb;
    need[b] = sn;
  }
  const int eb = block_scan(sb, part), en = block_scan(sn, part);
  for (int b = b0; b < b1; ++b) {
    back[b] = sat_add(back[b], eb);
    need[b] = sat_add(need[b], en);
  }
  __syncthreads();

  const int cap = static_cast<int>(p.capacity);
  const int had_free = min(max(p.n_free[0], 0), cap);
  const int top = min(sat_add(had_free, back[B - 1]), cap);   // of the stack after the pushes
  const int64_t width = p.max_pages;
  // entry i of the stack after the pushes, 0 <= i < top
  auto stack_at = [&](int i) {
    if (i < had_free) return p.free_pages[i];
    const int k = i - had_free, b = upper(back, B, k);
    return p.page_table[b * width + (k - (b ? back[b - 1] : 0))];
  };
  auto served = [&](int b, bool bad) {
    const int start = b ? need[b - 1] : 0;
    return !bad && (need[b] == start || need[b] <= top);
  };

  const int gid = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
  // pages given back
  for (int i = gid; i < top - had_free; i += stride) p.free_pages[had_free + i] = stack_at(had_free + i);
  // pages taken: requests are served in order, so the pages that are taken are
  // the first ones asked for, up to the last request that fits
  const int fit = upper(need, B, top);      // requests before it end at or below top
  const int taken = fit ? need[fit - 1] : 0;
  for (int i = gid; i < taken; i += stride) {
    const int b = upper(need, B, i);
    p.page_table[b * width + pages(p.ctx_len[b]) + (i - (b ? need[b - 1] : 0))] = stack_at(top - 1 - i);
  }
  // tokens
  const int rows = min(cu[B], T);
  for (int t = gid; t < T; t += stride) {
    int64_t slot = -1;
    int pos = -1;
    if (t < rows) {
      const int b = upper(cu + 1, B, t);
      int64_t ctx, cnt;
      bool ended, bad;
      lengths(b, ctx, cnt, ended, bad);
      if (served(b, bad)) {
        pos = static_cast<int>(ctx) + t - cu[b];
        const int pi = pos >> lg, have = pages(ctx);
        const int id = pi < have ? p.page_table[b * width + pi]
                                 : stack_at(top - 1 - ((b ? need[b - 1] : 0) + pi - have));
        slot = (static_cast<int64_t>(id) << lg) + (pos & ((1 << lg) - 1));
      }
    }
    p.slot[t] = slot;
    p.pos[t] = pos;
  }
  if (blockIdx.x != 0) return;
  for (int b = tid; b < B; b += kPlanThreads) {
    int64_t ctx, cnt;
    bool ended, bad;
    lengths(b, ctx, cnt, ended, bad);
    const bool ok = served(b, bad);
    p.cu_new[b + 1] = min(cu[b + 1], T);
    p.kv_len[b] = ok && !ended ? static_cast<int>(ctx + cnt) : 0;
    p.status[b] = bad ? 2 : ok ? 0 : 1;
    if (p.ctx_next) p.ctx_next[b] = !ok ? static_cast<int>(ctx) : ended ? 0 : static_cast<int>(ctx + cnt);
  }
  if (tid == 0) {
    p.cu_new[0] = 0;
    p.n_free_out[0] = top - taken;
  }
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanArgs& a, hipStream_t s) {
  // A workgroup for every 256 tokens, or 1024 entries of the page tables (the
  // pages that move are not known here): a thread's lookups follow one another.
  // 8 requests of 2048 new tokens: 64 workgroups 6.3 us, 8: 11.6, one: 51.7; 64
  // ended requests of up to 4096 pages: 256 workgroups 7.0 us, 32: 14.5, one: 296;
  // 64 requests of up to 4096 new tokens: 512 workgroups 9.4 us, 256: 10.3, 128: 13.4.
  // No more for the table's sake than CUs: 4096 single tokens 33.9 us with 512, 26.4
  // with 16 to 256.
  const int64_t for_tokens = std::min<int64_t>((a.T + 255) / 256, 2 * device_cus());
  const int64_t for_table = std::min<int64_t>((a.B * a.max_pages + 1023) / 1024, device_cus());
  const int64_t groups = std::max(for_tokens, for_table);
  plan_kernel<<<dim3(static_cast<unsigned>(groups)), kPlanThreads,
                static_cast<size_t>(3 * a.B + 1) * sizeof(int), s>>>(a);
  return hipGetLastError();
}

}  // namespace rw4
