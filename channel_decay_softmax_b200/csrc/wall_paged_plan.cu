// wall_paged_plan.cu -- the block table, row offsets and slot map of one
// serving step, built on the GPU from the requests' lengths, and the return
// of finished requests' pages to the free stack.
//
// A step's plan is two prefix sums over the requests (their new tokens, and
// the pages those open beyond the ones held) and two scatters (the opened
// pages into the block table, the tokens into slots).  There is nothing to
// read but a few words a request and nothing to write but 8 bytes a token, so
// latency is all: one CTA scans 1024 requests at a time and opens the pages;
// the slots follow in the same launch while they are few, or from a grid of
// their own.  Measured: 4.0 us for five requests; 5.9 + 5.3 for 2048 (each row's
// slot follows from a search among the offsets that the first kernel writes).
#include "wall_internal.h"
#include "wall_paged.cuh"

namespace wall {
namespace {

using namespace paged;

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int* new_lens;
  const int* lens;
  int* table;
  const int* free_list;
  const int* free_count;
  int N, MP, NP, shift, T;
  int* cu;
  int* kv;
  long long* slots;
  int* admitted;
  int* lens_out;
  int* free_out;
  int* status;
};

// Inclusive sum over the CTA's kPlanThreads threads; `total` is the sum of all.
__device__ __forceinline__ long long block_incl_sum(long long x, long long* sw, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long in1 = paged::warp_incl_sum(x);
  __syncthreads();  // the previous sum's readers are done with sw
  if (lane == 31) sw[warp] = in1;
  __syncthreads();
  if (warp == 0) {
    const long long s = paged::warp_incl_sum(sw[lane]);
    sw[lane] = s;
  }
  __syncthreads();
  total = sw[31];
  return in1 + (warp > 0 ? sw[warp - 1] : 0);
}

// The slot of every token of the window [t0, t1) whose request is among
// [lo, hi] (request hi + 1 begins past the window).
__device__ __forceinline__ void write_slot(const PlanArgs& a, int t, int lo, int hi) {
  while (lo < hi) {  // the last request that begins at or before t
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  long long slot = -1;
  const int c0 = a.cu[lo], c1 = a.cu[lo + 1], kv = a.kv[lo];
  if (t < c1 && kv > 0) {
    const int pos = kv - (c1 - c0) + (t - c0);
    const int page = a.table[(long)lo * a.MP + (pos >> a.shift)];
    slot = ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1));
  }
  a.slots[t] = slot;
}

// Requests in order; the first whose pages exceed the stack and every later
// one that needs a page are refused (their cumulative need exceeds it too), so
// the admitted requests' pages are the top of the stack, in request order.
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(PlanArgs a, int slots_here) {
  __shared__ long long sw[32];
  start_next();
  const int lane = threadIdx.x & 31;
  const int PS1 = (1 << a.shift) - 1;
  int n_free = *a.free_count;
  if (threadIdx.x == 0 && (n_free < 0 || n_free > a.NP)) record_status(a.status, WALL_ERR_INVALID_ARG);
  n_free = min(max(n_free, 0), a.NP);
  long long rows0 = 0, need0 = 0;  // of the requests before these
  long long used = 0;
  for (int i0 = 0; i0 < a.N; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const bool real = i < a.N;
    const int nw_raw = real ? a.new_lens[i] : 0, len_raw = real ? a.lens[i] : 0;
    if (nw_raw < 0 || len_raw < 0) record_status(a.status, WALL_ERR_INVALID_ARG);
    const long long nw = max(nw_raw, 0), len = max(len_raw, 0);
    long long tot;
    const long long rows = rows0 + block_incl_sum(nw, sw, tot);
    rows0 += tot;
    const long long held = (len + PS1) >> a.shift, want = (len + nw + PS1) >> a.shift;
    const bool fits = want <= a.MP && rows <= a.T && len + nw <= 0x7fffffffll;
    const int need = real && fits ? (int)(want - held) : 0;
    const long long upto = need0 + block_incl_sum(need, sw, tot);
    need0 += tot;
    const bool in = real && fits && (need == 0 || upto <= n_free);
    // a row offset past the packed rows is no offset: clamped to their count
    if (real) {
      a.cu[i + 1] = (int)min(rows, (long long)a.T);
      a.kv[i] = in ? (int)(len + nw) : 0;
      a.admitted[i] = in ? 1 : 0;
      a.lens_out[i] = in ? (int)(len + nw) : (int)len;
    }
    if (i == 0) a.cu[0] = 0;
    if (in && need > 0) used = upto;
    // the opened pages: each thread its own while they are few, the warp
    // together for a prompt's
    const int mine = in ? need : 0;
    const long long rank = upto - need;  // pages opened before this request's
    if (mine > 0 && mine <= 4)
      for (int x = 0; x < mine; ++x)
        a.table[(long)i * a.MP + held + x] = a.free_list[n_free - 1 - (rank + x)];
    unsigned many = __ballot_sync(0xffffffffu, mine > 4);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int cnt = __shfl_sync(0xffffffffu, mine, src);
      const long long r0 = __shfl_sync(0xffffffffu, rank, src);
      const long long h0 = __shfl_sync(0xffffffffu, held, src);
      int* row = a.table + (long)(i - lane + src) * a.MP + h0;
      for (int x = lane; x < cnt; x += 32) row[x] = a.free_list[n_free - 1 - (r0 + x)];
    }
  }
  // the pages opened in all: the largest admitted cumulative need
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const long long y = __shfl_xor_sync(0xffffffffu, used, d);
    used = y > used ? y : used;
  }
  __syncthreads();  // cu, kv and the table are written (this CTA reads them below)
  if (lane == 0) sw[threadIdx.x >> 5] = used;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) used = sw[w] > used ? sw[w] : used;
    *a.free_out = n_free - (int)used;
    if (a.N == 0) a.cu[0] = 0;
  }
  if (slots_here)
    for (int t = threadIdx.x; t < a.T; t += kPlanThreads) {
      if (a.N > 0) write_slot(a, t, 0, a.N - 1);
      else a.slots[t] = -1;
    }
}

// Slots of kSlotRows packed rows a CTA: the requests that the rows touch are
// found by counting (every thread a share of the offsets), so the search for
// each row runs over those alone.
constexpr int kSlotRows = 1024, kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(PlanArgs a) {
  __shared__ int s_lo, s_hi;
  wait_before();
  const int t0 = blockIdx.x * kSlotRows, t1 = min(t0 + kSlotRows, a.T);
  if (threadIdx.x == 0) s_lo = s_hi = 0;
  __syncthreads();
  int lo = 0, hi = 0;  // requests that begin at or before the first / last row
  for (int i = 1 + threadIdx.x; i < a.N; i += kSlotThreads) {
    const int c = a.cu[i];
    lo += c <= t0;
    hi += c <= t1 - 1;
  }
  atomicAdd(&s_lo, lo);
  atomicAdd(&s_hi, hi);
  __syncthreads();
  for (int t = t0 + threadIdx.x; t < t1; t += kSlotThreads) write_slot(a, t, s_lo, s_hi);
}

// Finished requests' pages back on the stack, in request order, each request's
// in table order; their table rows become -1 and their lengths 0.  An entry that
// is no page is reported and dropped: a plan that opened it would lose tokens
// of a request that has nothing to do with it.
//
// The held entries of 1024 requests lie in one order, 8192 a round, and the pages
// among them are counted before any is stored.  64 requests of 60 pages 4.2 us,
// 1000 of 30 20.5, 4 of 1000 6.1.  (A warp for each request's entries, one request
// after the other: 30, 33 and 21 with the pages counted first, 20, 18 and 27 when
// they were not.)
constexpr int kReleaseEach = 8;
__global__ void __launch_bounds__(kPlanThreads, 1)
    release_kernel(const int* finished, int* lens, int* table, int* free_list, int* free_count,
                   int N, int MP, int NP, int shift, int* status) {
  __shared__ long long sw[32];
  __shared__ long long s_end[kPlanThreads];  // held entries up to and with each request
  __shared__ int s_pages[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int PS1 = (1 << shift) - 1;
  int n_free = *free_count;
  if (tid == 0 && (n_free < 0 || n_free > NP)) record_status(status, WALL_ERR_INVALID_ARG);
  n_free = min(max(n_free, 0), NP);
  long long before = n_free;
  for (int i0 = 0; i0 < N; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const bool done = i < N && finished[i] != 0;
    const int held = done ? (int)min((long long)MP, ((long long)max(lens[i], 0) + PS1) >> shift) : 0;
    if (done) lens[i] = 0;
    long long total;
    const long long end = block_incl_sum(held, sw, total);
    s_end[tid] = end;
    __syncthreads();
    for (long long e0 = 0; e0 < total; e0 += kPlanThreads * kReleaseEach) {
      // a warp's entries of the round are neighbours, 32 at a time
      const long long w0 = e0 + (long long)(tid & ~31) * kReleaseEach + lane;
      int* at[kReleaseEach];
      int id[kReleaseEach];
      int r = 0;  // the requests that end at or before the entry
#pragma unroll
      for (int step = kPlanThreads / 2; step > 0; step >>= 1)
        if (s_end[r + step - 1] <= w0) r += step;
#pragma unroll
      for (int x = 0; x < kReleaseEach; ++x) {
        const long long e = w0 + 32 * x;
        while (e < total && s_end[r] <= e) ++r;
        at[x] = e < total ? table + (long)(i0 + r) * MP + (e - (r > 0 ? s_end[r - 1] : 0)) : nullptr;
      }
#pragma unroll
      for (int x = 0; x < kReleaseEach; ++x) id[x] = at[x] ? *at[x] : -1;
      unsigned page[kReleaseEach];
      int n = 0;  // pages among the warp's entries
#pragma unroll
      for (int x = 0; x < kReleaseEach; ++x) {
        page[x] = __ballot_sync(0xffffffffu, (unsigned)id[x] < (unsigned)NP);
        n += __popc(page[x]);
      }
      if (lane == 0) s_pages[tid >> 5] = n;
      __syncthreads();
      int upto = s_pages[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      long long to = before + __shfl_sync(0xffffffffu, upto, tid >> 5) - n;
      before += __shfl_sync(0xffffffffu, upto, 31);
      __syncthreads();  // s_pages has been read
#pragma unroll
      for (int x = 0; x < kReleaseEach; ++x) {
        const long long mine = to + __popc(page[x] & ((1u << lane) - 1));
        to += __popc(page[x]);
        if (!at[x]) continue;
        *at[x] = -1;
        // no page, or more of them than the pool has: the table was not this stack's
        if (((page[x] >> lane) & 1u) && mine < NP) free_list[mine] = id[x];
        else record_status(status, WALL_ERR_INVALID_ARG);
      }
    }
    __syncthreads();  // s_end has been read
  }
  if (tid == 0) *free_count = (int)min(before, (long long)NP);
}

}  // namespace

// Tokens up to which the planning CTA writes the slots itself; beyond, a
// second launch with a CTA per 1024 rows.  (256 requests of 8, 16 and 32 tokens:
// 6.3, 8.3 and 10.7 us by the planning CTA, 10.4 in all three with the second
// launch; 2048 requests of 1, 2 and 4: 12.4, 14.4 and 18.5 against 14.6.)
constexpr int kSlotsHere = 4096;

int paged_plan(const int* new_lens, const int* lens, int* table, const int* free_list,
               const int* free_count, int N, int MP, int NP, int shift, int T, int* cu, int* kv,
               int64_t* slots, int* admitted, int* lens_out, int* free_out, cudaStream_t stream) {
  PlanArgs a;
  a.new_lens = new_lens; a.lens = lens; a.table = table; a.free_list = free_list;
  a.free_count = free_count; a.N = N; a.MP = MP; a.NP = NP; a.shift = shift; a.T = T;
  a.cu = cu; a.kv = kv; a.slots = reinterpret_cast<long long*>(slots); a.admitted = admitted;
  a.lens_out = lens_out; a.free_out = free_out; a.status = device_status();
  const bool here = T <= kSlotsHere || N == 0;
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, here ? 1 : 0);
  if (cudaGetLastError() != cudaSuccess) return WALL_ERR_CUDA;
  if (here) return WALL_OK;
  return launch_behind(slots_kernel, (T + kSlotRows - 1) / kSlotRows, kSlotThreads, 0, stream, a);
}

int paged_release(const int* finished, int* lens, int* table, int* free_list, int* free_count,
                  int N, int MP, int NP, int shift, cudaStream_t stream) {
  if (N == 0) return WALL_OK;
  release_kernel<<<1, kPlanThreads, 0, stream>>>(finished, lens, table, free_list, free_count, N,
                                                 MP, NP, shift, device_status());
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

}  // namespace wall
