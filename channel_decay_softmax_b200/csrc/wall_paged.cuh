// wall_paged.cuh -- what the paged-cache kernels share: the fixed-point gate
// prefix, bounded views of the request arrays, and the division of a ragged
// batch's key tiles over a grid.
//
// Layout of the paged Wall cache (one per layer): pages of PS positions,
//   k_pages [NP, HQ, PS, K]  k * 2^(R_c - P), head-major inside a page, so the
//                            rows one query head reads are PS * K contiguous
//                            elements (16 KB at PS = 64, K = 128, bf16)
//   v_pages [NP, H, PS, V]
//   r_pages [NP, HQ, K]      int32 anchors R_c, whole powers of two
// The prefix P is fixed point (24 fraction bits in 64): sums of gates are
// exact in every order, so a prompt appended in one piece, in chunks or token
// by token leaves the same bits, and P at position 10^6 is as fine as at 1.
// Anchors are whole numbers, so 2^(R_a - R_b) is an exact factor of a bf16
// operand.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "wall_common.cuh"

namespace wall {
namespace paged {

// Most of a call's kernels behind its first are launched while the one before
// still runs (launch_behind): that one lets them start (start_next), and they
// wait for it to have ended (wait_before) ahead of the first word that they
// read of it, or write that it reads.  Every CTA waits, on every path, so that
// the end of one means the end of all before it.  A call's first kernel is
// launched in stream order: all of them may read the call's inputs at once.
// Three single-token requests' attention takes 10.3 us so instead of 12.3, a
// mixed step (plan, append, attention) 132.9 instead of 137.6, uncaptured 140
// instead of 158.
__device__ __forceinline__ void start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
int launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                  const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

constexpr int kFrac = 24;
constexpr float kOne = 16777216.f;                 // 2^24
constexpr float kStep = 1.f / 16777216.f;          // 2^-24
constexpr float kGateFix = kInvLn2 * 16777216.f;   // fp32: 2^24 / ln 2
// A page's prefix may leave its anchor by at most this many powers of two:
// the key rows 2^(R_c - P) then stay normal numbers for |k| up to 2^26.
constexpr float kPageRange = 100.f;

// One token's gate in fixed point: rint of the fp32 product, clamped to 32
// signed bits (a single step of -128 powers of two forgets everything);
// 0 for NaN (the caller spreads the NaN itself).  The instruction saturates.
__device__ __forceinline__ int gate_fixed(float g) { return __float2int_rn(g * kGateFix); }
// The anchor of a page whose first position has prefix P: floor(P + 1/2).
__device__ __forceinline__ int page_anchor(long long P) {
  return (int)((P + (1ll << (kFrac - 1))) >> kFrac);
}

// The packed batch: request i owns rows [cu[i], cu[i+1]) of q, and keys
// [0, kv[i]) of its pages.  Offsets are clamped into [0, T] and lengths past
// `cap` (what the block table can hold) read as 0, a refused request's, so that
// a bad array can send a kernel neither out of bounds nor through tiles without
// end.
struct Batch {
  const int* cu;
  const int* kv;
  int N;
  int T;
  int cap;
  __device__ __forceinline__ int keys(int i) const {
    const int n = kv[i];
    return n > cap ? 0 : n;
  }
  __device__ __forceinline__ int clamp_row(int r) const { return min(max(r, 0), T); }
  __device__ __forceinline__ int start(int i) const { return clamp_row(cu[i]); }
  __device__ __forceinline__ int rows(int i) const {
    return max(0, clamp_row(cu[i + 1]) - clamp_row(cu[i]));
  }
};

// ---------------------------------------------------------------------------
// Units of attention work.  A request's n query rows are cut into blocks of
// TB rows; a unit is (request, head, block), its work the TB-key tiles that
// some row of the block sees.  The block's first row sits at position
// ctx + b * TB (any alignment), so a full block's last tile is b + c1 with
// c1 = floor((ctx + TB - 1) / TB), and with a window its first one
// max(0, b + f): the tiles before block b are closed forms, and neither a
// table nor a loop is needed to find the work of a range.
//
// A request with fewer keys than rows (kv < n: one that the page plan
// refused has kv = 0) sees nothing: its units have one empty tile each.
struct Request {
  int i, t0, n, kv, ctx;  // row range, keys, position of its first row
  int nb;                 // blocks
  int c1, last, f;        // see above; last: last tile of the last block
  bool dead;
};

template <int TB>
__device__ __forceinline__ int floor_tile(int x) {
  static_assert((TB & (TB - 1)) == 0, "a power of two");
  return x >> (TB == 128 ? 7 : TB == 64 ? 6 : 5);  // arithmetic shift: floor for x < 0 too
}

template <int TB>
__device__ __forceinline__ Request request_of(const Batch& bt, int i, int window) {
  Request r;
  r.i = i;
  r.t0 = bt.start(i);
  r.n = bt.rows(i);
  r.kv = bt.keys(i);
  r.ctx = r.kv - r.n;
  r.dead = r.kv < r.n;
  r.nb = (r.n + TB - 1) / TB;
  r.c1 = floor_tile<TB>(r.ctx + TB - 1);
  r.last = floor_tile<TB>(r.ctx + r.n - 1);
  r.f = window > 0 ? floor_tile<TB>(r.ctx - window + 1) : -(1 << 28);
  return r;
}
__device__ __forceinline__ int tile_lo(const Request& r, int b) {
  return r.dead ? 0 : max(0, b + r.f);
}
__device__ __forceinline__ int tile_hi(const Request& r, int b) {
  return r.dead ? 0 : (b < r.nb - 1 ? b + r.c1 : r.last);
}
__device__ __forceinline__ int unit_tiles(const Request& r, int b) {
  return tile_hi(r, b) - tile_lo(r, b) + 1;
}
// tiles of blocks [0, b), b < nb (all full blocks)
__device__ __forceinline__ long long tiles_before(const Request& r, int b) {
  if (r.dead) return b;
  const long long m = b;
  long long s = m * (m - 1) / 2 + m * (r.c1 + 1);  // sum of (x + c1 + 1)
  const long long k = m - 1 + r.f;                 // the last of them starts at max(0, k)
  if (k > 0) {
    const long long lo = r.f > 0 ? r.f : 1;        // sum of max(0, x + f), x < b
    s -= (lo + k) * (k - lo + 1) / 2;
  }
  return s;
}
__device__ __forceinline__ long long tiles_per_head(const Request& r) {
  return tiles_before(r, r.nb - 1) + unit_tiles(r, r.nb - 1);
}

// Which requests a kernel takes: those of n_min to n_max rows.
struct Pick {
  int n_min, n_max;
};

// What a CTA spends on a unit beside its tiles (its queries' load, the first
// and the masked tiles' longer softmax, the epilogue) counts as U tiles in
// front of them: a unit has U + tiles places.
template <int TB, int U>
__device__ __forceinline__ long long request_places(const Batch& bt, int i, int window, int heads,
                                                    const Pick& pk) {
  const int n = bt.rows(i);
  if (n < pk.n_min || n > pk.n_max || n == 0) return 0;
  const Request r = request_of<TB>(bt, i, window);
  return heads * (tiles_per_head(r) + (long long)U * r.nb);
}

// A CTA's position in the flattened places (request, head, block, place).
struct Cursor {
  Request r;
  int h, b;      // unit
  int p;         // place in the unit
  int n_tiles;   // the unit's tiles
};
// The tiles [ta, tb) of the unit among the next `left` places, and how many of
// the places the unit takes.  (ta == tb: only places before its first tile.)
struct Run {
  int ta, tb, places;
};
template <int U>
__device__ __forceinline__ Run run_of(const Cursor& c, long long left) {
  Run r;
  const long long to_end = U + c.n_tiles - c.p;
  r.places = (int)(left < to_end ? left : to_end);
  r.ta = max(0, c.p - U);
  r.tb = max(0, c.p + r.places - U);
  return r;
}

// The division: CTA c of G takes places [W c / G, W (c+1) / G) of the batch's
// W, so every CTA gets the same work to within one tile, whatever the lengths.
// A unit cut by a boundary is joined afterwards from its parts.
struct Share {
  long long W;
  int G;
  __device__ __forceinline__ long long begin(int c) const { return W * c / G; }
  // the CTA that holds place x
  __device__ __forceinline__ int owner(long long x) const {
    return (int)(((x + 1) * G + W - 1) / W) - 1;
  }
  // the CTA that holds the last tile of a unit whose place p is place x
  template <int U>
  __device__ __forceinline__ int last_owner(const Cursor& c, long long x) const {
    return owner(x - c.p + U + c.n_tiles - 1);
  }
};

// Scratch of the start search (shared memory).
struct FindScratch {
  long long warp_sum[32];
  long long total;
  long long base;
  int req;
};

__device__ __forceinline__ long long warp_incl_sum(long long x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if ((int)(threadIdx.x & 31) >= d) x += y;
  }
  return x;
}

// Called by all threads of the CTA.  Fills `sh` (the division) and, when this
// CTA has work, `fs.req` and `fs.base`: the request that holds its first place
// and the places before that request.  No more CTAs share the work than leave
// each `least` places.
template <int TB, int U>
__device__ __forceinline__ bool find_start(const Batch& bt, int window, int heads, const Pick& pk,
                                           int least, int cta, int n_cta, FindScratch& fs,
                                           Share& sh) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int nw = (nt + 31) >> 5;
  long long mine = 0;
  for (int i = tid; i < bt.N; i += nt) mine += request_places<TB, U>(bt, i, window, heads, pk);
  // the total (and, when each thread has one request, the scan itself)
  const long long incl = warp_incl_sum(mine);
  if (lane == 31) fs.warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const long long v = lane < nw ? fs.warp_sum[lane] : 0;
    const long long s = warp_incl_sum(v);
    if (lane < nw) fs.warp_sum[lane] = s - v;  // exclusive
    if (lane == 31) fs.total = s;
  }
  __syncthreads();
  sh.W = fs.total;
  const long long most = (sh.W + least - 1) / least;
  sh.G = (int)(most < n_cta ? most : n_cta);
  if (cta >= sh.G) return false;
  const long long x = sh.begin(cta);
  if (bt.N <= nt) {
    const long long after = fs.warp_sum[warp] + incl;
    if (x >= after - mine && x < after) {
      fs.req = tid;
      fs.base = after - mine;
    }
    __syncthreads();
    return true;
  }
  long long before = 0;
  for (int i0 = 0; i0 < bt.N; i0 += nt) {
    const int i = i0 + tid;
    const long long one = i < bt.N ? request_places<TB, U>(bt, i, window, heads, pk) : 0;
    const long long in1 = warp_incl_sum(one);
    __syncthreads();
    if (lane == 31) fs.warp_sum[warp] = in1;
    __syncthreads();
    long long off = before;
    for (int w = 0; w < warp; ++w) off += fs.warp_sum[w];
    const long long after = off + in1;
    if (x >= after - one && x < after) {
      fs.req = i;
      fs.base = after - one;
    }
    for (int w = 0; w < nw; ++w) before += fs.warp_sum[w];
    if (x < before) break;  // the same for all threads
  }
  __syncthreads();
  return true;
}

// The cursor at flattened place x, x inside request `req`, which begins at `base`.
template <int TB, int U>
__device__ __forceinline__ Cursor cursor_at(const Batch& bt, int window, int req, long long base,
                                            long long x) {
  Cursor c;
  c.r = request_of<TB>(bt, req, window);
  long long rem = x - base;
  const long long per_head = tiles_per_head(c.r) + (long long)U * c.r.nb;
  c.h = (int)(rem / per_head);
  rem -= c.h * per_head;
  int lo = 0, hi = c.r.nb - 1;  // the last block that begins at or before rem
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tiles_before(c.r, mid) + (long long)U * mid <= rem) lo = mid;
    else hi = mid - 1;
  }
  c.b = lo;
  c.p = (int)(rem - tiles_before(c.r, lo) - (long long)U * lo);
  c.n_tiles = unit_tiles(c.r, lo);
  return c;
}

// To the next unit (there is one: the caller's places do not end here).
template <int TB>
__device__ __forceinline__ void next_unit(const Batch& bt, int window, int heads, const Pick& pk,
                                          Cursor& c) {
  c.p = 0;
  if (++c.b == c.r.nb) {
    c.b = 0;
    if (++c.h == heads) {
      c.h = 0;
      int i = c.r.i + 1;
      for (; i < bt.N; ++i) {
        const int n = bt.rows(i);
        if (n >= pk.n_min && n <= pk.n_max && n > 0) break;
      }
      if (i >= bt.N) return;
      c.r = request_of<TB>(bt, i, window);
    }
  }
  c.n_tiles = unit_tiles(c.r, c.b);
}

// What the merge of a cut unit needs, written by the CTA that begins it.
struct PartDesc {
  int t0, rows, h;  // first token; rows (tokens, or tokens x heads of a kv head); (kv) head
  int last_cta;     // < 0: this CTA begins no unit that another one ends
};

// A scaled query's channel x as an operand, y = x 2^e: finite where x is, at most
// the largest bf16 number.  Growth by 2^128 and more from a page to a row (whose
// keys there count 2^27 fold at least) then adds nothing where the query or the
// key is 0, instead of 0 * inf.  The callers look for such growth in a vector of
// channels first: done for each channel, this cost drafts 8 % and fp32 rows 5 %.
constexpr float kMostQuery = 3.38953139e38f;
__device__ __forceinline__ float bound_query(float y, float x) {
  return fabsf(y) > kMostQuery && fabsf(x) < INFINITY ? copysignf(kMostQuery, y) : y;
}
__device__ __forceinline__ float grown_query(float x, float e) {
  return bound_query(x * exp2f(e > 127.f ? 127.f : e), x);
}

// 2^(sink - m), in log2: a sink of -inf is none, also beside m = -inf (a row that
// sees nothing).
__device__ __forceinline__ float sink_weight(float sink, float m) {
  return sink == -INFINITY ? 0.f : exp2f(sink - m);
}

// A page's id, or -1 for an entry outside the pool (reported by the caller).
__device__ __forceinline__ int page_of(const int* table, long row, int slot, int num_pages) {
  const int id = table[row + slot];
  return (unsigned)id < (unsigned)num_pages ? id : -1;
}

}  // namespace paged
}  // namespace wall
