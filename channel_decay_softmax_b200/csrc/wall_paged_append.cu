// wall_paged_append.cu -- new tokens into the paged Wall cache: the gate
// prefix, the pages' anchors, the rescaled key rows and the value rows.
//
//   e_t = rint(g_t 2^24 / ln 2),  P_t = P_{t-1} + e_t   (fixed point)
//   R_c = floor(P + 1/2) at page c's first position
//   p_t = P_t - R_{page(t)},   k_pages row = k_t 2^(-p_t),   v_pages row = v_t
//
// Per (token, query head, channel) 2 bytes of g come in and 4 of p and 2 of
// the key row go out (bf16), with k and v shared by a group: memory-bound.
// Three ways, by how many tokens a request may bring:
//   one     a warp takes a request's 128 channels: no scan at all
//   few     a CTA takes one request and 64 channels and walks the tokens in
//           blocks aligned to the pages, shared by sixteen half-warps: every one
//           sums its own tokens' gates, the sums are scanned in shared memory, and
//           each then forms its tokens from its own prefix -- three barriers a
//           block, its loads all in flight at once
//   many    the blocks ("runs") side by side: a pass over g leaves each run's
//           sums, a scan over a request's runs makes them prefixes (exact in
//           any order, being integers), and the same kernel forms each run
//           from its own; g is read twice, the second time mostly from L2
// Measured: 48 requests of one token 3.3 us (four dependent loads); six prompts
// of 301 to 2500 tokens (110 MB, 16.8 us at the copy rate) 43 us, 35 of them the
// last pass, which issue bounds (64 % of the slots: 8 values' fixed-point steps,
// conversions and exp2 a thread and token).
#include "wall_internal.h"
#include "wall_paged.cuh"

namespace wall {
namespace {

using namespace paged;

constexpr int kWarps = 8;   // of a CTA
constexpr int kOneSlab = 128;  // one token a request: a warp's channels, four a lane
// Blocks of RL positions: a CTA takes 64 channels, sixteen half-warps of RL / 16
// tokens each, four channels a lane.  (CTAs of 128 channels and 512 threads
// keep the same threads resident in half as many CTAs, whose barriers then
// leave the SM idle: 40.5 against 38.6 us for six prompts of 301 to 2500 tokens.)
constexpr int kSlab = 64;
constexpr int W = 16;

struct AppendArgs {
  const void *k, *v, *g;
  Batch bt;
  const long long* slots;
  int H, HQ, K, V, shift, NP;
  void *kp, *vp;
  int* rp;
  const long long* carry_in;
  long long* carry_out;
  float* p;
  int* status;
  int k_slabs;
  long long* runs;  // [run, C]: sums of the runs' gates, then the prefixes before them
};

// Run r of request i -- its r-th block of RL positions -- has place
// cu[i] / RL + 2 i + r: a request of n rows has n / RL + 2 runs at most, so no
// two share a place, and a place's request is found without a table.
template <int RL>
struct Run {
  int i, t0, n, kv, ctx;  // the request (i < 0: the place is empty)
  int base;               // first position of the run's block
  bool none;              // nothing new, or refused by the plan (in its first place)
};
template <int RL>
__device__ __forceinline__ Run<RL> run_at(const Batch& bt, int place) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = bt.N;  // the last request whose places begin at or before this one
  while (len > 1) {
    const int step = (len + 31) / 32, x = lo + lane * step;
    const bool le = lane * step < len && bt.start(x) / RL + 2 * x <= place;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    len = min(step, len - (cnt - 1) * step);
    lo += (cnt - 1) * step;
  }
  Run<RL> r;
  r.i = lo;
  r.t0 = bt.start(lo);
  r.n = bt.rows(lo);
  r.kv = bt.keys(lo);
  r.ctx = r.kv - r.n;
  r.none = r.n == 0 || r.ctx < 0;
  const int k = place - (r.t0 / RL + 2 * lo);
  r.base = r.none ? 0 : (r.ctx / RL + k) * RL;
  if (r.none ? k != 0 : r.base >= r.kv) r.i = -1;
  return r;
}

template <typename T>
struct Quad;  // four consecutive elements
template <>
struct Quad<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* x) {
    u = *reinterpret_cast<const uint2*>(x);
  }
  __device__ __forceinline__ void zero() { u = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* x, const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(x) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <>
struct Quad<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* x) { u = *reinterpret_cast<const float4*>(x); }
  __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* x, const float* f) {
    *reinterpret_cast<float4*>(x) = make_float4(f[0], f[1], f[2], f[3]);
  }
};

// The prefix beyond the page's anchor, in 32 bits from token to token: inside a
// page's range it fits with room to spare.  (Before a page's first token it
// need not, and is then right modulo 2^32, as the token's own value is small.)
// What leaves the range is reported: a step that overflows (`lost` < 0), or a
// value past it.
__device__ __forceinline__ int from_anchor(long long P, int R) {
  return (int)(P - ((long long)R << kFrac));
}
__device__ __forceinline__ int add_step(int d, int e, int& lost) {
  const int s = (int)((unsigned)d + (unsigned)e);
  lost |= (d ^ s) & (e ^ s);
  return s;
}
// p of a token, and whether it leaves the range that the key row 2^-p k stays a
// number in.
__device__ __forceinline__ float token_prefix(int d, bool& wide) {
  const float p = __int2float_rn(d) * kStep;
  wide |= fabsf(p) > kPageRange;
  return p;
}

// A slot as the pool's position (below 2^31), or -1 (reported) where it lies
// outside the pool.
__device__ __forceinline__ int slot_row(long long slot, const AppendArgs& a, bool& bad) {
  if (slot < 0 || slot >> a.shift >= a.NP) {
    bad = true;
    return -1;
  }
  return (int)slot;
}

// Rows of one value slab (32 vectors of 16 bytes) of tokens [ta, tb).
template <typename T>
__device__ __forceinline__ void copy_values(const AppendArgs& a, int ta, int tb, int vslab) {
  const int warps = blockDim.x >> 5;
  constexpr int EV = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = (vslab * 32 + lane) * EV;
  if (ch >= a.H * a.V) return;
  const int h = ch / a.V, n = ch - h * a.V;
  const int mask = (1 << a.shift) - 1;
  const T* v = static_cast<const T*>(a.v);
  T* vp = static_cast<T*>(a.vp);
  for (int t = ta + warp; t < tb; t += warps) {
    bool bad = false;
    const int row = slot_row(a.slots[t], a, bad);
    if (bad) continue;  // the key slabs report it
    *reinterpret_cast<uint4*>(vp + ((((long)(row >> a.shift) * a.H + h) << a.shift) + (row & mask)) * a.V + n) =
        *reinterpret_cast<const uint4*>(v + (long)t * a.H * a.V + ch);
  }
}

// Gates and keys of this warp's tokens [xa, xb) of its TPW, zeros elsewhere.
template <typename T, int TPW>
__device__ __forceinline__ void load_tokens(const T* p, int stride, int xa, int xb, bool live,
                                            Quad<T> (&q)[TPW]) {
#pragma unroll
  for (int x = 0; x < TPW; ++x) {
    q[x].zero();
    if (x >= xa && x < xb && live) q[x].load(p + x * stride);
  }
}
// The tokens' gate steps and their sums; `nan`: some gate is none.
template <typename T, int TPW>
__device__ __forceinline__ void gate_steps(const Quad<T> (&g)[TPW], int (&step)[TPW][4],
                                           long long* out, bool& nan) {
  long long sum[4] = {0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < TPW; ++x) {
    float f[4];
    g[x].get(f);
    const float t = (f[0] + f[1]) + (f[2] + f[3]);
    nan |= t != t;  // (or infinities of both signs: looked at again)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      step[x][e] = gate_fixed(f[e]);
      sum[e] += step[x][e];
    }
  }
  longlong2* o = reinterpret_cast<longlong2*>(out);
  o[0] = make_longlong2(sum[0], sum[1]);
  o[1] = make_longlong2(sum[2], sum[3]);
}
__device__ __forceinline__ void load4(const long long* p, long long (&x)[4]) {
  const longlong2 u = reinterpret_cast<const longlong2*>(p)[0],
                  v = reinterpret_cast<const longlong2*>(p)[1];
  x[0] = u.x; x[1] = u.y; x[2] = v.x; x[3] = v.y;
}
__device__ __forceinline__ void store4(long long* p, const long long (&x)[4]) {
  reinterpret_cast<longlong2*>(p)[0] = make_longlong2(x[0], x[1]);
  reinterpret_cast<longlong2*>(p)[1] = make_longlong2(x[2], x[3]);
}

// Blocks of RL positions, a page or several.  kRuns: the CTA takes one run, from its prefix; else all blocks of request blockIdx.x.
template <typename T, int RL, bool kRuns>
__global__ void __launch_bounds__(kWarps * 32, RL == 64 && sizeof(T) == 2 ? 4 : 2)
    append_kernel(AppendArgs a) {
  constexpr int TPW = RL / W;
  __shared__ __align__(16) long long s_sum[W][kSlab];  // the groups' sums, then their prefixes
  __shared__ __align__(16) int s_first[RL / 32][kSlab];  // gate steps of the tokens that begin pages
  const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
  int i, t0, n, kv, base;
  bool none;
  if constexpr (kRuns) {
    const Run<RL> r = run_at<RL>(a.bt, blockIdx.x);
    if (r.i < 0) {
      wait_before();
      return;
    }
    i = r.i; t0 = r.t0; n = r.n; kv = r.kv; none = r.none; base = r.base;
  } else {
    i = blockIdx.x;
    t0 = a.bt.start(i); n = a.bt.rows(i); kv = a.bt.keys(i);
    none = n == 0 || kv < n;  // nothing new, or refused by the plan
    base = (kv - n) / RL * RL;
  }
  const int ctx = kv - n;
  if ((int)blockIdx.y >= a.k_slabs) {
    if (none) {
      if constexpr (kRuns) wait_before();
      return;
    }
    const int ta = kRuns ? t0 + max(base, ctx) - ctx : t0;
    const int tb = kRuns ? t0 + min(base + RL, kv) - ctx : t0 + n;
    copy_values<T>(a, ta, tb, blockIdx.y - a.k_slabs);
    if constexpr (kRuns) wait_before();
    return;
  }
  const int C = a.HQ * a.K;
  const int c = blockIdx.y * kSlab + lane * 4;
  const bool live = c < C;  // the last slab may be short
  const int h = live ? c / a.K : 0, ch = live ? c - h * a.K : 0;
  const int PS1 = (1 << a.shift) - 1;
  if (none) {
    if constexpr (kRuns) wait_before();
    if (live && grp == 0 && a.carry_out != a.carry_in) {
      long long x[4];
      load4(a.carry_in + (long)i * C + c, x);
      store4(a.carry_out + (long)i * C + c, x);
    }
    return;
  }
  const T* g = static_cast<const T*>(a.g) + c;
  const T* k = static_cast<const T*>(a.k) + h / (a.HQ / a.H) * a.K + ch;
  T* kp = static_cast<T*>(a.kp) + ch;
  // the prefix before the block, of the channel that this thread scans
  const int sc = blockIdx.y * kSlab + threadIdx.x;
  const bool scans = threadIdx.x < kSlab && sc < C;
  long long carry = 0;
  if (!kRuns && scans && ctx > 0) carry = a.carry_in[(long)i * C + sc];
  bool wide = false, bad = false;
  for (;; base += RL) {
    const int o0 = base + grp * TPW;  // this group's first position
    const int xa = max(0, ctx - o0), xb = min(TPW, kv - o0);  // its tokens [xa, xb)
    const int tw = t0 + o0 - ctx;  // their place among the packed rows (below 0 before the first)
    const int po = o0 & ~PS1;      // its page: TPW divides a page
    Quad<T> gq[TPW], kq[TPW];
    load_tokens(g + (long)tw * C, C, xa, xb, live, gq);
    load_tokens(k + (long)tw * a.H * a.K, a.H * a.K, xa, xb, live, kq);
    int row[TPW];
#pragma unroll
    for (int x = 0; x < TPW; ++x)
      row[x] = x >= xa && x < xb ? slot_row(a.slots[tw + x], a, bad) : -1;
    // a page begun by an earlier call: its anchor stands in the pool
    int4 R = make_int4(0, 0, 0, 0);
    if (xa < xb && po < ctx) {
      int first = -1;
#pragma unroll
      for (int x = TPW - 1; x >= 0; --x) first = x >= xa && x < xb ? row[x] : first;
      if (first >= 0 && live)
        R = *reinterpret_cast<const int4*>(a.rp + (long)(first >> a.shift) * C + c);
    }
    int step[TPW][4];
    bool nan = false;
    gate_steps(gq, step, &s_sum[grp][lane * 4], nan);
    if (po == o0)
      *reinterpret_cast<int4*>(&s_first[(o0 - base) >> 5][lane * 4]) =
          make_int4(step[0][0], step[0][1], step[0][2], step[0][3]);
    if constexpr (kRuns) {
      wait_before();
      if (scans) carry = a.runs[(long)blockIdx.x * C + sc];
    }
    __syncthreads();
    if (threadIdx.x < kSlab) {
#pragma unroll 4
      for (int w = 0; w < W; ++w) {
        const long long x = s_sum[w][threadIdx.x];
        s_sum[w][threadIdx.x] = carry;
        carry += x;
      }
    }
    __syncthreads();
    long long P[4];
    if (xa < xb && po >= ctx) {  // a page that begins here, at a token of this call
      load4(&s_sum[(po - base) / TPW][lane * 4], P);
      const int4 e = *reinterpret_cast<const int4*>(&s_first[(po - base) >> 5][lane * 4]);
      R = make_int4(page_anchor(P[0] + e.x), page_anchor(P[1] + e.y), page_anchor(P[2] + e.z),
                    page_anchor(P[3] + e.w));
      if (po == o0 && row[0] >= 0 && live)
        *reinterpret_cast<int4*>(a.rp + (long)(row[0] >> a.shift) * C + c) = R;
    }
    load4(&s_sum[grp][lane * 4], P);
    int d[4] = {from_anchor(P[0], R.x), from_anchor(P[1], R.y), from_anchor(P[2], R.z),
                from_anchor(P[3], R.w)};
    float* pw = a.p + (long)tw * C + c;
    int lost = 0;
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      if (x < xa || x >= xb || !live) continue;
      float kf[4], pv[4];
      kq[x].get(kf);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[e] = add_step(d[e], step[x][e], lost);
        pv[e] = token_prefix(d[e], wide);
      }
      if (x == 0 && po == o0) lost = 0;  // the page's first token
      if (nan) {  // a NaN gate makes its token's p and key row NaN
        float f[4];
        Quad<T> gx;
        gx.load(g + ((long)tw + x) * C);
        gx.get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) pv[e] = f[e] != f[e] ? f[e] : pv[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) kf[e] *= exp2f(-pv[e]);
      *reinterpret_cast<float4*>(pw + x * C) = make_float4(pv[0], pv[1], pv[2], pv[3]);
      if (row[x] >= 0)
        Quad<T>::store(kp + ((((long)(row[x] >> a.shift) * a.HQ + h) << a.shift) + (row[x] & PS1)) * a.K, kf);
    }
    wide |= lost < 0;
    if (kRuns || base + RL >= kv) break;
    __syncthreads();  // the prefixes have been read
  }
  if (scans && base + RL >= kv) a.carry_out[(long)i * C + sc] = carry;
  if (wide) record_status(a.status, WALL_ERR_RANGE);
  if (bad) record_status(a.status, WALL_ERR_INVALID_ARG);
}

// Each run's sum of gate steps, a CTA per (run, 64 channels).
template <typename T, int RL>
__global__ void __launch_bounds__(kWarps * 32) run_sums_kernel(AppendArgs a) {
  constexpr int TPW = RL / W;
  __shared__ __align__(16) long long s_sum[W][kSlab];
  start_next();
  const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const Run<RL> r = run_at<RL>(a.bt, blockIdx.x);
  if (r.i < 0 || r.none) return;
  const int C = a.HQ * a.K;
  const int c = blockIdx.y * kSlab + lane * 4;
  const int o0 = r.base + grp * TPW;
  const int xa = max(0, r.ctx - o0), xb = min(TPW, r.kv - o0);
  Quad<T> gq[TPW];
  load_tokens(static_cast<const T*>(a.g) + ((long)r.t0 + o0 - r.ctx) * C + c, C, xa, xb, c < C, gq);
  int step[TPW][4];
  bool nan = false;
  gate_steps(gq, step, &s_sum[grp][lane * 4], nan);
  __syncthreads();
  const int x = threadIdx.x;
  if (x < kSlab && blockIdx.y * kSlab + x < C) {
    long long t = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) t += s_sum[w][x];
    a.runs[(long)blockIdx.x * C + blockIdx.y * kSlab + x] = t;
  }
}

// The runs' sums of one request and 32 channels become the prefixes before
// them, from the request's carry: eight warps, a share of the runs each.
template <int RL>
__global__ void __launch_bounds__(256) run_scan_kernel(AppendArgs a) {
  __shared__ long long s_part[8][32];
  start_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x, C = a.HQ * a.K, c = blockIdx.y * 32 + lane;
  const int t0 = a.bt.start(i), n = a.bt.rows(i), kv = a.bt.keys(i), ctx = kv - n;
  wait_before();
  if (n == 0 || ctx < 0) return;
  const int count = (kv - 1) / RL - ctx / RL + 1;
  const int each = (count + 7) / 8, r0 = warp * each, r1 = min(count, r0 + each);
  long long* s = a.runs + ((long)t0 / RL + 2 * i) * C + c;
  long long part = 0;
  if (c < C) {
#pragma unroll 8
    for (int r = r0; r < r1; ++r) part += s[(long)r * C];
  }
  s_part[warp][lane] = part;
  __syncthreads();
  if (c >= C) return;
  long long P = ctx > 0 ? a.carry_in[(long)i * C + c] : 0;
  for (int w = 0; w < warp; ++w) P += s_part[w][lane];
#pragma unroll 8
  for (int r = r0; r < r1; ++r) {
    const long long x = s[(long)r * C];
    s[(long)r * C] = P;
    P += x;
  }
}

// One token a request: a warp per (request, 128 channels), then per (request,
// 32 vectors of values).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) append_one_kernel(AppendArgs a, int v_slabs) {
  const int lane = threadIdx.x & 31;
  const long w = (long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int per = a.k_slabs + v_slabs;
  const int i = (int)(w / per), slab = (int)(w - (long)i * per);
  if (i >= a.bt.N) return;
  const int t = a.bt.start(i), n = a.bt.rows(i), kv = a.bt.keys(i);
  const bool none = n == 0 || kv < n;
  if (n > 1 && slab == 0 && lane == 0) record_status(a.status, WALL_ERR_INVALID_ARG);
  const int PS1 = (1 << a.shift) - 1;
  const long long slot = none ? 0 : a.slots[t];
  const long long pg = slot >> a.shift;
  const bool bad = !none && (slot < 0 || pg >= a.NP);
  const int page = (int)pg;
  if (slab >= a.k_slabs) {
    constexpr int EV = 16 / sizeof(T);
    const int ch = ((slab - a.k_slabs) * 32 + lane) * EV;
    if (none || bad || ch >= a.H * a.V) return;
    const int h = ch / a.V, x = ch - h * a.V;
    *reinterpret_cast<uint4*>(static_cast<T*>(a.vp) +
                              ((((long)page * a.H + h) << a.shift) + (int)(slot & PS1)) * a.V + x) =
        *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + (long)t * a.H * a.V + ch);
    return;
  }
  const int C = a.HQ * a.K, c = slab * kOneSlab + lane * 4;
  if (c >= C) return;
  const int h = c / a.K, ch = c - h * a.K;
  longlong2 u = make_longlong2(0, 0), v = u;
  if (none || kv > n) {
    const longlong2* src = reinterpret_cast<const longlong2*>(a.carry_in + (long)i * C + c);
    u = src[0];
    v = src[1];
  }
  longlong2* dst = reinterpret_cast<longlong2*>(a.carry_out + (long)i * C + c);
  if (none) {
    if (a.carry_out != a.carry_in) {
      dst[0] = u;
      dst[1] = v;
    }
    return;
  }
  Quad<T> gq, kq;
  gq.load(static_cast<const T*>(a.g) + (long)t * C + c);
  kq.load(static_cast<const T*>(a.k) + ((long)t * a.H + h / (a.HQ / a.H)) * a.K + ch);
  float f[4], kf[4], pv[4];
  gq.get(f);
  kq.get(kf);
  const int step[4] = {gate_fixed(f[0]), gate_fixed(f[1]), gate_fixed(f[2]), gate_fixed(f[3])};
  const long long before[4] = {u.x, u.y, v.x, v.y};
  const long long P[4] = {u.x + step[0], u.y + step[1], v.x + step[2], v.y + step[3]};
  const bool begins = ((kv - n) & PS1) == 0;  // the token begins its page
  int4 r4 = make_int4(0, 0, 0, 0);
  int4* rp = reinterpret_cast<int4*>(a.rp + (long)page * C + c);
  if (begins) {
    r4 = make_int4(page_anchor(P[0]), page_anchor(P[1]), page_anchor(P[2]), page_anchor(P[3]));
    if (!bad) *rp = r4;
  } else if (!bad) {
    r4 = *rp;
  }
  const int R[4] = {r4.x, r4.y, r4.z, r4.w};
  bool wide = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    int lost = 0;
    pv[e] = token_prefix(add_step(from_anchor(before[e], R[e]), step[e], lost), wide);
    wide |= !begins && lost < 0;
    if (f[e] != f[e]) pv[e] = f[e];
    kf[e] *= exp2f(-pv[e]);
  }
  *reinterpret_cast<float4*>(a.p + (long)t * C + c) = make_float4(pv[0], pv[1], pv[2], pv[3]);
  if (!bad)
    Quad<T>::store(static_cast<T*>(a.kp) + ((((long)page * a.HQ + h) << a.shift) + (int)(slot & PS1)) * a.K + ch,
                   kf);
  dst[0] = make_longlong2(P[0], P[1]);
  dst[1] = make_longlong2(P[2], P[3]);
  if (wide) record_status(a.status, WALL_ERR_RANGE);
  if (bad) record_status(a.status, WALL_ERR_INVALID_ARG);
}

// Blocks that a request's tokens may touch up to which one CTA walks them: a
// block costs the walk about 1.5 us, the three launches of the runs' way 7 us
// in all.
constexpr int kWalkBlocks = 4;
int block_len(int shift) { return shift == 7 ? 128 : 64; }
int blocks_of(int max_new, int shift) { return (max_new + block_len(shift) - 2) / block_len(shift) + 1; }
long run_places(int N, int T, int shift) { return (long)T / block_len(shift) + 2l * N; }

template <typename T, int RL>
int append_tokens(AppendArgs& a, int max_new, int v_slabs, cudaStream_t stream) {
  const int slabs = a.k_slabs + v_slabs;
  if (blocks_of(max_new, a.shift) <= kWalkBlocks) {
    append_kernel<T, RL, false><<<dim3(a.bt.N, slabs), kWarps * 32, 0, stream>>>(a);
  } else {
    const int places = (int)run_places(a.bt.N, a.bt.T, a.shift);
    run_sums_kernel<T, RL><<<dim3(places, a.k_slabs), kWarps * 32, 0, stream>>>(a);
    if (launch_behind(run_scan_kernel<RL>, dim3(a.bt.N, ceil_div((long)a.HQ * a.K, 32)), 256, 0, stream, a) ||
        launch_behind(append_kernel<T, RL, true>, dim3(places, slabs), kWarps * 32, 0, stream, a))
      return WALL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

template <typename T>
int append(AppendArgs& a, int max_new, cudaStream_t stream) {
  const int v_slabs = ceil_div((long)a.H * a.V * sizeof(T), 32 * 16);
  if (max_new == 1) {
    a.k_slabs = ceil_div((long)a.HQ * a.K, kOneSlab);
    const long warps = (long)a.bt.N * (a.k_slabs + v_slabs);
    append_one_kernel<T><<<ceil_div(warps, kWarps), kWarps * 32, 0, stream>>>(a, v_slabs);
    return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
  }
  return a.shift == 7 ? append_tokens<T, 128>(a, max_new, v_slabs, stream)
                      : append_tokens<T, 64>(a, max_new, v_slabs, stream);
}

}  // namespace

size_t paged_append_ws(int N, int T, int HQ, int K, int shift, int max_new) {
  if (max_new == 1 || blocks_of(max_new, shift) <= kWalkBlocks) return 0;
  return sizeof(long long) * (size_t)run_places(N, T, shift) * HQ * K;
}

int paged_append(const PagedAppendProblem& pb, void* ws, cudaStream_t stream) {
  AppendArgs a;
  a.k = pb.k; a.v = pb.v; a.g = pb.g;
  a.bt.cu = pb.cu; a.bt.kv = pb.kv; a.bt.N = pb.N; a.bt.T = pb.T;
  a.bt.cap = 0x7fffffff - 2 * 128;  // positions a block or two further are still ints
  a.slots = reinterpret_cast<const long long*>(pb.slots);
  a.H = pb.H; a.HQ = pb.HQ; a.K = pb.K; a.V = pb.V; a.shift = pb.shift; a.NP = pb.NP;
  a.kp = pb.k_pages; a.vp = pb.v_pages; a.rp = pb.r_pages;
  a.carry_in = reinterpret_cast<const long long*>(pb.carry_in);
  a.carry_out = reinterpret_cast<long long*>(pb.carry_out);
  a.p = pb.p;
  a.status = device_status();
  a.k_slabs = ceil_div((long)pb.HQ * pb.K, kSlab);
  a.runs = static_cast<long long*>(ws);
  return pb.dtype == WALL_BF16 ? append<__nv_bfloat16>(a, pb.max_new, stream)
                               : append<float>(a, pb.max_new, stream);
}

}  // namespace wall
