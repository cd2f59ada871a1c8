// wall_paged_append.cu -- new tokens into the paged Wall cache: the gate
// prefix, the pages' anchors, the rescaled key rows and the value rows.
//
//   e_t = rint(g_t 2^24 / ln 2),  P_t = P_{t-1} + e_t   (fixed point)
//   R_c = floor(P + 1/2) at page c's first position
//   p_t = P_t - R_{page(t)},   k_pages row = k_t 2^(-p_t),   v_pages row = v_t
//
// Per (token, query head, channel) 2 bytes of g come in and 4 of p and 2 of
// the key row go out (bf16), with k and v shared by a group: memory-bound.
// A CTA takes one request and 128 channels and walks the request's tokens in
// blocks aligned to the pages, eight warps a block: every warp sums its own
// tokens' gates, the sums meet in shared memory, and each warp then forms its
// tokens from its own prefix, so a block costs two barriers and its loads are
// all in flight at once.
#include "wall_internal.h"
#include "wall_paged.cuh"

namespace wall {
namespace {

using namespace paged;

constexpr int kSlab = 128;  // channels of a CTA: four a lane
constexpr int kWarps = 8;

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
};

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

// p of a token and the factor 2^-p of its key row from its prefix and its
// page's anchor.  A prefix that left the page's range is reported (the row
// would leave the numbers that bf16 has); a NaN gate makes both NaN.
__device__ __forceinline__ void token_factor(long long P, int R, float g, float& p, float& f,
                                             bool& wide) {
  const long long d = P - ((long long)R << kFrac);
  const int lo = (int)d;
  p = __int2float_rn(lo) * kStep;
  wide |= d != (long long)lo || fabsf(p) > kPageRange;
  if (g != g) p = g;
  f = exp2f(-p);
}

// The page of a slot, or -1 (reported) where the slot lies outside the pool.
__device__ __forceinline__ int slot_page(long long slot, const AppendArgs& a, bool& bad) {
  const long long page = slot >> a.shift;
  if (slot < 0 || page >= a.NP) {
    bad = true;
    return -1;
  }
  return (int)page;
}

// Rows of one value slab (32 vectors of 16 bytes) of tokens [ta, tb).
template <typename T>
__device__ __forceinline__ void copy_values(const AppendArgs& a, int ta, int tb, int vslab) {
  constexpr int EV = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = (vslab * 32 + lane) * EV;
  if (ch >= a.H * a.V) return;
  const int h = ch / a.V, n = ch - h * a.V;
  const int mask = (1 << a.shift) - 1;
  const T* v = static_cast<const T*>(a.v);
  T* vp = static_cast<T*>(a.vp);
  for (int t = ta + warp; t < tb; t += kWarps) {
    bool bad = false;
    const long long slot = a.slots[t];
    const int page = slot_page(slot, a, bad);
    if (bad) continue;  // the key slabs report it
    *reinterpret_cast<uint4*>(vp + ((((long)page * a.H + h) << a.shift) + (int)(slot & mask)) * a.V + n) =
        *reinterpret_cast<const uint4*>(v + (long)t * a.H * a.V + ch);
  }
}

// TPW tokens a warp: blocks of 8 TPW positions, a page or several.
template <typename T, int TPW>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendArgs a) {
  constexpr int RL = TPW * kWarps;
  __shared__ long long s_sum[kWarps][kSlab];
  __shared__ int s_R[RL / 32][kSlab];  // anchors of the pages that begin in the block
  const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = a.bt.start(i), n = a.bt.rows(i), kv = a.bt.kv[i];
  const bool none = n == 0 || kv < n;  // nothing new, or refused by the plan
  if ((int)blockIdx.y >= a.k_slabs) {
    if (!none) copy_values<T>(a, t0, t0 + n, blockIdx.y - a.k_slabs);
    return;
  }
  const int C = a.HQ * a.K;
  const int c = blockIdx.y * kSlab + lane * 4;
  const bool live = c < C;  // the last slab may be short
  const int h = live ? c / a.K : 0, ch = live ? c - h * a.K : 0;
  const int hk = h / (a.HQ / a.H);
  const int PS1 = (1 << a.shift) - 1;
  const int ctx = kv - n;
  long long carry[4] = {0, 0, 0, 0};
  if (live && (none || ctx > 0)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) carry[e] = a.carry_in[(long)i * C + c + e];
  }
  if (none) {
    if (live && warp == 0 && a.carry_out != a.carry_in) {
#pragma unroll
      for (int e = 0; e < 4; ++e) a.carry_out[(long)i * C + c + e] = carry[e];
    }
    return;
  }
  const T* g = static_cast<const T*>(a.g);
  const T* k = static_cast<const T*>(a.k);
  T* kp = static_cast<T*>(a.kp);
  bool wide = false, bad = false;
  for (int base = ctx / RL * RL; base < kv; base += RL) {
    const int o0 = base + warp * TPW;  // this warp's first position
    Quad<T> gq[TPW], kq[TPW];
    long long slot[TPW];
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      const int pos = o0 + x;
      const bool in = pos >= ctx && pos < kv;
      const long t = t0 + pos - ctx;
      gq[x].zero();
      kq[x].zero();
      slot[x] = in ? a.slots[t] : -1;
      if (in && live) {
        gq[x].load(g + t * C + c);
        kq[x].load(k + (t * a.H + hk) * a.K + ch);
      }
    }
    long long sum[4] = {0, 0, 0, 0};
    int first[4];  // this warp's first token's gate, for the anchor
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      float f[4];
      gq[x].get(f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = gate_fixed(f[e]);
        if (x == 0) first[e] = d;
        sum[e] += d;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s_sum[warp][lane * 4 + e] = sum[e];
    __syncthreads();
    long long P[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) P[e] = carry[e];
    for (int w = 0; w < kWarps; ++w) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long s = s_sum[w][lane * 4 + e];
        if (w < warp) P[e] += s;
        carry[e] += s;
      }
    }
    // a page that begins here, at a token of this call
    if ((o0 & PS1) == 0 && o0 >= ctx && o0 < kv) {
      const int page = slot_page(slot[0], a, bad);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int R = page_anchor(P[e] + first[e]);
        s_R[(o0 - base) >> 5][lane * 4 + e] = R;
        if (page >= 0 && live) a.rp[(long)page * C + c + e] = R;
      }
    }
    __syncthreads();
    const int po = o0 & ~PS1;  // this warp's page: TPW divides a page
    int R[4] = {0, 0, 0, 0};
    if (po >= ctx) {
#pragma unroll
      for (int e = 0; e < 4; ++e) R[e] = po < kv ? s_R[(po - base) >> 5][lane * 4 + e] : 0;
    } else {
      // begun by an earlier call: its anchor stands in the pool
      const int xf = max(o0, ctx);
      if (xf < min(o0 + TPW, kv)) {
        const int page = slot_page(a.slots[t0 + xf - ctx], a, bad);
        if (page >= 0 && live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) R[e] = a.rp[(long)page * C + c + e];
        }
      }
    }
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      const int pos = o0 + x;
      if (pos < ctx || pos >= kv || !live) continue;
      const long t = t0 + pos - ctx;
      float f[4], kf[4], pv[4], fac;
      gq[x].get(f);
      kq[x].get(kf);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        P[e] += gate_fixed(f[e]);
        token_factor(P[e], R[e], f[e], pv[e], fac, wide);
        kf[e] *= fac;
      }
      *reinterpret_cast<float4*>(a.p + t * C + c) = make_float4(pv[0], pv[1], pv[2], pv[3]);
      const int page = slot_page(slot[x], a, bad);
      if (page >= 0)
        Quad<T>::store(kp + ((((long)page * a.HQ + h) << a.shift) + (int)(slot[x] & PS1)) * a.K + ch, kf);
    }
  }
  if (live && warp == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) a.carry_out[(long)i * C + c + e] = carry[e];
  }
  if (wide) record_status(a.status, WALL_ERR_RANGE);
  if (bad) record_status(a.status, WALL_ERR_INVALID_ARG);
}

template <typename T>
int append(const AppendArgs& a, cudaStream_t stream) {
  const int v_slabs = ceil_div((long)a.H * a.V * sizeof(T), 32 * 16);
  const dim3 grid(a.bt.N, a.k_slabs + v_slabs);
  if (a.shift == 7)
    append_kernel<T, 16><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    append_kernel<T, 8><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

}  // namespace

size_t paged_append_ws(int N, int T, int HQ, int K, int shift, int max_new) {
  (void)N; (void)T; (void)HQ; (void)K; (void)shift; (void)max_new;
  return 0;
}

int paged_append(const PagedAppendProblem& pb, void* ws, cudaStream_t stream) {
  (void)ws;
  AppendArgs a;
  a.k = pb.k; a.v = pb.v; a.g = pb.g;
  a.bt.cu = pb.cu; a.bt.kv = pb.kv; a.bt.N = pb.N; a.bt.T = pb.T;
  a.slots = reinterpret_cast<const long long*>(pb.slots);
  a.H = pb.H; a.HQ = pb.HQ; a.K = pb.K; a.V = pb.V; a.shift = pb.shift; a.NP = pb.NP;
  a.kp = pb.k_pages; a.vp = pb.v_pages; a.rp = pb.r_pages;
  a.carry_in = reinterpret_cast<const long long*>(pb.carry_in);
  a.carry_out = reinterpret_cast<long long*>(pb.carry_out);
  a.p = pb.p;
  a.status = device_status();
  a.k_slabs = ceil_div((long)pb.HQ * pb.K, kSlab);
  return pb.dtype == WALL_BF16 ? append<__nv_bfloat16>(a, stream) : append<float>(a, stream);
}

}  // namespace wall
