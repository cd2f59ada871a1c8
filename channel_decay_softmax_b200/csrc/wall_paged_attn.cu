// wall_paged_attn.cu -- attention of new tokens over the paged Wall cache: the
// general kernel (any dtype and head size), the join of units that two or more
// CTAs share, and the choice of kernels.
//
//   s_ij = scale sum_n q_in 2^(p_in + R_{page(i),n} - R_{page(j),n}) k_jn
//   o_i  = sum_j softmax(s_i, sink)_j v_j,   j <= i, i - j < window
// where k_jn is the cached row (k 2^(R - P)), p the token's prefix beyond its
// page's anchor and R the pages' whole-number anchors: the query meets each
// page once, scaled, and the inner loop has no gate arithmetic.
#include <algorithm>

#include "wall_paged_attn.h"

namespace wall {
namespace {

using namespace paged;

// ---------------------------------------------------------------------------
// general kernel: 32 query rows of one head against tiles of 32 keys, fp32
// throughout.  Four warps of eight rows; lane = key for the scores (a key's
// channels from shared memory, the rows' by broadcast: one load of keys feeds
// eight rows), then lane = VPL value channels for P V (two up to V = 64, so
// that no lane idles), P by broadcast from shared memory four keys at a time.
// A row's reference is raised only when a score passes it by 2^8, and its sum
// is kept by lanes until the end.  Measured: six fp32 requests of up to 70 rows
// over up to 970 keys (K = V = 64) 30 us, from 68: a tile's chain of page, load,
// scores and P V is what is left, three CTAs a SM to cover it (lines of the next
// tile sent ahead to the L2 gain nothing).  Three CTAs leave a thread 168
// registers, over which the forms of this kernel and of flagged_kernel spill up
// to 96 bytes.

constexpr int GR = kGeneralRows;
constexpr int kGenWarps = 4, kGenThreads = kGenWarps * 32;
constexpr int kRowsPerWarp = GR / kGenWarps;

size_t gen_smem(int K, int V) {
  return sizeof(float) * (size_t)(GR * K + GR * (K + 4) + GR * V + GR * GR);
}


// Tiles [ta, tb) of the row block: softmax state of this warp's rows.
template <typename T, int VPL>
__device__ __forceinline__ void gen_tiles(const AttnArgs& a, const Request& r, int h, int row0,
                                          int lo_tile, int ta, int tb, float* smem,
                                          float (&m)[kRowsPerWarp], float (&l)[kRowsPerWarp],
                                          float (&acc)[kRowsPerWarp][VPL]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = a.K, V = a.V;
  float* sQ = smem;              // [GR][K]
  float* sK = sQ + GR * K;       // [GR][K + 4]
  float* sV = sK + GR * (K + 4); // [GR][V]
  float* sP = sV + GR * V + (tid >> 5) * (kRowsPerWarp * GR);  // this warp's [rows][keys]
  const T* q = static_cast<const T*>(a.q);
  const T* kp = static_cast<const T*>(a.kp);
  const T* vp = static_cast<const T*>(a.vp);
  const int kh = h / (a.HQ / a.H);
  const long trow = (long)r.i * a.MP;
  const int ni = min(GR, r.n - row0);
  const int win = a.window > 0 ? a.window : 0x7fffffff;
  const int w0 = warp * kRowsPerWarp;
#pragma unroll
  for (int x = 0; x < kRowsPerWarp; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
#pragma unroll
    for (int e = 0; e < VPL; ++e) acc[x][e] = 0.f;
  }
  if (r.dead) return;
  // the rows' own pages: two at most, since a page has 32 positions or more
  const int pos0 = r.ctx + row0;
  const int own0 = pos0 >> a.shift, own1 = (pos0 + ni - 1) >> a.shift;
  const int page0 = own0 < a.MP ? page_of(a.table, trow, own0, a.NP) : -1;
  const int page1 = own1 < a.MP ? page_of(a.table, trow, own1, a.NP) : -1;
  int at = -1;  // table slot whose scaled queries are in sQ
  for (int t = ta; t < tb; ++t) {
    const int j0 = (lo_tile + t) * GR;
    const int slot = j0 >> a.shift;
    const int page = slot < a.MP ? page_of(a.table, trow, slot, a.NP) : -1;
    if (page < 0) {  // the same for the whole CTA: an entry outside the pool
      if (tid == 0) record_status(a.status, WALL_ERR_INVALID_ARG);
      continue;
    }
    __syncthreads();  // the last tile's readers are done
    const int off = j0 & ((1 << a.shift) - 1);
    const T* kt = kp + ((((long)page * a.HQ + h) << a.shift) + off) * K;
    const T* vt = vp + ((((long)page * a.H + kh) << a.shift) + off) * V;
    const int nk = r.kv - j0;  // keys of the tile; what lies behind them is not read
#pragma unroll 4
    for (int idx = tid; idx < GR * (K / 8); idx += kGenThreads) {
      const int j = idx / (K / 8), c = (idx - j * (K / 8)) * 8;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (j < nk) load8(kt + j * K + c, x);
      *reinterpret_cast<float4*>(sK + j * (K + 4) + c) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(sK + j * (K + 4) + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
#pragma unroll 4
    for (int idx = tid; idx < GR * (V / 8); idx += kGenThreads) {
      const int j = idx / (V / 8), c = (idx - j * (V / 8)) * 8;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (j < nk) load8(vt + j * V + c, x);
      *reinterpret_cast<float4*>(sV + j * V + c) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(sV + j * V + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (slot != at) {
      // the rows against this page: scale * log2(e) * q * 2^(p + R - R_c); rows
      // of an earlier page see nothing of it
      const int* Rc = a.rp + ((long)page * a.HQ + h) * K;
      const int* R0 = a.rp + ((long)max(page0, 0) * a.HQ + h) * K;
      const int* R1 = a.rp + ((long)max(page1, 0) * a.HQ + h) * K;
      const long e0 = ((long)(r.t0 + row0) * a.HQ + h) * K;
#pragma unroll 2
      for (int idx = tid; idx < ni * (K / 8); idx += kGenThreads) {
        const int row = idx / (K / 8), c = (idx - row * (K / 8)) * 8;
        const int rs = (pos0 + row) >> a.shift;
        const int* Rr = rs == own0 ? R0 : R1;
        float qv[8], pv[8];
        load8(q + e0 + (long)row * a.HQ * K + c, qv);
        load8(a.p + e0 + (long)row * a.HQ * K + c, pv);
        const int4 u0 = *reinterpret_cast<const int4*>(Rr + c), u1 = *reinterpret_cast<const int4*>(Rr + c + 4);
        const int4 w0 = *reinterpret_cast<const int4*>(Rc + c), w1 = *reinterpret_cast<const int4*>(Rc + c + 4);
        const int d[8] = {u0.x - w0.x, u0.y - w0.y, u0.z - w0.z, u0.w - w0.w,
                          u1.x - w1.x, u1.y - w1.y, u1.z - w1.z, u1.w - w1.w};
        const bool sees = rs >= slot;
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          pv[e] += (float)d[e];
          most = fmaxf(most, pv[e]);
          qv[e] *= a.scale_log2;
        }
        if (most <= kPageRange) {
#pragma unroll
          for (int e = 0; e < 8; ++e) qv[e] = sees ? qv[e] * exp2f(pv[e]) : 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) qv[e] = sees ? grown_query(qv[e], pv[e]) : 0.f;
        }
        store8(sQ + row * K + c, qv);
      }
      at = slot;
    }
    __syncthreads();
    if (w0 >= ni) continue;  // warps past the block's rows only keep step
    float d[kRowsPerWarp];
#pragma unroll
    for (int x = 0; x < kRowsPerWarp; ++x) d[x] = 0.f;
    const float* krow = sK + lane * (K + 4);
#pragma unroll 4
    for (int c = 0; c < K; c += 4) {
      const float4 kx = *reinterpret_cast<const float4*>(krow + c);
#pragma unroll
      for (int x = 0; x < kRowsPerWarp; ++x) {
        const float4 qx = *reinterpret_cast<const float4*>(sQ + (w0 + x) * K + c);
        d[x] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, d[x]))));
      }
    }
    const int j = j0 + lane;
    unsigned seen[kRowsPerWarp], every = 0xffffffffu;
    __syncwarp();  // the last tile's P has been read
#pragma unroll
    for (int x = 0; x < kRowsPerWarp; ++x) {
      const int pos = r.ctx + row0 + w0 + x;
      const bool vis = w0 + x < ni && j <= pos && j < r.kv && pos - j < win;
      seen[x] = __ballot_sync(0xffffffffu, vis);
      if (w0 + x < ni) every &= seen[x];
      // (m = -inf: the row's first key)
      if (__any_sync(0xffffffffu, vis && d[x] > m[x] + 8.f)) {
        float mx = vis ? d[x] : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, m[x]);
        const float alpha = exp2f(m[x] - mx);
        l[x] *= alpha;
        m[x] = mx;
#pragma unroll
        for (int e = 0; e < VPL; ++e) acc[x][e] *= alpha;
      }
      const float p = vis ? exp2f(d[x] - (m[x] == -INFINITY ? 0.f : m[x])) : 0.f;
      l[x] += p;
      sP[x * GR + lane] = p;
    }
    __syncwarp();
    const float* vcol = sV + (lane * VPL < V ? lane * VPL : 0);
#pragma unroll 1
    for (int jj = 0; jj < GR; jj += 4) {
      float v[4][VPL];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        if constexpr (VPL == 4) {
          const float4 u = *reinterpret_cast<const float4*>(vcol + (jj + z) * V);
          v[z][0] = u.x; v[z][1] = u.y; v[z][2] = u.z; v[z][3] = u.w;
        } else {
          const float2 u = *reinterpret_cast<const float2*>(vcol + (jj + z) * V);
          v[z][0] = u.x; v[z][1] = u.y;
        }
      }
#pragma unroll
      for (int x = 0; x < kRowsPerWarp; ++x) {
        const float4 p4 = *reinterpret_cast<const float4*>(sP + x * GR + jj);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
        // a masked key's value row may hold anything (NaN included): it is
        // skipped, not multiplied by zero
        const unsigned bits = every == 0xffffffffu ? 15u : seen[x] >> jj;
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if ((bits >> z) & 1u) {
#pragma unroll
            for (int e = 0; e < VPL; ++e) acc[x][e] = fmaf(p[z], v[z][e], acc[x][e]);
          }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kRowsPerWarp; ++x)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], o);
}

// The finished rows of a block: o = acc / l and lse, the sink's weight in l.
template <typename T, int VPL>
__device__ __forceinline__ void write_row(const AttnArgs& a, long token, int h, int lane, float m,
                                          float l, const float (&acc)[VPL]) {
  float mf = m, lt = l, f = 1.f;
  if (a.sink) {
    const float sk = a.sink[h] * kLog2e;
    mf = fmaxf(m, sk);
    f = m == -INFINITY ? 0.f : exp2f(m - mf);
    lt = l * f + sink_weight(sk, mf);
  }
  const float inv = lt > 0.f || lt != lt ? f / lt : 0.f;  // a row that sees nothing: 0
  if (lane * VPL < a.V) {
    T* o = static_cast<T*>(a.o) + ((long)token * a.HQ + h) * a.V + lane * VPL;
    struct alignas(sizeof(T) * VPL) Out { T x[VPL]; } out;  // one store a lane
#pragma unroll
    for (int e = 0; e < VPL; ++e) out.x[e] = from_f32<T>(acc[e] * inv);
    *reinterpret_cast<Out*>(o) = out;
  }
  if (lane == 0 && a.lse) a.lse[token * a.HQ + h] = lt == 0.f ? -INFINITY : (mf + log2f(lt)) * kLn2;
}

template <typename T, int VPL>
__global__ void __launch_bounds__(kGenThreads, 3) general_kernel(AttnArgs a, Pick pk, Parts parts) {
  extern __shared__ __align__(16) float gen_shared[];
  __shared__ FindScratch fs;
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  start_next();
  wait_before();
  if (threadIdx.x == 0) parts.desc[cta].last_cta = -1;
  Share sh;
  if (!find_start<GR, 0>(a.bt, a.window, a.HQ, pk, 1, cta, parts.n_cta, fs, sh)) return;
  const long long x0 = sh.begin(cta), x1 = sh.begin(cta + 1);
  Cursor c = cursor_at<GR, 0>(a.bt, a.window, fs.req, fs.base, x0);
  for (long long x = x0; x < x1;) {
    const Run run = run_of<0>(c, x1 - x);
    const int ta = run.ta, tb = run.tb;
    float m[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][VPL];
    gen_tiles<T, VPL>(a, c.r, c.h, c.b * GR, tile_lo(c.r, c.b), ta, tb, gen_shared, m, l, acc);
    const int ni = min(GR, c.r.n - c.b * GR);
    const bool whole = ta == 0 && tb == c.n_tiles;
    const int slot = ta == 0 ? 1 : 0;
    float* po = parts.o(cta, slot, a.V);
    float* pm = parts.ml(cta, slot, a.V);
#pragma unroll
    for (int y = 0; y < kRowsPerWarp; ++y) {
      const int row = warp * kRowsPerWarp + y;
      if (row >= ni) continue;
      if (whole) {
        write_row<T, VPL>(a, c.r.t0 + c.b * GR + row, c.h, lane, m[y], l[y], acc[y]);
      } else {
        if (lane * VPL < a.V) {
#pragma unroll
          for (int e = 0; e < VPL; e += 2)
            *reinterpret_cast<float2*>(po + (size_t)row * a.V + lane * VPL + e) =
                make_float2(acc[y][e], acc[y][e + 1]);
        }
        if (lane == 0) {
          pm[row * 2] = m[y];
          pm[row * 2 + 1] = l[y];
        }
      }
    }
    if (!whole && slot == 1 && threadIdx.x == 0) {
      PartDesc d;
      d.t0 = c.r.t0 + c.b * GR; d.rows = min(GR, c.r.n - c.b * GR); d.h = c.h;
      d.last_cta = sh.last_owner<0>(c, x);
      parts.desc[cta] = d;
    }
    x += run.places;
    if (x < x1) next_unit<GR>(a.bt, a.window, a.HQ, pk, c);
  }
}

// The units that the tensor-core kernel flagged, again and whole: a grid over
// (request's 128-row block, head, 32 rows of it), whose CTAs read one word and
// leave when nothing is flagged.
template <typename T, int VPL>
__global__ void __launch_bounds__(kGenThreads, 3) flagged_kernel(AttnArgs a, UnitFlags flags) {
  extern __shared__ __align__(16) float gen_shared[];
  wait_before();
  if (*flags.any(a.HQ) == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int at = 0;  // (block, head, quarter) items before the request
  for (int i = 0; i < a.bt.N; ++i) {
    const int n = a.bt.rows(i);
    if (n < 2) continue;
    const Request r = request_of<GR>(a.bt, i, a.window);
    const int items = r.nb * a.HQ;  // 32-row blocks of every head
    const int first = ((int)blockIdx.x - at % (int)gridDim.x + (int)gridDim.x) % (int)gridDim.x;
    for (int x = first; x < items; x += gridDim.x) {
      const int b = x / a.HQ, h = x - b * a.HQ;
      if (!flags.has(flags.place(r, b * GR / kChunkRows), h, a.HQ, UnitFlags::kAgain)) continue;
      float m[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][VPL];
      gen_tiles<T, VPL>(a, r, h, b * GR, tile_lo(r, b), 0, unit_tiles(r, b), gen_shared, m, l, acc);
#pragma unroll
      for (int y = 0; y < kRowsPerWarp; ++y) {
        const int row = b * GR + warp * kRowsPerWarp + y;
        if (row < n) write_row<T, VPL>(a, r.t0 + row, h, lane, m[y], l[y], acc[y]);
      }
    }
    at = (at + items) % (int)gridDim.x;
  }
}

// ---------------------------------------------------------------------------
// Joining the units that more than one CTA worked on: o = sum of the parts
// weighted by 2^(m_part - m), over the sum of their l, in the order of the
// CTAs (the same bits every time).  One warp a row; 4 channels a lane.
// One launch joins all of a call's parts, of the kernels that it may run: 4 us
// for decode, 10 where all CTAs cut a 128-row unit (20 MB of parts).
constexpr int kJoinThreads = 256, kJoinY = 4;
struct JoinSet {
  Parts parts;
  int group;  // > 0: a part's rows are tokens of `group` heads of one kv head
};
struct JoinSets {
  JoinSet s[2];
  int n;
};
template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 4) join_kernel(AttnArgs a, JoinSets sets) {
  start_next();
  wait_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool second = (int)blockIdx.x >= sets.s[0].parts.n_cta;
  const Parts parts = second ? sets.s[1].parts : sets.s[0].parts;
  const int group = second ? sets.s[1].group : sets.s[0].group;
  const int cta = blockIdx.x - (second ? sets.s[0].parts.n_cta : 0);
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.bt.N; i += kJoinThreads)
      if (a.bt.rows(i) > a.max_new || (a.bt.rows(i) > 0 && a.bt.kv[i] > a.bt.cap))
        record_status(a.status, WALL_ERR_INVALID_ARG);
  const PartDesc d = parts.desc[cta];
  if (d.last_cta < 0) return;
  const int np = d.last_cta - cta + 1;
  const int stride = gridDim.y * (kJoinThreads / 32);
  const size_t step = parts.stride(a.V) * 2;  // from a CTA's part to the next CTA's
#pragma unroll 1
  for (int row = blockIdx.y * (kJoinThreads / 32) + warp; row < d.rows; row += stride) {
    // part s > 0 is at s * step from CTA `cta`'s slot 0; part 0 is its slot 1
    const float2* ml = reinterpret_cast<const float2*>(parts.ml(cta, 0, a.V)) + row;
    const float* o = parts.o(cta, 0, a.V) + row * a.V + (lane * 4 < a.V ? lane * 4 : 0);
    float m = -INFINITY;
#pragma unroll 1
    for (int s = lane; s < np; s += 32) m = fmaxf(m, ml[(s == 0 ? step : s * step * 2) / 4].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s0 = 0; s0 < np; s0 += 32) {
      float f = 0.f;
      const int s = s0 + lane;
      if (s < np) {
        const float2 y = ml[(s == 0 ? step : s * step * 2) / 4];
        if (y.x != -INFINITY) {
          f = exp2f(y.x - m);
          l = fmaf(y.y, f, l);
        }
      }
      const int cnt = min(32, np - s0);
      const float* os = o + s0 * step;
      auto add = [&](float4 x, int j) {
        const float fj = __shfl_sync(0xffffffffu, f, j);
        if (fj != 0.f) {
          acc[0] = fmaf(x.x, fj, acc[0]);
          acc[1] = fmaf(x.y, fj, acc[1]);
          acc[2] = fmaf(x.z, fj, acc[2]);
          acc[3] = fmaf(x.w, fj, acc[3]);
        }
      };
      auto part = [&](int j) {
        return *reinterpret_cast<const float4*>(os + (s0 + j == 0 ? step / 2 : j * step));
      };
      int j = 0;
#pragma unroll 1
      for (; j + 4 <= cnt; j += 4) {
        float4 x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = part(j + y);
#pragma unroll
        for (int y = 0; y < 4; ++y) add(x[y], j + y);
      }
#pragma unroll 1
      for (; j < cnt; j += 2) {  // most units have two parts
        const float4 x0 = part(j), x1 = part(min(j + 1, cnt - 1));
        add(x0, j);
        if (j + 1 < cnt) add(x1, j + 1);
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (group > 0) write_row<T, 4>(a, d.t0 + row / group, d.h * group + row % group, lane, m, l, acc);
    else write_row<T, 4>(a, d.t0 + row, d.h, lane, m, l, acc);
  }
}

template <typename T>
int join(const AttnArgs& a, const JoinSets& sets, cudaStream_t stream) {
  int ctas = 0, rows = 0;
  for (int i = 0; i < sets.n; ++i) {
    const JoinSet& s = sets.s[i];
    ctas += s.parts.n_cta;
    rows = std::max(rows, s.parts.rows);
  }
  return launch_behind(join_kernel<T>, dim3(ctas, std::min(kJoinY, ceil_div(rows, kJoinThreads / 32))),
                       kJoinThreads, 0, stream, a, sets);
}

template <typename T, int VPL>
int launch_general(const AttnArgs& a, const Pick& pk, const Parts& parts, bool first, cudaStream_t stream) {
  static bool attr[kMaxDevices] = {};
  if (!set_max_smem_once(general_kernel<T, VPL>, (int)gen_smem(128, 128), attr)) return WALL_ERR_CUDA;
  if (first) {
    general_kernel<T, VPL><<<parts.n_cta, kGenThreads, gen_smem(a.K, a.V), stream>>>(a, pk, parts);
    return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
  }
  return launch_behind(general_kernel<T, VPL>, parts.n_cta, kGenThreads, gen_smem(a.K, a.V), stream, a,
                       pk, parts);
}
template <typename T>
int run_general(const AttnArgs& a, const Pick& pk, const Parts& parts, bool first, cudaStream_t stream) {
  return a.V <= 64 ? launch_general<T, 2>(a, pk, parts, first, stream)
                   : launch_general<T, 4>(a, pk, parts, first, stream);
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

template <int VPL>
int launch_flagged(const AttnArgs& a, const UnitFlags& flags, cudaStream_t stream) {
  using T = __nv_bfloat16;
  static bool attr[kMaxDevices] = {};
  if (!set_max_smem_once(flagged_kernel<T, VPL>, (int)gen_smem(128, 128), attr)) return WALL_ERR_CUDA;
  return launch_behind(flagged_kernel<T, VPL>, kGeneralCtas, kGenThreads, gen_smem(a.K, a.V), stream, a,
                       flags);
}
int run_flagged(const AttnArgs& a, const UnitFlags& flags, cudaStream_t stream) {
  return a.V <= 64 ? launch_flagged<2>(a, flags, stream) : launch_flagged<4>(a, flags, stream);
}

// Which kernels a call runs: single-token rows stream through the decode
// kernel and rows of requests of more through the tensor cores where these
// kernels cover the shape; the general kernel takes what is left.  A call whose
// requests all have at most kShortRows rows (drafts) needs the decode kernel
// alone, in a form for that many: 16 requests of 2 to 8 rows take 78 us so, 111
// as units of 128 rows.  Beside longer requests the few rows stay with those: a
// further launch costs each such call 5 us, and single tokens through the form
// for many rows 57 us where their own takes 39.
struct Route {
  bool decode;    // the decode kernel, for requests of fewer than n_min rows
  bool chunk;     // the tensor-core kernel, for requests of n_min or more
  int n_min;
  bool general;   // the general kernel
  Pick rows;      // the requests it takes
};
Route route_of(int dtype, int max_new, int H, int HQ, int K, int V) {
  Route r;
  r.decode = decode_rows_supported(dtype, H, HQ, K, V);
  r.n_min = r.decode && few_rows(max_new) ? kShortRows + 1 : 2;
  r.chunk = max_new >= r.n_min && chunk_rows_supported(dtype, K, V);
  r.rows.n_min = r.decode ? r.n_min : 1;
  r.rows.n_max = r.chunk ? 1 : 0x7fffffff;
  r.general = !r.decode || (max_new >= r.n_min && !r.chunk);
  return r;
}

struct AttnWs {
  size_t dec_desc, dec_data, chunk_desc, chunk_data, qh, flags, gen_desc, gen_data, total;
};
int decode_part_rows(int max_new, int G) { return few_rows(max_new) ? max_new * G : G; }
AttnWs attn_ws(const Route& r, int N, int T, int max_new, int H, int HQ, int K, int V) {
  AttnWs w;
  size_t off = 0;
  auto take = [&](bool need, int ctas, int rows, size_t& desc, size_t& data) {
    desc = off;
    off += need ? al256(sizeof(PartDesc) * ctas) : 0;
    data = off;
    off += need ? al256(sizeof(float) * 2 * ctas * Parts::stride_of(rows, V)) : 0;
  };
  take(r.decode, kSms, decode_part_rows(max_new, HQ / H), w.dec_desc, w.dec_data);
  take(r.chunk, kSms, kChunkRows, w.chunk_desc, w.chunk_data);
  w.qh = off;
  off += r.chunk ? al256((size_t)2 * T * HQ * K) : 0;
  w.flags = off;
  off += r.chunk ? al256(sizeof(int) * (size_t)UnitFlags::count(N, T, HQ)) : 0;
  take(r.general, kGeneralCtas, GR, w.gen_desc, w.gen_data);
  w.total = off;
  return w;
}

Parts parts_at(void* ws, size_t desc, size_t data, int rows, int ctas) {
  Parts p;
  p.desc = reinterpret_cast<PartDesc*>(static_cast<char*>(ws) + desc);
  p.data = reinterpret_cast<float*>(static_cast<char*>(ws) + data);
  p.rows = rows;
  p.n_cta = ctas;
  return p;
}

}  // namespace

size_t paged_attn_ws(int dtype, int N, int T, int max_new, int H, int HQ, int K, int V) {
  return attn_ws(route_of(dtype, max_new, H, HQ, K, V), N, T, max_new, H, HQ, K, V).total;
}

int paged_attn(const PagedAttnProblem& pb, void* ws, cudaStream_t stream) {
  AttnArgs a;
  a.q = pb.q; a.p = pb.p;
  a.bt.cu = pb.cu; a.bt.kv = pb.kv; a.bt.N = pb.N; a.bt.T = pb.T;
  a.bt.cap = pb.MP << pb.shift;
  a.table = pb.table; a.MP = pb.MP; a.NP = pb.NP; a.shift = pb.shift;
  a.H = pb.H; a.HQ = pb.HQ; a.K = pb.K; a.V = pb.V;
  a.kp = pb.k_pages; a.vp = pb.v_pages; a.rp = pb.r_pages;
  a.sink = pb.sink;
  a.scale_log2 = pb.scale * kLog2e;
  a.window = pb.window;
  a.max_new = pb.max_new;
  a.o = pb.o; a.lse = pb.lse;
  a.status = device_status();
  const Route r = route_of(pb.dtype, pb.max_new, pb.H, pb.HQ, pb.K, pb.V);
  a.n_min = r.n_min;
  const AttnWs w = attn_ws(r, pb.N, pb.T, pb.max_new, pb.H, pb.HQ, pb.K, pb.V);
  UnitFlags flags = {};
  if (r.chunk) {
    flags.f = reinterpret_cast<int*>(static_cast<char*>(ws) + w.flags);
    flags.places_n = (int)UnitFlags::places(pb.N, pb.T);
    flags.total = UnitFlags::count(pb.N, pb.T, pb.HQ);
  }
  JoinSets sets = {};
  if (r.decode) {
    const int G = pb.HQ / pb.H;
    const Parts p = parts_at(ws, w.dec_desc, w.dec_data, decode_part_rows(pb.max_new, G), kSms);
    const int rc = decode_rows(a, p, flags, stream);  // clears the flags
    if (rc) return rc;
    sets.s[sets.n++] = {p, G};
  } else if (r.chunk && cudaMemsetAsync(flags.f, 0, sizeof(int) * flags.total, stream) != cudaSuccess) {
    return WALL_ERR_CUDA;
  }
  if (r.chunk) {
    const Parts p = parts_at(ws, w.chunk_desc, w.chunk_data, kChunkRows, kSms);
    const int rc = chunk_rows(a, p, flags, static_cast<char*>(ws) + w.qh, stream);
    if (rc) return rc;
    sets.s[sets.n++] = {p, 0};
  }
  if (r.general) {
    const Parts p = parts_at(ws, w.gen_desc, w.gen_data, GR, kGeneralCtas);
    const int rc = pb.dtype == WALL_BF16 ? run_general<__nv_bfloat16>(a, r.rows, p, sets.n == 0, stream)
                                         : run_general<float>(a, r.rows, p, sets.n == 0, stream);
    if (rc) return rc;
    sets.s[sets.n++] = {p, 0};
  }
  const int rc = pb.dtype == WALL_BF16 ? join<__nv_bfloat16>(a, sets, stream)
                                       : join<float>(a, sets, stream);
  if (rc) return rc;
  return r.chunk ? run_flagged(a, flags, stream) : WALL_OK;
}

}  // namespace wall
