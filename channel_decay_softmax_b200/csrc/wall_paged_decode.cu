// wall_paged_decode.cu -- the single-token rows of a paged batch (bf16, K and
// V in {64, 128}, up to 8 query heads a kv head).
//
// Memory-bound: a row reads its request's key rows (per query head), value
// rows (shared by the G heads of a kv head) and anchors once.  One CTA per SM
// streams an even share of the batch's 32-key tiles of (request, kv head):
// the last warp's lane 0 keeps a ring of TMA stages full (per tile one box of
// 64 channels x 32 rows x G heads per 128 bytes of key row -- the pages are
// head-major, so each head's piece is contiguous -- the value boxes and the
// page's anchors), and the tile's G heads have WPH warps each that take
// alternate stages with a softmax state of their own (a stage is the same
// warp's in every round, the stages being a multiple of WPH: a wait on a
// barrier's parity tells a phase only from the one before, which its waiter
// has to have seen): lane = key for the
// scores, then lane = VD / 32 value channels for P V.  The share runs across
// requests and heads, so the ring never drains between them, and a batch of
// any lengths loads every SM alike.
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "wall_paged_attn.h"

namespace wall {
namespace {

using namespace sm100;
using namespace paged;

constexpr int kTile = 32;
constexpr int kUnit = 1;           // a unit's own cost, in tiles
constexpr int kBox = kTile * 128;  // 64 channels of 32 rows
constexpr int kMaxStages = 16;

struct DecodeLaunch {
  int G, stages, stage_bytes;
  int* clear;  // words to clear, for the kernels behind this one
  long clear_n;
};

template <int KD, int VD, int WPH>
__global__ void __launch_bounds__(288, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, AttnArgs a, Parts parts,
                        DecodeLaunch dl) {
  constexpr int VPL = VD / 32, QPL = KD / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ FindScratch fs;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int G = dl.G, stages = dl.stages;
  const int oV = G * (KD / 64) * kBox;               // within a stage
  const int oR = oV + (VD / 64) * kBox;              // anchors int32 [G][KD]
  const int nw = G * WPH;                            // consumer warps
  float* qts = reinterpret_cast<float*>(smem + stages * dl.stage_bytes);  // [nw][KD]
  float* xch = qts + nw * KD;                        // [G][WPH - 1][32][VPL + 2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(xch + G * (WPH - 1) * 32 * (VPL + 2));
  auto full = [&](int st) { return smem_u32(&bars[st]); };
  auto empty = [&](int st) { return smem_u32(&bars[stages + st]); };
  auto xfull = [&](int g) { return smem_u32(&bars[2 * stages + g]); };
  auto xempty = [&](int g) { return smem_u32(&bars[2 * stages + G + g]); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;
  const Pick pk = {1, 1};
  start_next();
  for (long i = (long)cta * blockDim.x + threadIdx.x; i < dl.clear_n; i += (long)gridDim.x * blockDim.x)
    dl.clear[i] = 0;
  if (threadIdx.x == 0) {
    parts.desc[cta].last_cta = -1;
    for (int st = 0; st < stages; ++st) {
      mbar_init(full(st), 1);
      mbar_init(empty(st), G);  // one warp of each head takes the tile
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(xfull(g), WPH > 1 ? WPH - 1 : 1);
      mbar_init(xempty(g), 1);
    }
    fence_barrier_init();
  }
  Share sh;
  // three places a CTA at least: the join of more parts would cost what they save
  if (!find_start<kTile, kUnit>(a.bt, a.window, a.H, pk, 3, cta, parts.n_cta, fs, sh)) return;
  const long long x0 = sh.begin(cta), x1 = sh.begin(cta + 1);
  Cursor c = cursor_at<kTile, kUnit>(a.bt, a.window, fs.req, fs.base, x0);
  if (warp == nw) {
    // ------------------------------------------------------------ TMA
    // the lanes hold the next 32 entries of the block table; lane 0 copies
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const uint32_t bytes = (uint32_t)(oR + G * KD * 4);
    const uint64_t once = l2_evict_first();
    const int PS1 = (1 << a.shift) - 1;
    int seq = 0;
    bool ok = true;
    int st = 0;
    uint32_t phase = 1;  // of the empty barrier, from the second round on
    for (long long x = x0; ok && x < x1;) {
      const Run run = run_of<kUnit>(c, x1 - x);
      const int lo = tile_lo(c.r, c.b);
      int slot0 = -32, ids = -1;
      for (int t = run.ta; t < run.tb; ++t) {
        const int j0 = (lo + t) * kTile;
        const int slot = j0 >> a.shift;
        if (slot >= slot0 + 32) {
          slot0 = slot;
          ids = !c.r.dead && slot + lane < a.MP
                    ? page_of(a.table, (long)c.r.i * a.MP, slot + lane, a.NP) : -1;
        }
        const int page = __shfl_sync(0xffffffffu, ids, slot - slot0);
        if (seq >= stages &&
            !__all_sync(0xffffffffu, mbar_wait(empty(st), phase, a.status))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (page < 0 && !c.r.dead) record_status(a.status, WALL_ERR_INVALID_ARG);
          const uint32_t sb = sbase + st * dl.stage_bytes;
          mbar_expect_tx(full(st), bytes);
          // a page that is none: past the pool's end, where the copy reads zeros
          const int kz = page >= 0 ? page * a.HQ + c.h * G : a.NP * a.HQ;
          const int vz = page >= 0 ? page * a.H + c.h : a.NP * a.H;
#pragma unroll
          for (int bx = 0; bx < KD / 64; ++bx)
            tma_load_3d_hint(sb + bx * G * kBox, &tm_k, full(st), bx * 64, j0 & PS1, kz, once);
#pragma unroll
          for (int bx = 0; bx < VD / 64; ++bx)
            tma_load_3d_hint(sb + oV + bx * kBox, &tm_v, full(st), bx * 64, j0 & PS1, vz, once);
          bulk_load(sb + oR, a.rp + ((long)max(page, 0) * a.HQ + (long)c.h * G) * KD, G * KD * 4,
                    full(st));
        }
        __syncwarp();
        ++seq;
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
      }
      x += run.places;
      if (x < x1) next_unit<kTile>(a.bt, a.window, a.H, pk, c);
    }
    // no copy may still be landing when the CTA exits
    for (int q = seq > stages ? seq - stages : 0; q < seq; ++q)
      mbar_wait(full(q % stages), (uint32_t)((q / stages) & 1), a.status);
  } else if (warp < nw) {
    // ------------------------------------------------------------ query heads
    const int g = warp % G, par = warp / G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    float* qt = qts + warp * KD;
    const int win = a.window > 0 ? a.window : 0x7fffffff;
    int st = 0;           // stage and phase of the CTA's next tile
    uint32_t phase = 0;
    int n_seg = 0;
    bool ok = true;
    for (long long x = x0; x < x1;) {
      const Run run = run_of<kUnit>(c, x1 - x);
      const int ta = run.ta, tb = run.tb;
      if (ta == tb) {  // the unit's tiles are the next CTA's
        x += run.places;
        if (x < x1) next_unit<kTile>(a.bt, a.window, a.H, pk, c);
        continue;
      }
      const int kh = c.h, h = kh * G + g;
      const int pos = c.r.kv - 1;  // of the row; its request's last key
      const int lo_key = c.r.dead ? 0 : max(0, pos - win + 1);
      const int lo_tile = tile_lo(c.r, c.b);
      // the query and its prefix beyond the anchor of its own page
      float qv[QPL], pv[QPL];
      int Rq[QPL];
      {
        const long e = ((long)c.r.t0 * a.HQ + h) * KD + lane * QPL;
        const int slot = pos >> a.shift;
        const int page = !c.r.dead && slot < a.MP
                             ? page_of(a.table, (long)c.r.i * a.MP, slot, a.NP) : -1;
#pragma unroll
        for (int y = 0; y < QPL; ++y) {
          qv[y] = to_f32(q[e + y]) * a.scale_log2;
          pv[y] = a.p[e + y];
          Rq[y] = page >= 0 ? a.rp[((long)page * a.HQ + h) * KD + lane * QPL + y] : 0;
        }
      }
      float m = -INFINITY, l = 0.f, acc[VPL];
#pragma unroll
      for (int y = 0; y < VPL; ++y) acc[y] = 0.f;
      int page_at = -1;
      for (int t = ta; t < tb; ++t) {
        const int cs = st;
        const uint32_t cp = phase;
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
        if (!ok || cs % WPH != par) continue;  // another warp's stage
        {
          const bool got = mbar_wait(full(cs), cp, a.status);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            continue;
          }
        }
        const uint8_t* sb = smem + cs * dl.stage_bytes;
        const int j0 = (lo_tile + t) * kTile;
        if ((j0 >> a.shift) != page_at) {
          // the query against this page: scale * log2(e) * q * 2^(p + R - R_c)
          const int* R = reinterpret_cast<const int*>(sb + oR) + g * KD + lane * QPL;
          __syncwarp();
#pragma unroll
          for (int y = 0; y < QPL; ++y) qt[lane * QPL + y] = qv[y] * exp2f(pv[y] + (float)(Rq[y] - R[y]));
          __syncwarp();
          page_at = j0 >> a.shift;
        }
        float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int bx = 0; bx < KD / 64; ++bx) {
          const uint8_t* krow = sb + (bx * G + g) * kBox + lane * 128;
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8) {
            const uint4 u = *reinterpret_cast<const uint4*>(krow + ((c8 ^ (lane & 7)) << 4));
            const float4 qa = *reinterpret_cast<const float4*>(qt + bx * 64 + c8 * 8);
            const float4 qb = *reinterpret_cast<const float4*>(qt + bx * 64 + c8 * 8 + 4);
            const __nv_bfloat162* hv = reinterpret_cast<const __nv_bfloat162*>(&u);
            const float2 f0 = __bfloat1622float2(hv[0]), f1 = __bfloat1622float2(hv[1]);
            const float2 f2 = __bfloat1622float2(hv[2]), f3 = __bfloat1622float2(hv[3]);
            d4[0] = fmaf(f0.x, qa.x, d4[0]); d4[1] = fmaf(f0.y, qa.y, d4[1]);
            d4[2] = fmaf(f1.x, qa.z, d4[2]); d4[3] = fmaf(f1.y, qa.w, d4[3]);
            d4[0] = fmaf(f2.x, qb.x, d4[0]); d4[1] = fmaf(f2.y, qb.y, d4[1]);
            d4[2] = fmaf(f3.x, qb.z, d4[2]); d4[3] = fmaf(f3.y, qb.w, d4[3]);
          }
        }
        const int j = j0 + lane;
        const bool vis = !c.r.dead && j <= pos && j >= lo_key;
        const float s = vis ? (d4[0] + d4[1]) + (d4[2] + d4[3]) : -INFINITY;
        float mt = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        const float m_new = fmaxf(m, mt);
        const float use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m - use);
        const float pr = vis ? exp2f(s - use) : 0.f;
        float ps = pr;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l = l * alpha + ps;
        m = m_new;
#pragma unroll
        for (int y = 0; y < VPL; ++y) acc[y] *= alpha;
        // P V over the visible keys alone: what the other rows of the page
        // hold (NaN included) does not enter
        const int vbx = (lane * VPL) / 64, vch = (lane * VPL) % 64;
        const uint8_t* vbase = sb + oV + vbx * kBox + (vch % 8) * 2;
        auto add_key = [&](int jj) {
          const float pj = __shfl_sync(0xffffffffu, pr, jj);
          const uint8_t* vp = vbase + jj * 128 + (((vch / 8) ^ (jj & 7)) << 4);
          if constexpr (VPL == 4) {
            const uint2 u = *reinterpret_cast<const uint2*>(vp);
            const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
            const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
            acc[0] = fmaf(pj, f0.x, acc[0]); acc[1] = fmaf(pj, f0.y, acc[1]);
            acc[2] = fmaf(pj, f1.x, acc[2]); acc[3] = fmaf(pj, f1.y, acc[3]);
          } else {
            const uint32_t u = *reinterpret_cast<const uint32_t*>(vp);
            const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
            acc[0] = fmaf(pj, f0.x, acc[0]); acc[1] = fmaf(pj, f0.y, acc[1]);
          }
        };
        const int ja = max(0, lo_key - j0), jb = c.r.dead ? 0 : min(kTile, pos + 1 - j0);
        if (ja == 0 && jb == kTile) {
#pragma unroll
          for (int jj = 0; jj < kTile; ++jj) add_key(jj);
        } else {
          for (int jj = ja; jj < jb; ++jj) add_key(jj);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(cs));
      }
      // the head's warps meet: the others hand their states to the first
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      if constexpr (WPH > 1) {
        float* xs = xch + ((g * (WPH - 1)) * 32 + lane) * (VPL + 2);
        if (par > 0) {
          const bool got = n_seg == 0 || mbar_wait(xempty(g), (uint32_t)((n_seg - 1) & 1), a.status);
          float* mine = xs + (par - 1) * 32 * (VPL + 2);
          if (got) {
#pragma unroll
            for (int y = 0; y < VPL; ++y) mine[y] = acc[y];
            mine[VPL] = ok ? m : -INFINITY;  // a part that lacks tiles counts as empty
            mine[VPL + 1] = ok ? l : 0.f;
          }
          __syncwarp();
          if (lane == 0 && got) mbar_arrive(xfull(g));
        } else {
          const bool got = mbar_wait(xfull(g), (uint32_t)(n_seg & 1), a.status);
          if (got) {
            float mf = m;
#pragma unroll
            for (int w = 0; w < WPH - 1; ++w) mf = fmaxf(mf, xs[w * 32 * (VPL + 2) + VPL]);
            const float f0 = m == -INFINITY ? 0.f : exp2f(m - mf);
            l *= f0;
#pragma unroll
            for (int y = 0; y < VPL; ++y) acc[y] *= f0;
#pragma unroll
            for (int w = 0; w < WPH - 1; ++w) {
              const float* o = xs + w * 32 * (VPL + 2);
              const float f = o[VPL] == -INFINITY ? 0.f : exp2f(o[VPL] - mf);
              if (f != 0.f) {
                l = fmaf(o[VPL + 1], f, l);
#pragma unroll
                for (int y = 0; y < VPL; ++y) acc[y] = fmaf(o[y], f, acc[y]);
              }
            }
            m = mf;
          }
          if (!__all_sync(0xffffffffu, got)) ok = false;
          __syncwarp();
          if (lane == 0) mbar_arrive(xempty(g));
        }
      }
      if (par == 0) {
        if (!ok) {  // given up on a wait (reported): an empty part
          m = -INFINITY;
          l = 0.f;
#pragma unroll
          for (int y = 0; y < VPL; ++y) acc[y] = 0.f;
        }
        if (ta == 0 && tb == c.n_tiles) {
          float mf = m, lt = l, f = 1.f;
          if (a.sink) {
            const float sk = a.sink[h] * kLog2e;
            mf = fmaxf(m, sk);
            f = m == -INFINITY ? 0.f : exp2f(m - mf);
            lt = l * f + exp2f(sk - mf);
          }
          const float inv = lt > 0.f || lt != lt ? f / lt : 0.f;
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((long)c.r.t0 * a.HQ + h) * VD + lane * VPL;
#pragma unroll
          for (int y = 0; y < VPL; y += 2)
            *reinterpret_cast<__nv_bfloat162*>(o + y) =
                __floats2bfloat162_rn(acc[y] * inv, acc[y + 1] * inv);
          if (lane == 0 && a.lse)
            a.lse[(long)c.r.t0 * a.HQ + h] = lt == 0.f ? -INFINITY : (mf + log2f(lt)) * kLn2;
        } else {
          const int slot = ta == 0 ? 1 : 0;
          float* po = parts.o(cta, slot, VD) + g * VD + lane * VPL;
#pragma unroll
          for (int y = 0; y < VPL; ++y) po[y] = acc[y];
          if (lane == 0) {
            float* pm = parts.ml(cta, slot, VD) + g * 2;
            pm[0] = m;
            pm[1] = l;
            if (slot == 1 && g == 0) {
              PartDesc d;
              d.t0 = c.r.t0; d.rows = G; d.h = kh;
              d.last_cta = sh.last_owner<kUnit>(c, x);
              parts.desc[cta] = d;
            }
          }
        }
      }
      ++n_seg;
      x += run.places;
      if (x < x1) next_unit<kTile>(a.bt, a.window, a.H, pk, c);
    }
  }
}

template <int KD, int VD, int WPH>
int launch(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  DecodeLaunch dl;
  dl.G = a.HQ / a.H;
  dl.clear = flags.f;
  dl.clear_n = flags.total;
  CUtensorMap tk, tv;
  if (!make_page_map(&tk, a.kp, (long)a.NP * a.HQ, 1 << a.shift, KD, kTile, dl.G) ||
      !make_page_map(&tv, a.vp, (long)a.NP * a.H, 1 << a.shift, VD, kTile, 1))
    return WALL_ERR_CUDA;
  const int oR = (dl.G * (KD / 64) + VD / 64) * kBox;
  dl.stage_bytes = (oR + dl.G * KD * 4 + 1023) & ~1023;
  const int tail = dl.G * WPH * KD * 4 + dl.G * (WPH - 1) * 32 * (VD / 32 + 2) * 4 +
                   (2 * kMaxStages + 2 * dl.G) * 8;
  dl.stages = (226 * 1024 - 1024 - tail) / dl.stage_bytes;
  if (dl.stages > kMaxStages) dl.stages = kMaxStages;
  dl.stages -= dl.stages % WPH;
  const int smem = dl.stages * dl.stage_bytes + tail + 1024;
  static bool attr[kMaxDevices] = {};
  if (!set_max_smem_once(paged_decode_kernel<KD, VD, WPH>, 226 * 1024, attr)) return WALL_ERR_CUDA;
  paged_decode_kernel<KD, VD, WPH><<<parts.n_cta, 32 * (dl.G * WPH + 1), smem, stream>>>(
      tk, tv, a, parts, dl);
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

template <int KD, int VD>
int launch_heads(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  // eight consumer warps where the head count lets them: fewer cannot keep up
  // with the copies
  const int G = a.HQ / a.H;
  if (G == 1) return launch<KD, VD, 8>(a, parts, flags, stream);
  if (G == 2) return launch<KD, VD, 4>(a, parts, flags, stream);
  if (G <= 4) return launch<KD, VD, 2>(a, parts, flags, stream);
  return launch<KD, VD, 1>(a, parts, flags, stream);
}

}  // namespace

namespace paged {

bool decode_rows_supported(int dtype, int H, int HQ, int K, int V) {
  return dtype == WALL_BF16 && (K == 64 || K == 128) && (V == 64 || V == 128) && HQ / H <= 8;
}

int decode_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  if (a.K == 128 && a.V == 128) return launch_heads<128, 128>(a, parts, flags, stream);
  if (a.K == 128) return launch_heads<128, 64>(a, parts, flags, stream);
  if (a.V == 128) return launch_heads<64, 128>(a, parts, flags, stream);
  return launch_heads<64, 64>(a, parts, flags, stream);
}

}  // namespace paged
}  // namespace wall
