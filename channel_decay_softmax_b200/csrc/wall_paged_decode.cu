// wall_paged_decode.cu -- the single-token rows of a paged batch, and the rows
// of one whose requests have at most eight (drafts); bf16, K and V in {64, 128},
// up to 8 query heads a kv head.
//
// Memory-bound: a request's rows read its key rows (per query head), value
// rows (shared by the G heads of a kv head) and anchors once.  One CTA per SM
// streams an even share of the batch's 32-key tiles of (request, kv head):
// the last warp's lane 0 keeps a ring of TMA stages full (per tile one box of
// 64 channels x 32 rows x G heads per 128 bytes of key row -- the pages are
// head-major, so each head's piece is contiguous -- the value boxes and the
// page's anchors), and the tile's G heads have WPH warps each that take
// alternate stages with a softmax state of their own.  A stage is the same
// warp's in every round (the stages are a multiple of WPH): a wait on a
// barrier's parity tells a phase only from the one before, which its waiter
// has to have seen.  The share runs across requests and heads, so the ring
// never drains between them, and a batch of any lengths loads every SM alike.
//
// So few rows give the tensor cores little to reuse, but as warp-level matrix
// products (m16n8k16: 16 keys, or 16 value channels, by 8 columns) the two
// contractions take a quarter of the instructions of fp32 FMAs, which unpack
// every element first and bound this kernel by issue and power (32 requests of
// 4096 to 16000 tokens: 506 us cold and 587 us at the 1000 W limit; so 450 and
// 453, 3.1 GB at 6.9 TB/s).
//
// One row: the 8 columns hold the one vector's parts, q 2^(...) as a sum of
// three bf16 (24 bits: nothing of the fp32 value is lost) and P as a sum of two
// (to 2^-16, beside the output's rounding of 2^-8).  Up to eight rows: the
// columns are the rows, and q 2^(...) is rounded to bf16 as the kernel for
// longer requests rounds it (its second part would spill: 91 us for the drafts
// that take 74); P keeps its two parts (72 us without, and the result's error
// 1.45 times the output rounding's instead of 1.2).  P's sum is of its fp32
// values, sums are fp32.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

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

// A query's operand in shared memory: per (lane & 3, part) the words of its
// k-steps, 80 bytes apart so that a warp's vector reads meet few banks twice
constexpr int kQGroup = 80, kQBytes = 1024;

__device__ __forceinline__ void ldsm4(uint32_t (&d)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&d)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two floats to bf16, the first in the low half
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// what a bf16 part leaves of a value; of an infinity nothing
__device__ __forceinline__ float rest_of(float x, float part) {
  return fabsf(part) == INFINITY ? 0.f : x - part;
}
// P's two bf16 parts: its leading 8 bits and the rest (to 2^-16 of it).  Neither
// is below 0, nor 0 where P is not: an infinite value stays infinite times both.
__device__ __forceinline__ float lead_of(float p) {
  return __uint_as_float(__float_as_uint(p) & 0xffff0000u);
}
__device__ __forceinline__ float trail_of(float p) {
  return fmaxf(p - lead_of(p), fminf(p, 1.17549435e-38f));  // 2^-126
}

// an 8 x 8 block of bf16 pairs, transposed among the lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(w));
  return d;
}
// x 2^e, in two steps: 2^e itself may lie outside fp32 where the product does not
__device__ __forceinline__ float times_pow2(float x, int e) {
  e = min(max(e, -252), 252);
  const int half = e >> 1;
  return x * __int_as_float((half + 127) << 23) * __int_as_float((e - half + 127) << 23);
}
// any half of the word that is an infinity or a NaN
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t pair_mask(int j, int ja, int jb) {  // keys j, j + 1 in [ja, jb)
  return (j >= ja && j < jb ? 0xffffu : 0u) | (j + 1 >= ja && j + 1 < jb ? 0xffff0000u : 0u);
}

struct DecodeLaunch {
  int G, stages, stage_bytes;
  int rows;  // requests of up to so many rows are this kernel's
  int* clear;  // words to clear, for the kernels behind this one
  long clear_n;
};

// kMany: requests of one to kShortRows rows, otherwise those of one
template <int KD, int VD, int WPH, bool kMany>
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
  uint8_t* qts = smem + stages * dl.stage_bytes;     // [nw] query operands
  constexpr int XW = (kMany ? kShortRows : 1) * (VD + 4);          // a warp's states: per row sums, m, l
  float* xch = reinterpret_cast<float*>(qts + nw * kQBytes);  // [G][WPH][XW]
  uint64_t* bars = reinterpret_cast<uint64_t*>(xch + nw * XW);
  auto full = [&](int st) { return smem_u32(&bars[st]); };
  auto empty = [&](int st) { return smem_u32(&bars[stages + st]); };
  auto xfull = [&](int g) { return smem_u32(&bars[2 * stages + g]); };
  auto xempty = [&](int g) { return smem_u32(&bars[2 * stages + G + g]); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;
  const Pick pk = {1, dl.rows};
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
    uint8_t* qt = qts + warp * kQBytes;
    // this lane's place among the fragments: row or column lane / 4, pair lane % 4
    const int quad = lane >> 2, pr4 = lane & 3;
    // columns 2j hold the first part, odd ones the second and third in turns
    const int part = (quad & 1) == 0 ? 0 : (quad & 2) == 0 ? 1 : 2;
    // ldmatrix rows: of a key tile (keys, then channels on), of a value tile
    // (channels, then keys on); both 128-byte rows with the 128-byte swizzle
    const int sw = lane & 7;
    const uint32_t krow = (sw + ((lane >> 3) & 1) * 8) * 128, kch = lane >> 4;
    const uint32_t vrow = (sw + (lane >> 4) * 8) * 128, vch = (lane >> 3) & 1;
    uint32_t qb[KD / 8];  // the query's fragments, two words a k-step
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
      const int kh = c.h, h = kh * G + g, n = c.r.n;
      const int lo_tile = tile_lo(c.r, c.b);
      // this warp's tiles of the run, one after the other
      auto each_tile = [&](auto body) {
        for (int t = ta; t < tb; ++t) {
          const int cs = st;
          const uint32_t cp = phase;
          if (++st == stages) {
            st = 0;
            phase ^= 1;
          }
          if (!ok || cs % WPH != par) continue;  // another warp's stage
          if (!__all_sync(0xffffffffu, mbar_wait(full(cs), cp, a.status))) {
            ok = false;
            continue;
          }
          body(smem + cs * dl.stage_bytes, (lo_tile + t) * kTile);
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(cs));
        }
      };
      float* mine = xch + (g * WPH + par) * XW;
      // the first of the head's warps has taken the last run's state from here
      auto may_lay = [&] {
        if (!__all_sync(0xffffffffu, ok)) ok = false;
        return par == 0 || n_seg == 0 ||
               __all_sync(0xffffffffu, mbar_wait(xempty(g), (uint32_t)((n_seg - 1) & 1), a.status));
      };
      bool laid;
      int page_at = -1;
      if constexpr (!kMany) {
        const int pos = c.r.kv - 1;  // of the row; its request's last key
        const int lo_key = c.r.dead ? 0 : max(0, pos - win + 1);
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
        float m = -INFINITY, l = 0.f;
        float acc[VD / 16][4];  // channels 16 c + quad (parts 0, 1) and + 8
  #pragma unroll
        for (int y = 0; y < VD / 16; ++y)
  #pragma unroll
          for (int e = 0; e < 4; ++e) acc[y][e] = 0.f;
        each_tile([&](const uint8_t* sb, int j0) {
          if ((j0 >> a.shift) != page_at) {
            // the query against this page: scale * log2(e) * q * 2^(p + R - R_c),
            // its three parts to the words that the fragments read
            const int* R = reinterpret_cast<const int*>(sb + oR) + g * KD + lane * QPL;
            __syncwarp();
  #pragma unroll
            for (int y = 0; y < QPL; y += 2) {
              const float e0 = pv[y] + (float)(Rq[y] - R[y]);
              const float e1 = pv[y + 1] + (float)(Rq[y + 1] - R[y + 1]);
              float x0 = qv[y] * exp2f(e0), x1 = qv[y + 1] * exp2f(e1);
              if (fmaxf(e0, e1) > kPageRange) {
                x0 = grown_query(qv[y], e0);
                x1 = grown_query(qv[y + 1], e1);
              }
              const int ch = lane * QPL + y, pair = (ch & 15) >> 1;
              uint8_t* w = qt + (pair & 3) * 3 * kQGroup + ((ch >> 4) * 2 + (pair >> 2)) * 4;
  #pragma unroll
              for (int z = 0; z < 3; ++z) {
                const uint32_t h = pack2(x0, x1);
                *reinterpret_cast<uint32_t*>(w + z * kQGroup) = h;
                x0 = rest_of(x0, low_of(h));
                x1 = rest_of(x1, high_of(h));
              }
            }
            __syncwarp();
  #pragma unroll
            for (int y = 0; y < KD / 8; y += 4) {
              const uint4 u = *reinterpret_cast<const uint4*>(qt + (pr4 * 3 + part) * kQGroup + y * 4);
              qb[y] = u.x; qb[y + 1] = u.y; qb[y + 2] = u.z; qb[y + 3] = u.w;
            }
            page_at = j0 >> a.shift;
          }
          // scores of keys quad + 8 i: 16 keys an instruction
          float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          const uint32_t kb = smem_u32(sb) + g * kBox + krow;
  #pragma unroll
          for (int ks = 0; ks < KD / 16; ++ks) {
            const uint32_t at = kb + (ks / 4) * G * kBox + ((((ks & 3) * 2 + kch) ^ sw) << 4);
  #pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t ka[4];
              ldsm4(ka, at + y * 16 * 128);
              mma16816(d[y], ka, qb[ks * 2], qb[ks * 2 + 1]);
            }
          }
          const int ja = max(0, lo_key - j0), jb = c.r.dead ? 0 : min(kTile, pos + 1 - j0);
          float sc[4], mt = -INFINITY;
  #pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float lo = d[y >> 1][(y & 1) * 2 + 1];
            sc[y] = d[y >> 1][(y & 1) * 2] + (lo + __shfl_xor_sync(0xffffffffu, lo, 1));
            const int j = quad + 8 * y;
            if (j < ja || j >= jb) sc[y] = -INFINITY;
            mt = fmaxf(mt, sc[y]);
          }
  #pragma unroll
          for (int o = 16; o > 2; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
          if (mt > m) {  // the same for the whole warp
            const float alpha = exp2f(m - mt);
            l *= alpha;
  #pragma unroll
            for (int y = 0; y < VD / 16; ++y)
  #pragma unroll
              for (int e = 0; e < 4; ++e) acc[y][e] *= alpha;
            m = mt;
          }
          const float use = m == -INFINITY ? 0.f : m;
          uint32_t pw[4];  // a key's P: first part and second
          float ps = 0.f;
  #pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int j = quad + 8 * y;
            const float p = j < ja || j >= jb ? 0.f : exp2f(sc[y] - use);
            ps += p;
            pw[y] = pack2(lead_of(p), trail_of(p));
          }
  #pragma unroll
          for (int o = 16; o > 2; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
          l += ps;
          // P V.  Of the keys that the row does not see the values count as 0:
          // what those rows of the page hold (NaN included) does not enter.
          const uint32_t vb = smem_u32(sb) + oV + vrow;
          auto add_values = [&](auto all) {
  #pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              uint32_t pb[2], keep[2];
  #pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t w0 = __shfl_sync(0xffffffffu, pw[ks * 2 + y], pr4 * 8);
                const uint32_t w1 = __shfl_sync(0xffffffffu, pw[ks * 2 + y], pr4 * 8 + 4);
                pb[y] = __byte_perm(w0, w1, (quad & 1) == 0 ? 0x5410 : 0x7632);
                const int j = ks * 16 + y * 8 + pr4 * 2;
                keep[y] = pair_mask(j, ja, jb);
              }
  #pragma unroll
              for (int y = 0; y < VD / 16; ++y) {
                uint32_t va[4];
                ldsm4_t(va, vb + (y / 4) * kBox + ks * 16 * 128 + ((((y & 3) * 2 + vch) ^ sw) << 4));
                if constexpr (!decltype(all)::value) {
                  va[0] &= keep[0];
                  va[1] &= keep[0];
                  va[2] &= keep[1];
                  va[3] &= keep[1];
                }
                mma16816(acc[y], va, pb[0], pb[1]);
              }
            }
          };
          if (ja == 0 && jb == kTile) add_values(std::true_type{});
          else add_values(std::false_type{});
        });
        laid = may_lay();
        if (laid) {
#pragma unroll
          for (int y = 0; y < VD / 16; ++y) {
            if ((y & 3) != pr4) continue;  // the quad's lanes hold the same
            mine[y * 16 + quad] = acc[y][0] + acc[y][1];
            mine[y * 16 + 8 + quad] = acc[y][2] + acc[y][3];
          }
          if (lane == 0) {
            mine[VD] = ok ? m : -INFINITY;  // a part that lacks tiles counts as empty
            mine[VD + 1] = ok ? l : 0.f;
          }
        }
      } else {
        // Up to eight rows: the columns are rows.  Lane: fragments of row
        // `quad`, scores and sums of rows r0, r0 + 1.
        const int r0 = pr4 * 2, ctx = c.r.kv - n;
        // q 2^p of row `quad`, channels 8 y + r0 and the next, and the anchors of
        // the two pages that the rows may lie in
        const bool real = quad < n && !c.r.dead;
        const int slot0 = ctx >> a.shift;
        int* Rq = reinterpret_cast<int*>(qt);
        __syncwarp();
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int page = !c.r.dead && slot0 + z < a.MP
                               ? page_of(a.table, (long)c.r.i * a.MP, slot0 + z, a.NP) : -1;
          for (int y = lane; y < KD; y += 32)
            Rq[z * KD + y] = page >= 0 ? a.rp[((long)page * a.HQ + h) * KD + y] : 0;
        }
        __syncwarp();
        Rq += (((ctx + quad) >> a.shift) > slot0 ? KD : 0) + r0;
        float2 xq[KD / 8];
        {
          const long own = ((long)(c.r.t0 + (real ? quad : 0)) * a.HQ + h) * KD + r0;
#pragma unroll
          for (int y = 0; y < KD / 8; ++y) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(q + own + y * 8);
            const float2 p = *reinterpret_cast<const float2*>(a.p + own + y * 8);
            xq[y] = make_float2(real ? low_of(w) * a.scale_log2 * exp2f(p.x) : 0.f,
                                real ? high_of(w) * a.scale_log2 * exp2f(p.y) : 0.f);
          }
        }
        // keys [lo, hi) that the lane's two rows see
        int lo[2], hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool real = r0 + x < n && !c.r.dead;
          lo[x] = real ? max(0, ctx + r0 + x - win + 1) : 0;
          hi[x] = real ? ctx + r0 + x + 1 : 0;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[VD / 16][4];
#pragma unroll
        for (int y = 0; y < VD / 16; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[y][e] = 0.f;  // channels 16 y + quad (rows r0, r0 + 1) and + 8
        uint32_t qh[KD / 8];  // the rows' fragments
        each_tile([&](const uint8_t* sb, int j0) {
          if ((j0 >> a.shift) != page_at) {
            page_at = j0 >> a.shift;
            const int* R = reinterpret_cast<const int*>(sb + oR) + g * KD + r0;
            float most = 0.f;
#pragma unroll
            for (int y = 0; y < KD / 8; ++y) {
              const int2 rc = *reinterpret_cast<const int2*>(R + y * 8);
              const int2 ro = *reinterpret_cast<const int2*>(Rq + y * 8);
              const float x0 = times_pow2(xq[y].x, ro.x - rc.x), x1 = times_pow2(xq[y].y, ro.y - rc.y);
              most = fmaxf(most, fmaxf(fabsf(x0), fabsf(x1)));
              qh[y] = pack2(x0, x1);
            }
            if (most > kMostQuery) {
#pragma unroll
              for (int y = 0; y < KD / 8; ++y)
                qh[y] = pack2(bound_query(low_of(qh[y]), xq[y].x), bound_query(high_of(qh[y]), xq[y].y));
            }
          }
          // scores of keys quad + 8 i
          float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          const uint32_t kb = smem_u32(sb) + g * kBox + krow;
#pragma unroll
          for (int ks = 0; ks < KD / 16; ++ks) {
            const uint32_t at = kb + (ks / 4) * G * kBox + ((((ks & 3) * 2 + kch) ^ sw) << 4);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t ka[4];
              ldsm4(ka, at + y * 16 * 128);
              mma16816(d[y], ka, qh[ks * 2], qh[ks * 2 + 1]);
            }
          }
          float mt[2] = {m[0], m[1]};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = j0 + quad + 8 * i;
              float& v = d[i >> 1][(i & 1) * 2 + x];
              if (j < lo[x] || j >= hi[x]) v = -INFINITY;
              mt[x] = fmaxf(mt[x], v);
            }
#pragma unroll
          for (int o = 16; o > 2; o >>= 1)
#pragma unroll
            for (int x = 0; x < 2; ++x) mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], o));
          if (__any_sync(0xffffffffu, mt[0] > m[0] || mt[1] > m[1])) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float alpha = mt[x] > m[x] ? exp2f(m[x] - mt[x]) : 1.f;
              l[x] *= alpha;
#pragma unroll
              for (int y = 0; y < VD / 16; ++y) {
                acc[y][x] *= alpha;
                acc[y][2 + x] *= alpha;
              }
              m[x] = mt[x];
            }
          }
          uint32_t ph[4], pl[4];  // P's fragments of keys 8 i on: first and second part
          float ps[2] = {0.f, 0.f};
          const float use[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = j0 + quad + 8 * i;
              p[x] = j < lo[x] || j >= hi[x] ? 0.f : exp2f(d[i >> 1][(i & 1) * 2 + x] - use[x]);
              ps[x] += p[x];
            }
            ph[i] = transpose8(__byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632));
            pl[i] = transpose8(pack2(trail_of(p[0]), trail_of(p[1])));
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) ps[x] += __shfl_xor_sync(0xffffffffu, ps[x], o);
            l[x] += ps[x];
          }
          // P V.  A value row counts as 0 where no row sees its key.  One that
          // some rows see and others do not must be finite for these products
          // (0 * inf); where one is not, the rows go one by one.
          const uint32_t vb = smem_u32(sb) + oV + vrow;
          auto value = [&](uint32_t (&va)[4], int ks, int y, int ja, int jb) {
            ldsm4_t(va, vb + (y / 4) * kBox + ks * 16 * 128 + ((((y & 3) * 2 + vch) ^ sw) << 4));
            const uint32_t k0 = pair_mask(ks * 16 + r0, ja, jb), k1 = pair_mask(ks * 16 + 8 + r0, ja, jb);
            va[0] &= k0;
            va[1] &= k0;
            va[2] &= k1;
            va[3] &= k1;
          };
          auto seen_from = [&](int row) { return c.r.dead ? kTile : max(0, max(0, ctx + row - win + 1) - j0); };
          auto seen_to = [&](int row) { return c.r.dead ? 0 : min(kTile, ctx + row + 1 - j0); };
          const int ja = seen_from(0), jb = seen_to(n - 1);  // by some row
          const bool part = seen_from(n - 1) > 0 || seen_to(0) < kTile;
          bool split = false;
          if (part) {
            uint32_t bad = 0;
#pragma unroll 1
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll 4
              for (int y = 0; y < VD / 16; ++y) {
                uint32_t va[4];
                value(va, ks, y, ja, jb);
                bad |= not_finite(va[0]) | not_finite(va[1]) | not_finite(va[2]) | not_finite(va[3]);
              }
            split = __any_sync(0xffffffffu, bad != 0);
          }
          if (!part) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
              for (int y = 0; y < VD / 16; ++y) {
                uint32_t va[4];
                ldsm4_t(va, vb + (y / 4) * kBox + ks * 16 * 128 + ((((y & 3) * 2 + vch) ^ sw) << 4));
                mma16816(acc[y], va, ph[ks * 2], ph[ks * 2 + 1]);
                mma16816(acc[y], va, pl[ks * 2], pl[ks * 2 + 1]);
              }
          } else {
#pragma unroll 1
            for (int row = 0; row < (split ? n : 1); ++row) {
              const int from = split ? seen_from(row) : ja, to = split ? seen_to(row) : jb;
              const bool take0 = !split || row == r0, take1 = !split || row == r0 + 1;
#pragma unroll
              for (int y = 0; y < VD / 16; ++y) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                  uint32_t va[4];
                  value(va, ks, y, from, to);
                  mma16816(t, va, ph[ks * 2], ph[ks * 2 + 1]);
                  mma16816(t, va, pl[ks * 2], pl[ks * 2 + 1]);
                }
                acc[y][0] += take0 ? t[0] : 0.f;
                acc[y][1] += take1 ? t[1] : 0.f;
                acc[y][2] += take0 ? t[2] : 0.f;
                acc[y][3] += take1 ? t[3] : 0.f;
              }
            }
          }
        });
        laid = may_lay();
        if (laid) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float* row = mine + (r0 + x) * (VD + 4);
            if (r0 + x >= n) continue;
#pragma unroll
            for (int y = 0; y < VD / 16; ++y) {
              row[y * 16 + quad] = acc[y][x];
              row[y * 16 + 8 + quad] = acc[y][2 + x];
            }
            if (quad == 0) {
              row[VD] = ok ? m[x] : -INFINITY;
              row[VD + 1] = ok ? l[x] : 0.f;
            }
          }
        }
      }
      // The head's warps meet: each has laid its state into shared memory in
      // the channels' order (one that gave up on a wait has not, nor tells of
      // it), and the first joins them.
      __syncwarp();
      if (!laid) ok = false;
      else if (par > 0 && lane == 0) mbar_arrive(xfull(g));
      if (par == 0) {
        if (WPH > 1 && !__all_sync(0xffffffffu, mbar_wait(xfull(g), (uint32_t)(n_seg & 1), a.status)))
          ok = false;
        const bool whole = ta == 0 && tb == c.n_tiles;
        const int slot = ta == 0 ? 1 : 0;
        for (int row = 0; row < n; ++row) {
          float m = -INFINITY, l = 0.f, o_sum[VPL];
#pragma unroll
          for (int y = 0; y < VPL; ++y) o_sum[y] = 0.f;
          if (ok) {  // otherwise (reported): an empty part
            const float* xs = mine + row * (VD + 4);
#pragma unroll
            for (int w = 0; w < WPH; ++w) m = fmaxf(m, xs[w * XW + VD]);
#pragma unroll
            for (int w = 0; w < WPH; ++w) {
              const float* o = xs + w * XW;
              const float f = o[VD] == -INFINITY ? 0.f : exp2f(o[VD] - m);
              if (f != 0.f) {
                l = fmaf(o[VD + 1], f, l);
#pragma unroll
                for (int y = 0; y < VPL; ++y) o_sum[y] = fmaf(o[lane * VPL + y], f, o_sum[y]);
              }
            }
          }
          if (whole) {
            float mf = m, lt = l, f = 1.f;
            if (a.sink) {
              const float sk = a.sink[h] * kLog2e;
              mf = fmaxf(m, sk);
              f = m == -INFINITY ? 0.f : exp2f(m - mf);
              lt = l * f + sink_weight(sk, mf);
            }
            const float inv = lt > 0.f || lt != lt ? f / lt : 0.f;
            const long at = (long)(c.r.t0 + row) * a.HQ + h;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + at * VD + lane * VPL;
#pragma unroll
            for (int y = 0; y < VPL; y += 2)
              *reinterpret_cast<__nv_bfloat162*>(o + y) =
                  __floats2bfloat162_rn(o_sum[y] * inv, o_sum[y + 1] * inv);
            if (lane == 0 && a.lse) a.lse[at] = lt == 0.f ? -INFINITY : (mf + log2f(lt)) * kLn2;
          } else {
            const int at = row * G + g;
            float* po = parts.o(cta, slot, VD) + at * VD + lane * VPL;
#pragma unroll
            for (int y = 0; y < VPL; ++y) po[y] = o_sum[y];
            if (lane == 0) {
              float* pm = parts.ml(cta, slot, VD) + at * 2;
              pm[0] = m;
              pm[1] = l;
            }
          }
        }
        if (!whole && slot == 1 && g == 0 && lane == 0) {
          PartDesc d;
          d.t0 = c.r.t0; d.rows = G * n; d.h = kh;
          d.last_cta = sh.last_owner<kUnit>(c, x);
          parts.desc[cta] = d;
        }
        __syncwarp();
        if (WPH > 1 && lane == 0) mbar_arrive(xempty(g));
      }
      ++n_seg;
      x += run.places;
      if (x < x1) next_unit<kTile>(a.bt, a.window, a.H, pk, c);
    }
  }
}

template <int KD, int VD, int WPH, bool kMany>
int launch(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  DecodeLaunch dl;
  dl.G = a.HQ / a.H;
  dl.rows = kMany ? a.max_new : 1;
  dl.clear = flags.f;
  dl.clear_n = flags.total;
  CUtensorMap tk, tv;
  if (!make_page_map(&tk, a.kp, (long)a.NP * a.HQ, 1 << a.shift, KD, kTile, dl.G) ||
      !make_page_map(&tv, a.vp, (long)a.NP * a.H, 1 << a.shift, VD, kTile, 1))
    return WALL_ERR_CUDA;
  const int oR = (dl.G * (KD / 64) + VD / 64) * kBox;
  dl.stage_bytes = (oR + dl.G * KD * 4 + 1023) & ~1023;
  const int tail = dl.G * WPH * (kQBytes + (kMany ? kShortRows : 1) * (VD + 4) * 4) +
                   (2 * kMaxStages + 2 * dl.G) * 8;
  dl.stages = (226 * 1024 - 1024 - tail) / dl.stage_bytes;
  if (dl.stages > kMaxStages) dl.stages = kMaxStages;
  dl.stages -= dl.stages % WPH;
  const int smem = dl.stages * dl.stage_bytes + tail + 1024;
  const int threads = 32 * (dl.G * WPH + 1);
  static bool attr[kMaxDevices] = {};
  auto* kernel = paged_decode_kernel<KD, VD, WPH, kMany>;
  if (!set_max_smem_once(kernel, 226 * 1024, attr)) return WALL_ERR_CUDA;
  kernel<<<parts.n_cta, threads, smem, stream>>>(tk, tv, a, parts, dl);
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

template <int KD, int VD, bool kMany>
int launch_heads(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  // warps a head: enough to keep up with the copies
  const int G = a.HQ / a.H;
  if (G == 1) return launch<KD, VD, 4, kMany>(a, parts, flags, stream);
  if (G <= 4) return launch<KD, VD, 2, kMany>(a, parts, flags, stream);
  return launch<KD, VD, 1, kMany>(a, parts, flags, stream);
}

template <bool kMany>
int rows_of(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  if (a.K == 128 && a.V == 128) return launch_heads<128, 128, kMany>(a, parts, flags, stream);
  if (a.K == 128) return launch_heads<128, 64, kMany>(a, parts, flags, stream);
  if (a.V == 128) return launch_heads<64, 128, kMany>(a, parts, flags, stream);
  return launch_heads<64, 64, kMany>(a, parts, flags, stream);
}

}  // namespace

namespace paged {

bool decode_rows_supported(int dtype, int H, int HQ, int K, int V) {
  return dtype == WALL_BF16 && (K == 64 || K == 128) && (V == 64 || V == 128) && HQ / H <= 8;
}

int decode_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream) {
  return few_rows(a.max_new) ? rows_of<true>(a, parts, flags, stream) : rows_of<false>(a, parts, flags, stream);
}

}  // namespace paged
}  // namespace wall
