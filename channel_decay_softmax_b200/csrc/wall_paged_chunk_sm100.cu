// wall_paged_chunk_sm100.cu -- rows of requests with two or more new tokens
// over the paged Wall cache, on the tensor cores (tcgen05 + TMEM + TMA; bf16,
// K == V in {64, 128}): prompts, chunks of prompts, drafts.
//
// Math.  A unit is 128 query rows of one (request, head).  With R_I the anchor
// of the page that holds its first row,
//   Qh_i = q_i 2^(p_i + R_{page(i)} - R_I)       (a small kernel before this one)
//   s_ij = scale sum_n Qh_in (k_jn 2^(R_I,n - R_{page(j),n}))
// where k_j is the cached row.  The anchors are whole numbers, so scaling the
// key tile is exact: Qh is the only operand that is rounded (to bf16, half a
// step of 2^-8, as a tensor-core operand has to be).  P is rounded to bf16
// for P V; its sum is taken in fp32 before that.  A unit whose exponents pass
// +-100 on some channel, or whose partly masked tiles hold a value that is not
// finite (it would reach the masked rows as 0 * inf), is flagged, and the
// general kernel computes it again, exactly, behind this one.
//
// Work.  One CTA per SM takes an even share of the batch's (unit, 128-key
// tile) pairs in order (wall_paged.cuh): the tile pipeline's rings and
// barriers run on across the units, a prompt's short first blocks and long
// last ones balance to within a tile, and a few rows over a long context
// spread over all SMs and are joined afterwards.
//
// 12 warps (3 per SM sub-partition, 168 registers each):
//   warp 0      TMA, one thread: the key ring (3 stages, with the pages'
//               anchors), the value ring (2 stages), the units' Qh
//   warp 1      TMEM owner and MMA issuer (one thread)
//   warps 2-3   key rescale in place; partly masked tiles: value rows past the
//               request's end zeroed (pages end inside tiles; what they hold
//               there is another request's, or nothing), the others checked
//   warps 4-7   softmax of the CTA's even tiles, warps 8-11 of its odd ones:
//               one query row a thread, the two groups' (m, l, O) merged at a
//               unit's end
// TMEM columns: S0 [0,128), S1 [128,256), O_even [256, 256+V), O_odd behind it.
#include <cuda.h>

#include <type_traits>

#include "sm100_ptx.cuh"
#include "wall_paged_attn.h"

namespace wall {
namespace {

using namespace sm100;
using namespace paged;

constexpr int BM = kChunkRows;
constexpr int BN = kChunkRows;
constexpr int kThreads = 384;
constexpr int kKS = 3;                    // key stages
constexpr int kVS = 2;                    // value stages
constexpr float kRescaleThreshold = 8.f;  // log2 units: lazy O rescale
constexpr float kRescaleBound = 256.f;    // 2^kRescaleThreshold

template <int KD>
struct Smem {
  static constexpr int kT = BN * KD * 2;           // one 128-row bf16 tile
  static constexpr int kRows = BN / 32;            // most pages of a tile
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + kT;               // kKS stages
  static constexpr int oV = oK + kKS * kT;         // kVS stages
  static constexpr int oR = oV + kVS * kT;         // int[kKS][kRows][KD] anchors
  static constexpr int oX = oR + kKS * kRows * KD * 4;  // float[2][2 groups][2][BM]: m, l
  static constexpr int oBar = oX + 2 * 2 * 2 * BM * 4;
  static constexpr int kBars = 26;
  static constexpr int oMisc = oBar + kBars * 8;   // TMEM base, abort flag
  static constexpr int kBytes = oMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;     // slack for 1 KB alignment
};

// barrier slots, laid out from the stage counts
enum Bar {
  B_QFULL = 0,
  B_QEMPTY,
  B_KFULL,                      // + key stage
  B_KREADY = B_KFULL + kKS,     // + key stage, 2 rescale warps
  B_KEMPTY = B_KREADY + kKS,    // + key stage
  B_VFULL = B_KEMPTY + kKS,     // + value stage: ready for P V (2 arrivals)
  B_VEMPTY = B_VFULL + kVS,     // + value stage
  B_VRAW = B_VEMPTY + kVS,      // + value stage: a partly masked tile has landed
  B_SFULL = B_VRAW + kVS,       // + S buffer (2)
  B_PFULL = B_SFULL + 2,        // + group (2), 4 warps each
  B_PVDONE = B_PFULL + 2,       // + group (2)
  B_XCHG = B_PVDONE + 2,        // exchange of m, l between the groups (8 warps)
  B_OEMPTY,                     // both O accumulators read (8 warps)
  B_MMADONE,
  kNumBars,
};
static_assert(kNumBars <= Smem<128>::kBars, "barrier slots");

// bounded wait that also gives up once another role has given up
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, int* status,
                                         volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, 100000u)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > 1000000000ull) {
      record_status(status, WALL_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 2^e as bf16 bits: exact in the normal range, 0 below it
__device__ __forceinline__ uint32_t pow2_bf16(int e) {
  return e < -126 ? 0u : e > 127 ? 0x7F80u : uint32_t(e + 127) << 7;
}

// Any half of the word that is an infinity or a NaN
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// The CTA's run of tiles, unit by unit.
struct Segment {
  int t0;         // first query row of the unit among the packed ones
  int ni;         // its rows
  int pos0;       // position of the first
  int lo;         // first tile
  int ta, tb;     // the segment's tiles, counted from lo
};
__device__ __forceinline__ Segment segment_of(const Cursor& c, long long left) {
  Segment s;
  s.t0 = c.r.t0 + c.b * BM;
  s.ni = min(BM, c.r.n - c.b * BM);
  s.pos0 = c.r.ctx + c.b * BM;
  s.lo = tile_lo(c.r, c.b);
  s.ta = c.t;
  s.tb = (int)min((long long)c.n_tiles, c.t + left);
  return s;
}
// Whether every row of the unit sees all of the tile that begins at j0.
__device__ __forceinline__ bool sees_all(const Segment& s, bool dead, int j0, int win) {
  return !dead && j0 + BN - 1 <= s.pos0 && s.pos0 + s.ni - 1 - j0 < win;
}

template <int KD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, AttnArgs a, Parts parts,
                       UnitFlags flags) {
  using Lay = Smem<KD>;
  constexpr int V = KD;
  extern __shared__ uint8_t smem_raw[];
  __shared__ FindScratch fs;
  __shared__ Cursor s_cur[8];  // the softmax warps' places (their registers are full)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* sX = reinterpret_cast<float*>(smem + Lay::oX);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oMisc + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;
  const int HQ = a.HQ;
  const int win = a.window > 0 ? a.window : 0x7fffffff;
  const Pick pk = {2, 0x7fffffff};

  if (threadIdx.x == 0) {
    parts.desc[cta].last_cta = -1;
    mbar_init(bar(B_QFULL), 1);
    mbar_init(bar(B_QEMPTY), 1);
    for (int s = 0; s < kKS; ++s) {
      mbar_init(bar(B_KFULL + s), 1);
      mbar_init(bar(B_KREADY + s), 2);
      mbar_init(bar(B_KEMPTY + s), 1);
    }
    for (int s = 0; s < kVS; ++s) {
      mbar_init(bar(B_VFULL + s), 2);
      mbar_init(bar(B_VEMPTY + s), 1);
      mbar_init(bar(B_VRAW + s), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(B_SFULL + g), 1);
      mbar_init(bar(B_PFULL + g), 4);
      mbar_init(bar(B_PVDONE + g), 1);
    }
    mbar_init(bar(B_XCHG), 8);
    mbar_init(bar(B_OEMPTY), 8);
    mbar_init(bar(B_MMADONE), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  Share sh;
  if (!find_start<BM>(a.bt, a.window, HQ, pk, 2, cta, parts.n_cta, fs, sh)) return;
  const long long x0 = sh.begin(cta), x1 = sh.begin(cta + 1);
  const int n_tiles = (int)(x1 - x0);  // of this CTA
  Cursor c = cursor_at<BM>(a.bt, a.window, fs.req, fs.base, x0);
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int PS = 1 << a.shift;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA
    // One thread issues every copy, in the order in which the MMAs free their
    // places: S(0) S(1) PV(0) S(2) PV(1) S(3) ... complete in that order, so
    // key tile g (behind S(g - 3)), then value tile g - 2 (behind PV(g - 4))
    // never waits past a copy that could go.  A unit's Qh goes out once the
    // last S of the unit before has read its rows, two tiles into the unit.
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_q);
      Cursor cv = c;                    // of value tile (and unit) g - 2
      int seg_v = 0, k_out = 0, v_out = 0, q_out = 0;
      uint32_t raw = 0, raw_next = 0;   // per value stage: its last tile is a partly masked one;
                                        // parity of the next one's B_VRAW phase
      long long xk = x0, xv = x0;       // where the current units' segments begin
      Segment sk = segment_of(c, x1 - xk), sv = sk;
      int tk = sk.ta, tv = sv.ta;
      auto load_q = [&]() {
        mbar_expect_tx(bar(B_QFULL), Lay::kT);
        for (int bx = 0; bx < KD / 64; ++bx)
          tma_load_3d(sbase + Lay::oQ + bx * (BM * 128), &tm_q, bar(B_QFULL), bx * 64, cv.h, sv.t0);
        ++q_out;
      };
      // the pages that hold tile t's keys into stage st of the key or value ring
      auto load_tile = [&](auto keys_tag, const Cursor& cc, const Segment& s, int t, int st,
                           uint32_t full) {
        constexpr bool keys = decltype(keys_tag)::value;
        const CUtensorMap* tm = keys ? &tm_k : &tm_v;
        const uint32_t dst = sbase + (keys ? Lay::oK : Lay::oV) + st * Lay::kT;
        const int j0 = (s.lo + t) * BN;
        const int nk = cc.r.dead ? 0 : min(BN, cc.r.kv - j0);
        const int np = (nk + PS - 1) >> a.shift;
        const int heads = keys ? HQ : a.H, hd = keys ? cc.h : cc.h / (HQ / a.H);
        mbar_expect_tx(full, np * (PS * KD * 2 + (keys ? KD * 4 : 0)));
        for (int y = 0; y < np; ++y) {
          const int slot = (j0 >> a.shift) + y;
          const int page = slot < a.MP ? page_of(a.table, (long)cc.r.i * a.MP, slot, a.NP) : -1;
          // none: read past the pool's end, where the copy gives zeros
          // (expected only of pages wholly before the window)
          if (page < 0 && j0 + ((y + 1) << a.shift) > max(0, s.pos0 - win + 1))
            record_status(a.status, WALL_ERR_INVALID_ARG);
          const int z = page >= 0 ? page * heads + hd : a.NP * heads;
          for (int bx = 0; bx < KD / 64; ++bx)
            tma_load_3d(dst + bx * (BN * 128) + y * PS * 128, tm, full, bx * 64, 0, z);
          if constexpr (keys)
            bulk_load(sbase + Lay::oR + (st * Lay::kRows + y) * KD * 4,
                      a.rp + ((long)max(page, 0) * HQ + cc.h) * KD, KD * 4, full);
        }
      };
      load_q();
      for (int g = 0; g < n_tiles + 2; ++g) {
        if (g >= 2 && tv == sv.ta && seg_v > 0) {
          if (!wait_bar(bar(B_QEMPTY), (seg_v - 1) & 1, a.status, abort_flag)) break;
          load_q();
        }
        if (g < n_tiles) {
          const int st = g % kKS;
          if (g >= kKS && !wait_bar(bar(B_KEMPTY + st), (g / kKS - 1) & 1, a.status, abort_flag))
            break;
          load_tile(std::true_type{}, c, sk, tk, st, bar(B_KFULL + st));
          ++k_out;
          if (++tk == sk.tb && g + 1 < n_tiles) {
            xk += sk.tb - sk.ta;
            next_unit<BM>(a.bt, a.window, HQ, pk, c);
            sk = segment_of(c, x1 - xk);
            tk = sk.ta;
          }
        }
        if (g >= 2) {
          const int gv = g - 2, st = gv % kVS;
          if (gv >= kVS && !wait_bar(bar(B_VEMPTY + st), (gv / kVS - 1) & 1, a.status, abort_flag))
            break;
          // a partly masked tile goes to the rescale warps first, which then
          // make the two arrivals on B_VFULL
          const bool part = !sees_all(sv, cv.r.dead, (sv.lo + tv) * BN, win);
          if (part) {
            raw |= 1u << st;
            raw_next ^= 1u << st;
          } else {
            raw &= ~(1u << st);
            mbar_arrive(bar(B_VFULL + st));
          }
          load_tile(std::false_type{}, cv, sv, tv, st, bar((part ? B_VRAW : B_VFULL) + st));
          ++v_out;
          if (++tv == sv.tb && gv + 1 < n_tiles) {
            xv += sv.tb - sv.ta;
            next_unit<BM>(a.bt, a.window, HQ, pk, cv);
            sv = segment_of(cv, x1 - xv);
            tv = sv.ta;
            ++seg_v;
          }
        }
      }
      // no copy may still be landing in this CTA's shared memory at exit
      for (int t = max(0, k_out - kKS); t < k_out; ++t)
        mbar_wait(bar(B_KFULL + t % kKS), (t / kKS) & 1, a.status);
      for (int t = max(0, v_out - kVS); t < v_out; ++t) {
        const int st = t % kVS;
        if ((raw >> st) & 1u) mbar_wait(bar(B_VRAW + st), ((raw_next >> st) & 1u) ^ 1u, a.status);
        else mbar_wait(bar(B_VFULL + st), (t / kVS) & 1, a.status);
      }
      mbar_wait(bar(B_QFULL), (q_out - 1) & 1, a.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      const uint32_t idesc_qk = idesc_bf16(BM, BN, false, false);
      const uint32_t idesc_pv = idesc_bf16(BM, V, false, true);
      // two walks over the CTA's tiles: S runs two tiles ahead of P V
      Cursor cq = c;
      long long xq = x0;
      Segment sq = segment_of(cq, x1 - xq);
      int seg_q = 0, tq = sq.ta;
      auto issue_qk = [&](int g) -> bool {
        if (tq == sq.tb) {  // the next unit's rows
          xq += sq.tb - sq.ta;
          next_unit<BM>(a.bt, a.window, HQ, pk, cq);
          sq = segment_of(cq, x1 - xq);
          tq = sq.ta;
          ++seg_q;
        }
        const int st = g % kKS;
        if (tq == sq.ta && !wait_bar(bar(B_QFULL), seg_q & 1, a.status, abort_flag)) return false;
        if (!wait_bar(bar(B_KREADY + st), (g / kKS) & 1, a.status, abort_flag)) return false;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (g & 1) * 128;
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          const uint64_t da = sdesc_sw128(sbase + Lay::oQ + off, 16, 1024);
          const uint64_t db = sdesc_sw128(sbase + Lay::oK + st * Lay::kT + off, 16, 1024);
          umma_bf16_ss(d_tmem, da, db, idesc_qk, kk > 0 ? 1u : 0u);
        }
        umma_commit(bar(B_SFULL + (g & 1)));
        umma_commit(bar(B_KEMPTY + st));
        if (++tq == sq.tb) umma_commit(bar(B_QEMPTY));
        return true;
      };
      bool ok = issue_qk(0);
      if (ok && n_tiles > 1) ok = issue_qk(1);
      int seg = 0;
      long long x = x0;
      Segment s = segment_of(c, x1 - x);
      int t = s.ta;
      uint32_t begun = 0;  // groups with a tile in this segment
      for (int g = 0; ok && g < n_tiles; ++g) {
        if (t == s.tb) {
          x += s.tb - s.ta;
          next_unit<BM>(a.bt, a.window, HQ, pk, c);
          s = segment_of(c, x1 - x);
          t = s.ta;
          ++seg;
          begun = 0;
        }
        const int grp = g & 1, vs = g % kVS;
        if (t == s.ta && seg > 0 &&
            !wait_bar(bar(B_OEMPTY), (seg - 1) & 1, a.status, abort_flag)) break;
        if (!wait_bar(bar(B_VFULL + vs), (g / kVS) & 1, a.status, abort_flag)) break;
        if (!wait_bar(bar(B_PFULL + grp), (g >> 1) & 1, a.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t keep = (begun >> grp) & 1u;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          // A = P [128 rows x 16 keys] from TMEM (bf16 pairs over the S columns)
          const uint32_t da = tmem + grp * 128 + kk * 8;
          // B = V [16 keys x V channels], MN-major
          const uint64_t db =
              sdesc_sw128(sbase + Lay::oV + vs * Lay::kT + kk * 16 * 128, BN * 128, 1024);
          umma_bf16_ts(tmem + 256 + grp * V, da, db, idesc_pv, keep | (kk > 0 ? 1u : 0u));
        }
        begun |= 1u << grp;
        umma_commit(bar(B_PVDONE + grp));
        umma_commit(bar(B_VEMPTY + vs));
        ++t;
        if (g + 2 < n_tiles) ok = issue_qk(g + 2);
      }
      // every MMA of this CTA has completed before TMEM is released
      umma_commit(bar(B_MMADONE));
      mbar_wait(bar(B_MMADONE), 0, a.status);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ key rescale
    constexpr int kChunks = KD / 8;          // 16-byte chunks per row
    constexpr int kRowStep = 64 / kChunks;   // rows covered by one pass of 64 threads
    const int tid = threadIdx.x - 64;
    const int ch = tid % kChunks;
    const int rs = tid / kChunks;
    int g = 0;
    uint32_t raw = 0;  // parity of each value stage's next partly masked tile
    bool ok = true;
    for (long long x = x0; ok && x < x1;) {
      const Segment s = segment_of(c, x1 - x);
      const int slot_i = s.pos0 >> a.shift;
      const int page_i = !c.r.dead && slot_i < a.MP
                             ? page_of(a.table, (long)c.r.i * a.MP, slot_i, a.NP) : -1;
      int ri[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        ri[e] = page_i >= 0 ? __ldg(a.rp + ((long)page_i * HQ + c.h) * KD + ch * 8 + e) : 0;
      const int seen_from = max(0, s.pos0 - win + 1);
      bool flag = false;
      for (int t = s.ta; t < s.tb; ++t, ++g) {
        const int st = g % kKS;
        {
          const bool got = wait_bar(bar(B_KFULL + st), (g / kKS) & 1, a.status, abort_flag);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        }
        const int j0 = (s.lo + t) * BN;
        const int nk = c.r.dead ? 0 : min(BN, c.r.kv - j0);
        const int np = (nk + PS - 1) >> a.shift;
        uint8_t* kt = smem + Lay::oK + st * Lay::kT + (ch / 8) * (BN * 128);
        for (int y = 0; y < np; ++y) {
          const int* rc = reinterpret_cast<const int*>(smem + Lay::oR) + (st * Lay::kRows + y) * KD + ch * 8;
          __nv_bfloat162 f[4];
          bool far = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int e0 = ri[2 * e] - rc[2 * e], e1 = ri[2 * e + 1] - rc[2 * e + 1];
            far |= max(e0, e1) > (int)kAnchorRange;
            const uint32_t b = pow2_bf16(e0) | (pow2_bf16(e1) << 16);
            f[e] = *reinterpret_cast<const __nv_bfloat162*>(&b);
          }
          // a page wholly before the window may be gone: nothing is seen of it
          flag |= far && j0 + ((y + 1) << a.shift) > seen_from && j0 + (y << a.shift) < s.pos0 + s.ni;
          constexpr int kBatch = 32 / kRowStep;  // a 32-row piece of a page
#pragma unroll 1
          for (int r0 = y << a.shift; r0 < ((y + 1) << a.shift); r0 += 32) {
            uint4 w[kBatch];
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
              const int r = r0 + rs + z * kRowStep;
              w[z] = *reinterpret_cast<const uint4*>(kt + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
              const int r = r0 + rs + z * kRowStep;
              __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w[z]);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], f[e]);
              *reinterpret_cast<uint4*>(kt + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = w[z];
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_KREADY + st));
        if (!sees_all(s, c.r.dead, j0, win)) {
          const int vs = g % kVS;
          const bool got = wait_bar(bar(B_VRAW + vs), (raw >> vs) & 1u, a.status, abort_flag);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          raw ^= 1u << vs;
          uint8_t* vt = smem + Lay::oV + vs * Lay::kT + (ch / 8) * (BN * 128);
          uint32_t bad = 0;
          for (int r = rs; r < BN; r += kRowStep) {
            uint4* w = reinterpret_cast<uint4*>(vt + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
            if (r >= nk) {
              *w = make_uint4(0u, 0u, 0u, 0u);
            } else {
              const uint4 y = *w;
              bad |= not_finite(y.x) | not_finite(y.y) | not_finite(y.z) | not_finite(y.w);
            }
          }
          flag |= bad != 0;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_VFULL + vs));
        }
      }
      if (flag) flags.set(c.r, c.b, c.h, HQ);
      x += s.tb - s.ta;
      if (ok && x < x1) next_unit<BM>(a.bt, a.window, HQ, pk, c);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int grp = (warp - 4) >> 2;          // 0: even tiles of the CTA, 1: odd ones
    const int quarter = warp & 3;             // TMEM lane quarter of this warp
    const int r = quarter * 32 + lane;        // query row within the unit
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + grp * 128;
    const uint32_t o_addr = tmem + lane_base + 256 + grp * V;
    const float sl2 = a.scale_log2;
    int g0 = 0, n_seg = 0;  // the CTA's tiles before the segment
    bool ok = true;
    Cursor& cur = s_cur[warp - 4];
    if (lane == 0) cur = c;
    __syncwarp();
    for (; ok && g0 < n_tiles; ++n_seg) {
      const Segment s = segment_of(cur, n_tiles - g0);
      const bool dead = cur.r.dead;
      const bool row_ok = r < s.ni;
      const int i = s.pos0 + r;               // the row's position
      // a unit of few rows leaves whole warps without one: they keep step only
      const bool idle = quarter * 32 >= s.ni;
      const int n_here = s.tb - s.ta;
      float m_use = -INFINITY, l = 0.f;
      const int first = (g0 + grp) & 1;       // this group's first tile of the segment
      for (int y = first; y < n_here; y += 2) {
        const int g = g0 + y;
        const int j0 = (s.lo + s.ta + y) * BN;
        {
          const bool got = wait_bar(bar(B_SFULL + grp), (g >> 1) & 1, a.status, abort_flag);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        }
        if (idle) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PFULL + grp));
          continue;
        }
        tc_fence_after();
        const bool fast = sees_all(s, dead, j0, win);  // the same for the whole CTA
        bool done = false;
        // One pass when every row's running max is set: exponentials against
        // it, kept in registers and stored only if no row's sum exceeds
        // 2^threshold (then no term does; an overflow or NaN fails the test
        // too); else the two passes below.
        if (fast && __all_sync(0xffffffffu, !row_ok || m_use != -INFINITY)) {
          uint32_t pk1[64];
          float r0 = 0.f, r1 = 0.f;
          const float off = -m_use;
#pragma unroll
          for (int cc = 0; cc < BN; cc += 64) {
            uint32_t sv[64];
            tmem_ld32(s_addr + cc, sv);
            tmem_ld32(s_addr + cc + 32, sv + 32);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const float p0 = exp2f(fmaf(__uint_as_float(sv[e]), sl2, off));
              const float p1 = exp2f(fmaf(__uint_as_float(sv[e + 1]), sl2, off));
              const float p2 = exp2f(fmaf(__uint_as_float(sv[e + 2]), sl2, off));
              const float p3 = exp2f(fmaf(__uint_as_float(sv[e + 3]), sl2, off));
              r0 += p0 + p2;
              r1 += p1 + p3;
              pk1[(cc + e) / 2] = pack_bf16x2(p0, p1);
              pk1[(cc + e) / 2 + 1] = pack_bf16x2(p2, p3);
            }
          }
          if (!__any_sync(0xffffffffu, row_ok && !(r0 + r1 <= kRescaleBound))) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_st16(s_addr + cc * 16, pk1 + cc * 16);
            tmem_wait_st();
            l += r0 + r1;
            done = true;
          }
        }
        if (!done) {
          // pass 1: row max
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
          // the row's visible keys of the tile: [ja, jb)
          const int jb = row_ok && !dead ? min(BN, i + 1 - j0) : 0;
          const int ja = max(0, i - win + 1 - j0);
#pragma unroll 1
          for (int cc = 0; cc < BN; cc += 64) {
            uint32_t sv[64];
            tmem_ld32(s_addr + cc, sv);
            tmem_ld32(s_addr + cc + 32, sv + 32);
            tmem_wait_ld();
            if (fast) {
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                mx0 = fmaxf(mx0, __uint_as_float(sv[e]) * sl2);
                mx1 = fmaxf(mx1, __uint_as_float(sv[e + 1]) * sl2);
                mx2 = fmaxf(mx2, __uint_as_float(sv[e + 2]) * sl2);
                mx3 = fmaxf(mx3, __uint_as_float(sv[e + 3]) * sl2);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const bool vis = cc + e >= ja && cc + e < jb;
                mx0 = fmaxf(mx0, vis ? __uint_as_float(sv[e]) * sl2 : -INFINITY);
              }
            }
          }
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
          const bool resc = mx > m_use + kRescaleThreshold;
          const float m_new = resc ? mx : m_use;
          const float alpha = m_use == -INFINITY ? 0.f : exp2f(m_use - m_new);
          if (y > first) {
            // this group's previous P V has landed in its O before O is rescaled
            const bool got = wait_bar(bar(B_PVDONE + grp), ((g >> 1) - 1) & 1, a.status, abort_flag);
            if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
            tc_fence_after();
            if (__any_sync(0xffffffffu, resc)) {
              const float f = resc ? alpha : 1.f;
#pragma unroll 1
              for (int cc = 0; cc < V / 32; ++cc) {
                uint32_t ov[32];
                tmem_ld32(o_addr + cc * 32, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                tmem_st32(o_addr + cc * 32, ov);
              }
              tmem_wait_st();
            }
          }
          if (resc) l *= alpha;
          m_use = m_new;
          const float m_eff = m_use == -INFINITY ? 0.f : m_use;
          // pass 2: p = exp2(s - m), row sum, bf16 P over the consumed S columns
          float rs0 = 0.f, rs1 = 0.f;
#pragma unroll 1
          for (int cc = 0; cc < BN; cc += 32) {
            uint32_t sv[32];
            tmem_ld32(s_addr + cc, sv);
            tmem_wait_ld();
            float e32[32];
            if (fast) {
#pragma unroll
              for (int e = 0; e < 32; ++e) e32[e] = exp2f(fmaf(__uint_as_float(sv[e]), sl2, -m_eff));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const bool vis = cc + e >= ja && cc + e < jb;
                e32[e] = vis ? exp2f(fmaf(__uint_as_float(sv[e]), sl2, -m_eff)) : 0.f;
              }
            }
            uint32_t pk2[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              rs0 += e32[e];
              rs1 += e32[e + 1];
              pk2[e / 2] = pack_bf16x2(e32[e], e32[e + 1]);
            }
            tmem_st16(s_addr + cc / 2, pk2);
          }
          tmem_wait_st();
          l += rs0 + rs1;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + grp));
      }
      // ---- the unit's end, or the share's: merge the groups' (m, l, O)
      const int mine = (n_here - first + 1) >> 1;          // this group's tiles
      const int theirs = n_here - mine;
      if (ok && mine > 0) {
        const int g_last = g0 + first + 2 * (mine - 1);
        ok = __all_sync(0xffffffffu, wait_bar(bar(B_PVDONE + grp), (g_last >> 1) & 1, a.status,
                                              abort_flag));
      }
      float* xm = sX + (n_seg & 1) * (2 * 2 * BM);
      xm[(grp * 2) * BM + r] = m_use;
      xm[(grp * 2 + 1) * BM + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_XCHG));
      if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(B_XCHG), n_seg & 1, a.status, abort_flag));
      if (ok) {
        tc_fence_after();
        const float m0 = xm[0 * BM + r], l0 = xm[1 * BM + r];
        const float m1 = xm[2 * BM + r], l1 = xm[3 * BM + r];
        const bool has0 = grp == 0 ? mine > 0 : theirs > 0, has1 = grp == 0 ? theirs > 0 : mine > 0;
        const bool whole = s.ta == 0 && s.tb == cur.n_tiles;
        float m_f = fmaxf(m0, m1);
        if (whole && a.sink) m_f = fmaxf(m_f, a.sink[cur.h] * kLog2e);
        const float a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - m_f);
        const float a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - m_f);
        float lt = l0 * a0 + l1 * a1;
        float inv = 1.f;
        if (whole) {
          if (a.sink) lt += exp2f(a.sink[cur.h] * kLog2e - m_f);
          inv = lt > 0.f || lt != lt ? 1.f / lt : 0.f;  // a row that sees nothing: 0
        }
        const float f0 = a0 * inv, f1 = a1 * inv;
        const int slot = s.ta == 0 ? 1 : 0;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.o) + ((long)(s.t0 + r) * HQ + cur.h) * V;
        float* prow = parts.o(cta, slot, V) + (size_t)r * V;
        // each group writes half of the channels
        if (!idle) {
#pragma unroll 1
          for (int cc = grp * (V / 2); cc < (grp + 1) * (V / 2); cc += 32) {
            uint32_t ov0[32], ov1[32];
            if (has0) tmem_ld32(tmem + lane_base + 256 + cc, ov0);
            if (has1) tmem_ld32(tmem + lane_base + 256 + V + cc, ov1);
            tmem_wait_ld();
            float o32[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              // (a row whose weight is 0 had no key in the group: its O is 0)
              float v = has0 ? __uint_as_float(ov0[e]) * f0 : 0.f;
              if (has1) v = fmaf(__uint_as_float(ov1[e]), f1, v);
              o32[e] = v;
            }
            if (row_ok) {
              if (whole) {
                uint4* dst = reinterpret_cast<uint4*>(orow + cc);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  dst[e] = make_uint4(pack_bf16x2(o32[8 * e], o32[8 * e + 1]),
                                      pack_bf16x2(o32[8 * e + 2], o32[8 * e + 3]),
                                      pack_bf16x2(o32[8 * e + 4], o32[8 * e + 5]),
                                      pack_bf16x2(o32[8 * e + 6], o32[8 * e + 7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(prow + cc);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  dst[e] = make_float4(o32[4 * e], o32[4 * e + 1], o32[4 * e + 2], o32[4 * e + 3]);
              }
            }
          }
          tc_fence_before();
        }
        if (grp == 0 && row_ok) {
          if (whole) {
            if (a.lse)
              a.lse[(long)(s.t0 + r) * HQ + cur.h] = lt == 0.f ? -INFINITY : (m_f + log2f(lt)) * kLn2;
          } else {
            float* pm = parts.ml(cta, slot, V) + r * 2;
            pm[0] = m_f;
            pm[1] = lt;
          }
        }
        if (!whole && slot == 1 && warp == 4 && lane == 0) {
          PartDesc d;
          d.req = cur.r.i; d.h = cur.h; d.b = cur.b;
          d.last_cta = sh.owner(sh.begin(cta) + g0 + cur.n_tiles - 1);
          parts.desc[cta] = d;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_OEMPTY));
      g0 += n_here;
      if (ok && g0 < n_tiles) {
        Cursor nx = cur;
        next_unit<BM>(a.bt, a.window, HQ, pk, nx);
        __syncwarp();
        if (lane == 0) cur = nx;
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Qh = q * 2^(p + R_{page(i)} - R_I): rows of requests of two or more, a CTA a
// row at a time, eight channels a thread.  An exponent past +-kAnchorRange
// flags the row's unit.
__global__ void __launch_bounds__(256) chunk_queries_kernel(AttnArgs a, __nv_bfloat16* qh,
                                                            UnitFlags flags) {
  const int per_row = a.HQ * a.K / 8;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
  for (int t = blockIdx.x; t < a.bt.T; t += gridDim.x) {
    int lo = 0, hi = a.bt.N - 1;  // the last request that begins at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.bt.cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const Request r = request_of<BM>(a.bt, lo, a.window);
    if (t < r.t0 || t >= r.t0 + r.n || r.n < 2 || r.dead) continue;
    const int b = (t - r.t0) / BM;
    const int slot = (r.ctx + t - r.t0) >> a.shift, slot_i = (r.ctx + b * BM) >> a.shift;
    const long trow = (long)lo * a.MP;
    const int page = slot < a.MP ? page_of(a.table, trow, slot, a.NP) : -1;
    const int page_i = slot_i < a.MP ? page_of(a.table, trow, slot_i, a.NP) : -1;
    for (int x = threadIdx.x; x < per_row; x += blockDim.x) {
      const int off = x * 8;  // head and channel
      float qv[8], pv[8];
      load8(q + (long)t * a.HQ * a.K + off, qv);
      load8(a.p + (long)t * a.HQ * a.K + off, pv);
      if (page >= 0 && page_i >= 0 && page != page_i) {
        const int4* ra = reinterpret_cast<const int4*>(a.rp + (long)page * a.HQ * a.K + off);
        const int4* rb = reinterpret_cast<const int4*>(a.rp + (long)page_i * a.HQ * a.K + off);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int4 u = ra[e], w = rb[e];
          pv[4 * e] += (float)(u.x - w.x);
          pv[4 * e + 1] += (float)(u.y - w.y);
          pv[4 * e + 2] += (float)(u.z - w.z);
          pv[4 * e + 3] += (float)(u.w - w.w);
        }
      }
      bool wide = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        wide |= fabsf(pv[e]) > kAnchorRange;
        qv[e] *= exp2f(pv[e]);
      }
      if (wide) flags.set(r, b, off / a.K, a.HQ);
      store8(qh + (long)t * a.HQ * a.K + off, qv);
    }
  }
}

template <int KD>
int launch(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, __nv_bfloat16* qh,
           cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const int PS = 1 << a.shift;
  if (!make_tile_map(&tq, qh, a.bt.T, a.HQ, KD, BM) ||
      !make_page_map(&tk, a.kp, (long)a.NP * a.HQ, PS, KD, PS, 1) ||
      !make_page_map(&tv, a.vp, (long)a.NP * a.H, PS, KD, PS, 1))
    return WALL_ERR_CUDA;
  static bool attr[kMaxDevices] = {};
  if (!set_max_smem_once(paged_chunk_kernel<KD>, Smem<KD>::kAlloc, attr)) return WALL_ERR_CUDA;
  paged_chunk_kernel<KD><<<parts.n_cta, kThreads, Smem<KD>::kAlloc, stream>>>(tq, tk, tv, a, parts,
                                                                             flags);
  return cudaGetLastError() == cudaSuccess ? WALL_OK : WALL_ERR_CUDA;
}

}  // namespace

namespace paged {

bool chunk_rows_supported(int dtype, int K, int V) {
  return dtype == WALL_BF16 && K == V && (K == 64 || K == 128);
}

int chunk_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, void* qh,
               cudaStream_t stream) {
  if (cudaMemsetAsync(flags.f, 0, sizeof(int) * flags.count(a.bt.N, a.bt.T, a.HQ), stream) !=
      cudaSuccess)
    return WALL_ERR_CUDA;
  __nv_bfloat16* q16 = static_cast<__nv_bfloat16*>(qh);
  const int blocks = a.bt.T < kSms * 8 ? a.bt.T : kSms * 8;
  chunk_queries_kernel<<<blocks, 256, 0, stream>>>(a, q16, flags);
  if (cudaGetLastError() != cudaSuccess) return WALL_ERR_CUDA;
  return a.K == 128 ? launch<128>(a, parts, flags, q16, stream)
                    : launch<64>(a, parts, flags, q16, stream);
}

}  // namespace paged
}  // namespace wall
