// wall_paged_chunk_sm100.cu -- rows of requests with two or more new tokens
// over the paged Wall cache, on the tensor cores (tcgen05 + TMEM + TMA; bf16,
// K == V in {64, 128}): prompts, chunks of prompts, long drafts.
//
// Math.  A unit is 128 query rows of one (request, head).  With R_I the anchor
// of the page that holds its first row,
//   Qh_i = q_i 2^(p_i + R_{page(i)} - R_I)       (a small kernel before this one)
//   s_ij = scale sum_n Qh_in (k_jn 2^(R_I,n - R_{page(j),n}))
// where k_j is the cached row.  The anchors are whole numbers, so scaling the
// key tile is exact: Qh is the only operand that is rounded (to bf16, half a
// step of 2^-8, as a tensor-core operand has to be).  P is rounded to bf16
// for P V; its sum is taken in fp32 before that.  A unit whose exponents
// p_i + R_{page(i)} - R_I pass +-100 on some channel, or whose R_I - R_{page(j)}
// passes +100, or whose result is not finite (a value that is not reaches the
// rows that do not see it as 0 * inf; sums taken before a row's reference is
// raised may pass fp32), is flagged, and the general kernel computes it again,
// exactly, behind this one.
//
// Work.  One CTA per SM takes an even share of the batch's (unit, 128-key
// tile) pairs in order (wall_paged.cuh): the tile pipeline's rings and
// barriers run on across the units, a prompt's short first blocks and long
// last ones balance to within a tile, and a few rows over a long context
// spread over all SMs and are joined afterwards.
//
// Measured: an 8192-token prompt of 16 heads in 399 us with the queries' pass and
// the join, 689 TFLOP/s of its visible pairs (42 % of the dense bf16 rate).  A tile takes 2600 cycles where
// its MMAs are worth 1024 and its operands, copies and rescale hold the shared
// memory for 1800: the thread that issues the MMAs waits for S's keys, P and V
// in turn, and what it has issued runs out meanwhile.  Units of a few tiles
// (windows) pay for their start and end: 69 us for 23 GFLOP.
//
// 12 warps (3 per SM sub-partition, 168 registers each):
//   warp 0      walks the share's units, lays each one's figures into a ring in
//               shared memory for the other roles, and issues all TMA copies:
//               the key ring (3 stages, with the pages' anchors), the value
//               ring (2 stages), the units' Qh
//   warp 1      TMEM owner and MMA issuer (one thread)
//   warps 2-3   key rescale in place; zeros in place of the value rows past a
//               request's last key (pages end inside tiles; what they hold
//               there is an earlier request's, or nothing)
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
constexpr float kRaiseAbove = 256.f;      // a tile's sum of P that raises the row's reference
constexpr float kFlagAbove = 1.2676506e30f;  // 2^100: one that may not be held
// A key's factor 2^(R_I - R_page) below 2^-126 is no bf16 number.  A key row holds
// up to 2^100 |k|, so as long as the unit's Qh have exponents of at most kRise
// (gates <= 0 leave 1/2, an anchor's rounding), what such a factor leaves of a
// product is below 2^(kRise + 100 - 127) |q k| and counts as 0.  In a unit whose
// rows rise further the factor is applied in two steps instead.
constexpr float kRise = 1.f;
// A unit's own cost, in tiles.  An 8192-token prompt, windowed chunks and a mixed
// step take 399, 92.0 and 129.6 us; with 2: 406, 92.1, 130.4; with 4: 404, 91.6,
// 129.1; with 6: 413, 91.9, 127.7.
constexpr int kUnit = 3;

// The walk over the units as calls: it runs once a unit or less, and the code of
// this kernel's roles has to stay within what the instruction cache holds (at
// 122 KB of it every role ran a third slower than at 83 KB).
__device__ __noinline__ bool start_share(const Batch& bt, int window, int heads, int n_min, int cta, int n_cta,
                                         FindScratch& fs, Share& sh, long long& x0, long long& x1) {
  if (!find_start<BM, kUnit>(bt, window, heads, {n_min, 0x7fffffff}, kUnit + 2, cta, n_cta, fs, sh))
    return false;
  x0 = sh.begin(cta);
  x1 = sh.begin(cta + 1);
  return true;
}
__device__ __noinline__ void start_cursor(const Batch& bt, int window, const FindScratch& fs,
                                          long long x, Cursor& c) {
  c = cursor_at<BM, kUnit>(bt, window, fs.req, fs.base, x);
}
__device__ __noinline__ void advance(const Batch& bt, int window, int heads, int n_min, Cursor& c) {
  next_unit<BM>(bt, window, heads, {n_min, 0x7fffffff}, c);
}
__device__ __noinline__ int ending_cta(const Share& sh, const Cursor& c, long long x) {
  return sh.last_owner<kUnit>(c, x);
}

// A CTA's piece of one unit, as every role reads it.
struct Segment {
  int t0, ni;       // first query row among the packed ones, rows
  int pos0;         // position of the first row (far below 0 where the request sees nothing)
  int j0;           // first key of its first tile
  int cnt;          // tiles (0: the CTA's share has ended)
  int fa, fb;       // tiles [fa, fb) are seen whole by every row
  int kv;           // keys of the request (0 where it sees nothing)
  int from;         // first key that any row sees
  int h;
  int req;
  int page_i;       // the page whose anchor the unit's queries are taken against, or -1
  int place;        // of its flag
  int whole;        // the unit lies in this CTA alone
  int slot;         // else its part's slot
  int pad;
};
static_assert(sizeof(Segment) == 64, "four 16-byte words");
// Segments in flight: warp 0 writes the entry of segment s + 8 when its first
// key tile g is issued, behind S(g - 3), hence behind PV(g - 5), whose segment
// is s + 3 at least and began behind the epilogue of s + 2.
constexpr int kSegs = 8;

template <int KD>
struct Smem {
  static constexpr int kT = BN * KD * 2;           // one 128-row bf16 tile
  static constexpr int kRows = BN / 32;            // most pages of a tile
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + kT;               // kKS stages
  static constexpr int oV = oK + kKS * kT;         // kVS stages
  static constexpr int oR = oV + kVS * kT;         // int[kKS][kRows][KD] anchors
  static constexpr int oX = oR + kKS * kRows * KD * 4;  // float[2][2 groups][2][BM]: m, l
  static constexpr int oSeg = oX + 2 * 2 * 2 * BM * 4;  // Segment[kSegs]
  static constexpr int oBar = oSeg + kSegs * 64;
  static constexpr int kBars = 26 + kSegs;
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
  B_VRAW = B_VEMPTY + kVS,      // + value stage: a tile that the keys end in has landed
  B_SFULL = B_VRAW + kVS,       // + S buffer (2)
  B_PFULL = B_SFULL + 2,        // + group (2), 4 warps each
  B_PVDONE = B_PFULL + 2,       // + group (2)
  B_XCHG = B_PVDONE + 2,        // exchange of m, l between the groups (8 warps)
  B_OEMPTY,                     // both O accumulators read (8 warps)
  B_MMADONE,
  B_SEG,                        // + ring entry: a segment's figures are there
  kNumBars = B_SEG + kSegs,
};
static_assert(kNumBars <= Smem<128>::kBars, "barrier slots");

// Bounded wait that also gives up once another role has given up.  The wait
// itself is a call: inlined at each of its two dozen places it was a fifth of
// the kernel's code.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, int* status,
                                     volatile int* abort_flag) {
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
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, int* status,
                                         volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, status, abort_flag);
}
// the same for a copy that has to land before the CTA may end
__device__ __noinline__ void drain(uint32_t bar, uint32_t parity, int* status) {
  mbar_wait(bar, parity, status);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 2^e as bf16 bits: exact in the normal range, 0 below it, +inf above
__device__ __forceinline__ uint32_t pow2_bf16(int e) {
  return uint32_t(min(max(e + 127, 0), 255)) << 7;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Low word of a 128-byte-swizzle shared-memory descriptor (see sdesc_sw128);
// the high word is the same for all of this kernel's: stride 1024 between
// 8-row groups, version, swizzle mode.
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t keep) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(keep), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t keep) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(keep), "r"(kDescHi));
}

// Zeros in place of a value tile's rows from nk on, by the 64 threads of the
// rescale warps.
template <int KD>
__device__ __noinline__ void clear_rows(uint8_t* tile, int nk) {
  constexpr int kChunks = KD / 8, kRowStep = 64 / kChunks;
  const int tid = threadIdx.x - 64, ch = tid % kChunks;
  uint8_t* vt = tile + (ch / 8) * (BN * 128);
#pragma unroll 4
  for (int r = nk + tid / kChunks; r < BN; r += kRowStep)
    *reinterpret_cast<uint4*>(vt + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// The second step of a key tile's factors 2^(R_I - R_page) below 2^kLowest, on
// this thread's 16-byte chunk of channels: ri their R_I, rc the tile's pages'.
constexpr int kLowest = -126;
template <int KD>
__device__ __noinline__ void scale_again(uint8_t* tile, const int* rc, int4 ri0, int4 ri1, int shift) {
  constexpr int kChunks = KD / 8, kRowStep = 64 / kChunks;
  const int tid = threadIdx.x - 64, ch = tid % kChunks;
  uint8_t* kt = tile + (ch / 8) * (BN * 128);
  auto factor = [](int lo, int hi) {
    return pow2_bf16(min(lo - kLowest, 0)) | (pow2_bf16(min(hi - kLowest, 0)) << 16);
  };
  for (int r = tid / kChunks; r < BN; r += kRowStep) {
    const int4* c = reinterpret_cast<const int4*>(rc + (r >> shift) * KD + ch * 8);
    uint4* x = reinterpret_cast<uint4*>(kt + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
    const uint4 w = *x;
    *x = make_uint4(mul_bf16x2(w.x, factor(ri0.x - c[0].x, ri0.y - c[0].y)),
                    mul_bf16x2(w.y, factor(ri0.z - c[0].z, ri0.w - c[0].w)),
                    mul_bf16x2(w.z, factor(ri1.x - c[1].x, ri1.y - c[1].y)),
                    mul_bf16x2(w.w, factor(ri1.z - c[1].z, ri1.w - c[1].w)));
  }
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
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* sX = reinterpret_cast<float*>(smem + Lay::oX);
  Segment* segs = reinterpret_cast<Segment*>(smem + Lay::oSeg);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::oBar);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::oMisc + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;

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
    for (int s = 0; s < kSegs; ++s) mbar_init(bar(B_SEG + s), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  start_next();
  Share sh;
  long long x0, x1;
  if (!start_share(a.bt, a.window, a.HQ, a.n_min, cta, parts.n_cta, fs, sh, x0, x1)) {
    wait_before();
    return;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  wait_before();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA
    // Copies go out in the order in which the MMAs free their places: S(0)
    // S(1) PV(0) S(2) PV(1) S(3) ... complete in that order, so key tile g
    // (behind S(g - 3)), then value tile g - 2 (behind PV(g - 4)) never waits
    // past a copy that could go.  A unit's Qh goes out once the last S of the
    // unit before has read its rows, two tiles into the unit.  The lanes hold
    // the next 32 entries of the block table and issue a tile's boxes side by
    // side.
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_q);
    }
    constexpr int kBoxes = KD / 64;
    const int win = a.window > 0 ? a.window : 0x7fffffff;
    const int PS = 1 << a.shift;
    // 32 entries of a request's table row from `slot` on
    auto table_at = [&](int req, int slot) {
      return slot + lane < a.MP ? page_of(a.table, (long)req * a.MP, slot + lane, a.NP) : -1;
    };
    long long x = x0;
    Cursor c;
    start_cursor(a.bt, a.window, fs, x, c);
    int slot_k = 0, ids_k = 0, seg_k = -1;
    // the figures of the next unit that this CTA has tiles of, into the ring;
    // returns their number, 0 at the share's end
    auto open_segment = [&]() {
      Segment s;
      s.cnt = 0;
      while (x < x1) {
        const Run run = run_of<kUnit>(c, x1 - x);
        if (run.tb > run.ta) {
          s.t0 = c.r.t0 + c.b * BM;
          s.ni = min(BM, c.r.n - c.b * BM);
          s.pos0 = c.r.dead ? -(1 << 29) : c.r.ctx + c.b * BM;
          s.j0 = (tile_lo(c.r, c.b) + run.ta) * BN;
          s.cnt = run.tb - run.ta;
          // seen whole: the first row sees its last key, the last row its first
          s.fa = c.r.dead ? 0 : max(0, (max(s.pos0 + s.ni - win, 0) - s.j0 + BN - 1) >> 7);
          s.fb = c.r.dead ? 0 : max(0, (s.pos0 + 1 - s.j0) >> 7);
          s.kv = c.r.dead ? 0 : c.r.kv;
          s.from = c.r.dead ? 0 : max(0, s.pos0 - win + 1);
          s.h = c.h;
          s.req = c.r.i;
          slot_k = s.j0 >> a.shift;
          ids_k = c.r.dead ? -1 : table_at(s.req, slot_k);
          const int slot_i = s.pos0 >> a.shift;  // (one entry, the same for every lane)
          s.page_i = !c.r.dead && slot_i < a.MP
                         ? page_of(a.table, (long)s.req * a.MP, slot_i, a.NP) : -1;
          s.place = (int)flags.place(c.r, c.b);
          s.whole = run.ta == 0 && run.tb == c.n_tiles;
          s.slot = run.ta == 0 ? 1 : 0;
          if (lane == 0 && run.ta == 0 && !s.whole) {
            PartDesc d;
            d.t0 = c.r.t0 + c.b * BM; d.rows = min(BM, c.r.n - c.b * BM); d.h = s.h;
            d.last_cta = ending_cta(sh, c, x);
            parts.desc[cta] = d;
          }
        }
        x += run.places;
        if (x < x1) advance(a.bt, a.window, a.HQ, a.n_min, c);
        if (s.cnt > 0) break;
      }
      ++seg_k;
      if (lane == 0) {
        if (s.cnt > 0) segs[seg_k % kSegs] = s;
        else segs[seg_k % kSegs].cnt = 0;
        mbar_arrive(bar(B_SEG + seg_k % kSegs));
      }
      __syncwarp();
      return s.cnt;
    };
    // the pages that hold the keys from j0 on into a stage of a ring
    auto load_tile = [&](auto keys_tag, const Segment& s, int j0, int st, uint32_t full, int& slot0,
                         int& ids) {
      constexpr bool keys = decltype(keys_tag)::value;
      const CUtensorMap* tm = keys ? &tm_k : &tm_v;
      const uint32_t dst = sbase + (keys ? Lay::oK : Lay::oV) + st * Lay::kT;
      const int np = (max(0, min(BN, s.kv - j0)) + PS - 1) >> a.shift;
      const int slot = j0 >> a.shift;
      if (slot + (BN >> a.shift) > slot0 + 32) {
        slot0 = slot;
        ids = table_at(s.req, slot);
      }
      if (lane == 0) mbar_expect_tx(full, np * (PS * KD * 2 + (keys ? KD * 4 : 0)));
      const int y = lane / kBoxes, bx = lane % kBoxes;  // page of the tile, box of the page
      const int page = __shfl_sync(0xffffffffu, ids, slot - slot0 + y);
      if (y < np) {
        const int heads = keys ? a.HQ : a.H, hd = keys ? s.h : s.h / (a.HQ / a.H);
        // none: read past the pool's end, where the copy gives zeros (expected
        // only of pages wholly before the window)
        if (page < 0 && j0 + ((y + 1) << a.shift) > s.from)
          record_status(a.status, WALL_ERR_INVALID_ARG);
        tma_load_3d(dst + bx * (BN * 128) + y * PS * 128, tm, full, bx * 64, 0,
                    page >= 0 ? page * heads + hd : a.NP * heads);
        if (keys && bx == 0)
          bulk_load(sbase + Lay::oR + (st * Lay::kRows + y) * KD * 4,
                    a.rp + ((long)max(page, 0) * a.HQ + s.h) * KD, KD * 4, full);
      }
      __syncwarp();
    };
    auto waits = [&](int b, int parity) {
      return __all_sync(0xffffffffu, wait_bar(bar(b), parity & 1, a.status, abort_flag));
    };
    int left_k = 0, y_k = 0;            // key tiles left in the walker's segment; the next one
    int left_v = 0, y_v = 0, seg_v = -1;
    int slot_v = 0, ids_v = 0;
    int k_out = 0, v_out = 0, q_out = 0;
    uint32_t raw = 0, raw_next = 0;     // per value stage: the keys end in its last tile;
                                        // parity of the next one's B_VRAW phase
    bool more = true;                   // key tiles
    for (int g = 0;; ++g) {
      if (g >= 2 && left_v == 0) {      // value tile g - 2 opens a segment: its queries
        const Segment& s = segs[++seg_v % kSegs];
        left_v = s.cnt;
        if (left_v == 0) break;
        y_v = 0;
        slot_v = s.j0 >> a.shift;
        ids_v = s.kv > 0 ? table_at(s.req, slot_v) : -1;
        if (seg_v > 0 && !waits(B_QEMPTY, seg_v - 1)) break;
        if (lane == 0) mbar_expect_tx(bar(B_QFULL), Lay::kT);
        __syncwarp();
        if (lane < kBoxes)
          tma_load_3d(sbase + Lay::oQ + lane * (BM * 128), &tm_q, bar(B_QFULL), lane * 64, s.h, s.t0);
        ++q_out;
      }
      if (more) {
        if (left_k == 0) {
          left_k = open_segment();
          y_k = 0;
          more = left_k > 0;
        }
        if (more) {
          const int st = g % kKS;
          if (g >= kKS && !waits(B_KEMPTY + st, g / kKS - 1)) break;
          const Segment& s = segs[seg_k % kSegs];
          load_tile(std::true_type{}, s, s.j0 + y_k * BN, st, bar(B_KFULL + st), slot_k, ids_k);
          ++k_out;
          ++y_k;
          --left_k;
        }
      }
      if (g >= 2) {
        const int st = (g - 2) % kVS;
        if (g - 2 >= kVS && !waits(B_VEMPTY + st, (g - 2) / kVS - 1)) break;
        const Segment& s = segs[seg_v % kSegs];
        // a tile that the request's last key ends in goes to the rescale warps
        // first, which then make the two arrivals on B_VFULL
        const bool part = s.kv - (s.j0 + y_v * BN) < BN;
        if (part) {
          raw |= 1u << st;
          raw_next ^= 1u << st;
        } else {
          raw &= ~(1u << st);
          if (lane == 0) mbar_arrive(bar(B_VFULL + st));
        }
        load_tile(std::false_type{}, s, s.j0 + y_v * BN, st, bar((part ? B_VRAW : B_VFULL) + st),
                  slot_v, ids_v);
        ++v_out;
        ++y_v;
        --left_v;
      }
    }
    // no copy may still be landing in this CTA's shared memory at exit
    for (int t = max(0, k_out - kKS); t < k_out; ++t)
      drain(bar(B_KFULL + t % kKS), (t / kKS) & 1, a.status);
    for (int t = max(0, v_out - kVS); t < v_out; ++t) {
      const int st = t % kVS;
      if ((raw >> st) & 1u) drain(bar(B_VRAW + st), ((raw_next >> st) & 1u) ^ 1u, a.status);
      else drain(bar(B_VFULL + st), (t / kVS) & 1, a.status);
    }
    if (q_out > 0) drain(bar(B_QFULL), (q_out - 1) & 1, a.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(BM, V, false, true);
      // the descriptors' low words; what varies is the address
      const uint32_t q_lo = sdesc_lo(sbase + Lay::oQ, 16);
      const uint32_t k_lo = sdesc_lo(sbase + Lay::oK, 16);
      const uint32_t v_lo = sdesc_lo(sbase + Lay::oV, BN * 128);
      // S runs two tiles ahead of P V, each with its own count of segments and
      // tiles; left_*: tiles of the segment still to be issued
      int seg_q = -1, left_q = 0, seg_p = -1, left_p = 0;
      int gq = 0, st_q = 0;
      uint32_t par_k = 0;
      bool ok = true, more = true;  // key tiles
      auto open = [&](int& seg, int& left) {
        ++seg;
        ok = wait_bar(bar(B_SEG + seg % kSegs), (seg / kSegs) & 1, a.status, abort_flag);
        left = ok ? *reinterpret_cast<volatile int*>(&segs[seg % kSegs].cnt) : 0;
        return left > 0;
      };
      // S of the next key tile
      auto issue_qk = [&]() {
        if (left_q == 0) {  // the next unit's rows
          more = open(seg_q, left_q);
          if (!more) return;
          ok = wait_bar(bar(B_QFULL), seg_q & 1, a.status, abort_flag);
          if (!ok) return;
        }
        ok = wait_bar(bar(B_KREADY + st_q), par_k, a.status, abort_flag);
        if (!ok) return;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (gq & 1) * 128;
        const uint32_t kb = k_lo + st_q * (Lay::kT >> 4);
#pragma unroll 2
        for (int kk = 0; kk < KD / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
          mma_ss(d_tmem, q_lo + off, kb + off, idesc_qk, kk > 0 ? 1u : 0u);
        }
        umma_commit(bar(B_SFULL + (gq & 1)));
        umma_commit(bar(B_KEMPTY + st_q));
        if (--left_q == 0) umma_commit(bar(B_QEMPTY));
        ++gq;
        if (++st_q == kKS) {
          st_q = 0;
          par_k ^= 1;
        }
      };
      uint32_t begun = 0;  // groups with a tile in this segment
      for (int g = 0; ok; ++g) {
        // Two S in flight (S(g + 2) takes the place of P(g)).  Where the next
        // one opens a unit, its Qh may still be on its way: the last P V of
        // this unit goes first.
#pragma unroll 1
        while (ok && more && gq < g + 2 && !(left_q == 0 && gq == g + 1)) issue_qk();
        if (!ok || g >= gq) break;
        const int grp = g & 1, vs = g & (kVS - 1);
        if (left_p == 0) {
          if (!open(seg_p, left_p)) break;
          begun = 0;
          if (seg_p > 0 && !wait_bar(bar(B_OEMPTY), (seg_p - 1) & 1, a.status, abort_flag)) break;
        }
        if (!wait_bar(bar(B_VFULL + vs), (g / kVS) & 1, a.status, abort_flag)) break;
        if (!wait_bar(bar(B_PFULL + grp), (g >> 1) & 1, a.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t keep = (begun >> grp) & 1u;
        const uint32_t vb = v_lo + vs * (Lay::kT >> 4);
#pragma unroll 2
        for (int kk = 0; kk < BN / 16; ++kk)
          // A = P [128 rows x 16 keys] from TMEM (bf16 pairs over the S columns),
          // B = V [16 keys x V channels], MN-major
          mma_ts(tmem + 256 + grp * V, tmem + grp * 128 + kk * 8, vb + (kk * 16 * 128 >> 4), idesc_pv,
                 kk > 0 ? 1u : keep);
        begun |= 1u << grp;
        umma_commit(bar(B_PVDONE + grp));
        umma_commit(bar(B_VEMPTY + vs));
        --left_p;
      }
      // every MMA of this CTA has completed before TMEM is released
      umma_commit(bar(B_MMADONE));
      mbar_wait(bar(B_MMADONE), 0, a.status);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ key rescale
    constexpr int kChunks = KD / 8;          // 16-byte chunks per row
    constexpr int kRowStep = 64 / kChunks;   // rows covered by one pass of 64 threads
    constexpr int kBatch = 32 / kRowStep;    // rows a thread has of 32
    const int tid = threadIdx.x - 64;
    const int ch = tid % kChunks;
    const int rs = tid / kChunks;
    const int PS = 1 << a.shift;
    uint32_t raw = 0;  // parity of each value stage's next B_VRAW phase
    int g = 0;
    bool ok = true;
    auto end_values = [&](int gv, int nk) {
      const int vs = gv % kVS;
      if (!__all_sync(0xffffffffu, wait_bar(bar(B_VRAW + vs), (raw >> vs) & 1u, a.status, abort_flag)))
        return false;
      raw ^= 1u << vs;
      clear_rows<KD>(smem + Lay::oV + vs * Lay::kT, nk);
      if (lane == 0) mbar_arrive(bar(B_VFULL + vs));
      return true;
    };
    int nk1 = -1, nk2 = -1;  // keys of the last two tiles (-1: all)
    for (int seg = 0; ok; ++seg) {
      if (!__all_sync(0xffffffffu, wait_bar(bar(B_SEG + seg % kSegs), (seg / kSegs) & 1, a.status,
                                            abort_flag)))
        break;
      const Segment s = segs[seg % kSegs];
      if (s.cnt == 0) break;
      const bool rises = flags.has(s.place, s.h, a.HQ, UnitFlags::kRises);
      int ri[8];
      if (s.page_i >= 0) {
        const int4* r4 = reinterpret_cast<const int4*>(a.rp + ((long)s.page_i * a.HQ + s.h) * KD + ch * 8);
        const int4 u = __ldg(r4), w = __ldg(r4 + 1);
        ri[0] = u.x; ri[1] = u.y; ri[2] = u.z; ri[3] = u.w;
        ri[4] = w.x; ri[5] = w.y; ri[6] = w.z; ri[7] = w.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) ri[e] = 0;
      }
      bool flag = false;
      for (int y = 0; y < s.cnt; ++y, ++g) {
        const int st = g % kKS;
        if (!__all_sync(0xffffffffu, wait_bar(bar(B_KFULL + st), (g / kKS) & 1, a.status, abort_flag))) {
          ok = false;
          break;
        }
        const int j0 = s.j0 + y * BN;
        uint8_t* kt = smem + Lay::oK + st * Lay::kT + (ch / 8) * (BN * 128);
        // 2^(R_I - R_c) of the page that begins at the tile's row 32 z (rows past
        // the request's last page hold what an earlier tile left: scaled along,
        // and masked)
        uint32_t f0 = 0, f1 = 0, f2 = 0, f3 = 0;
        bool low = false;  // some factor lies below 2^-126 and is the first of two
        auto factors = [&](int z) {
          if ((z * 32 & (PS - 1)) != 0) return;
          const int4* rc = reinterpret_cast<const int4*>(
              reinterpret_cast<const int*>(smem + Lay::oR) + (st * Lay::kRows + (z * 32 >> a.shift)) * KD + ch * 8);
          const int4 u = rc[0], v = rc[1];
          int d[8] = {ri[0] - u.x, ri[1] - u.y, ri[2] - u.z, ri[3] - u.w,
                      ri[4] - v.x, ri[5] - v.y, ri[6] - v.z, ri[7] - v.w};
          int most = d[0];
#pragma unroll
          for (int e = 1; e < 8; ++e) most = max(most, d[e]);
          // beyond the operands' range, on a page that some row sees
          if (most > (int)kAnchorRange)
            flag |= j0 + z * 32 < min(s.kv, s.pos0 + s.ni) && j0 + z * 32 + PS > s.from;
          if (rises) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              low |= d[e] < kLowest;
              d[e] = max(d[e], kLowest);
            }
          }
          f0 = pow2_bf16(d[0]) | (pow2_bf16(d[1]) << 16);
          f1 = pow2_bf16(d[2]) | (pow2_bf16(d[3]) << 16);
          f2 = pow2_bf16(d[4]) | (pow2_bf16(d[5]) << 16);
          f3 = pow2_bf16(d[6]) | (pow2_bf16(d[7]) << 16);
        };
        auto vec = [&](int z, int x) {  // this thread's x-th vector of rows [32 z, 32 z + 32)
          const int r = z * 32 + rs + x * kRowStep;
          return reinterpret_cast<uint4*>(kt + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
        };
        auto load = [&](int z, uint4 (&w)[kBatch]) {
#pragma unroll
          for (int x = 0; x < kBatch; ++x) w[x] = *vec(z, x);
        };
        auto scale = [&](int z, uint4 (&w)[kBatch]) {
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            *vec(z, x) = make_uint4(mul_bf16x2(w[x].x, f0), mul_bf16x2(w[x].y, f1),
                                    mul_bf16x2(w[x].z, f2), mul_bf16x2(w[x].w, f3));
          }
        };
        // A shared-memory load takes hundreds of cycles while the tensor core
        // streams its operands: 32 rows (KD / 16 vectors a thread) are loaded
        // before the first is scaled.
#pragma unroll 1
        for (int z = 0; z < 4; ++z) {
          uint4 wa[kBatch];
          load(z, wa);
          factors(z);
          scale(z, wa);
        }
        if (low)
          scale_again<KD>(smem + Lay::oK + st * Lay::kT,
                          reinterpret_cast<const int*>(smem + Lay::oR) + st * Lay::kRows * KD,
                          make_int4(ri[0], ri[1], ri[2], ri[3]), make_int4(ri[4], ri[5], ri[6], ri[7]),
                          a.shift);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_KREADY + st));
        // The value tile of two tiles ago, where the keys end in it: by now it
        // has landed, and the keys that the next S need are scaled already.
        if (nk2 >= 0 && !end_values(g - 2, nk2)) {
          ok = false;
          break;
        }
        nk2 = nk1;
        nk1 = s.kv - j0 < BN ? max(0, s.kv - j0) : -1;
      }
      if (flag) flags.set(s.place, s.h, a.HQ);
    }
#pragma unroll 1
    for (int left = 2; ok && left > 0; --left) {
      if (nk2 >= 0) ok = end_values(g - left, nk2);
      nk2 = nk1;
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
    int g0 = 0;  // the CTA's tiles before the segment
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      if (!__all_sync(0xffffffffu, wait_bar(bar(B_SEG + seg % kSegs), (seg / kSegs) & 1, a.status,
                                            abort_flag)))
        break;
      const Segment& s = segs[seg % kSegs];
      const int cnt = s.cnt;
      if (cnt == 0) break;
      const bool row_ok = r < s.ni;
      // a unit of few rows leaves whole warps without one: they keep step only
      const bool idle = quarter * 32 >= s.ni;
      float m_use = -INFINITY, l = 0.f, raise = 0.f;
      const int first = (g0 + grp) & 1;       // this group's first tile of the segment
      for (int y = first; y < cnt; y += 2) {
        const int g = g0 + y;
        if (!__all_sync(0xffffffffu, wait_bar(bar(B_SFULL + grp), (g >> 1) & 1, a.status, abort_flag))) {
          ok = false;
          break;
        }
        if (idle) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PFULL + grp));
          continue;
        }
        tc_fence_after();
        const bool fast = y >= s.fa && y < s.fb;  // the same for the whole CTA
        // The row's visible keys of the tile are [ja, jb), both rising from row
        // to row.  Per 32 keys the whole warp decides whether all of its rows
        // see all of them, none sees any, or it has to look at each.
        const int dist = s.pos0 + r - (s.j0 + y * BN);  // from the tile's first key to the row
        const int jb = dist + 1, ja = a.window > 0 ? jb - a.window : -BN;
        const int last = min(31, s.ni - 1 - quarter * 32);  // the warp's last row
        auto all_seen = [&](int cc) {
          return fast || (cc >= ja - lane + last && cc + 32 <= jb - lane);
        };
        auto none_seen = [&](int cc) {
          return !fast && (cc >= jb - lane + last || cc + 32 <= ja - lane);
        };
        // The exponentials are taken against a reference of the row's own, its
        // max over the first keys that it sees; it need not be the max of all,
        // since P (bf16), its sum and O (fp32) are floating point: it is raised,
        // and O scaled, by whole powers of two when a tile's sum has passed
        // 2^8, and a tile that passes 2^100 flags the unit.  So S is read once,
        // and P can take its place 32 keys at a time.
        if (__any_sync(0xffffffffu, row_ok && m_use == -INFINITY)) {
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
          for (int cc = 0; cc < BN; cc += 32) {
            if (none_seen(cc)) continue;
            uint32_t sv[32];
            tmem_ld32(s_addr + cc, sv);
            tmem_wait_ld();
            if (all_seen(cc)) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                mx0 = fmaxf(mx0, __uint_as_float(sv[e]));
                mx1 = fmaxf(mx1, __uint_as_float(sv[e + 1]));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const bool vis = cc + e >= ja && cc + e < jb;
                mx0 = fmaxf(mx0, vis ? __uint_as_float(sv[e]) : -INFINITY);
              }
            }
          }
          if (m_use == -INFINITY) m_use = fmaxf(mx0, mx1) * sl2;
        }
        if (__any_sync(0xffffffffu, raise != 0.f)) {
          // (S of this tile came behind this group's last P V, so O is whole)
          const float f = exp2f(-raise);
#pragma unroll 1
          for (int cc = 0; cc < V / 32; ++cc) {
            uint32_t ov[32];
            tmem_ld32(o_addr + cc * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
            tmem_st32(o_addr + cc * 32, ov);
          }
          l *= f;
          m_use += raise;
        }
        const float off = m_use == -INFINITY ? 0.f : -m_use;
        float r0 = 0.f, r1 = 0.f;
        if (fast) {
#pragma unroll 1
          for (int cc = 0; cc < BN; cc += 32) {
            uint32_t sv[32], pk[16];
            tmem_ld32(s_addr + cc, sv);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float p0 = exp2f(fmaf(__uint_as_float(sv[e]), sl2, off));
              const float p1 = exp2f(fmaf(__uint_as_float(sv[e + 1]), sl2, off));
              const float p2 = exp2f(fmaf(__uint_as_float(sv[e + 2]), sl2, off));
              const float p3 = exp2f(fmaf(__uint_as_float(sv[e + 3]), sl2, off));
              r0 += p0 + p2;
              r1 += p1 + p3;
              pk[e / 2] = pack_bf16x2(p0, p1);
              pk[e / 2 + 1] = pack_bf16x2(p2, p3);
            }
            tmem_st16(s_addr + cc / 2, pk);
          }
        } else {
#pragma unroll 1
          for (int cc = 0; cc < BN; cc += 32) {
            uint32_t pk[16];
            if (none_seen(cc)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            } else {
              uint32_t sv[32];
              tmem_ld32(s_addr + cc, sv);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float p0 = exp2f(fmaf(__uint_as_float(sv[e]), sl2, off));
                float p1 = exp2f(fmaf(__uint_as_float(sv[e + 1]), sl2, off));
                p0 = cc + e >= ja && cc + e < jb ? p0 : 0.f;
                p1 = cc + e + 1 >= ja && cc + e + 1 < jb ? p1 : 0.f;
                r0 += p0;
                r1 += p1;
                pk[e / 2] = pack_bf16x2(p0, p1);
              }
            }
            tmem_st16(s_addr + cc / 2, pk);
          }
        }
        tmem_wait_st();
        r0 += r1;
        l += r0;
        raise = 0.f;
        if (row_ok && !(r0 <= kRaiseAbove)) {
          if (r0 <= kFlagAbove) raise = (float)((__float_as_int(r0) >> 23) - 127);
          else flags.set(s.place, s.h, a.HQ);  // NaN too
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + grp));
      }
      // ---- the unit's end, or the share's: merge the groups' (m, l, O)
      const int mine = (cnt - first + 1) >> 1;  // this group's tiles
      if (ok && mine > 0) {
        const int g_last = g0 + first + 2 * (mine - 1);
        ok = __all_sync(0xffffffffu, wait_bar(bar(B_PVDONE + grp), (g_last >> 1) & 1, a.status,
                                              abort_flag));
      }
      float* xm = sX + (seg & 1) * (2 * 2 * BM);
      xm[(grp * 2) * BM + r] = m_use;
      xm[(grp * 2 + 1) * BM + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_XCHG));
      if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(B_XCHG), seg & 1, a.status, abort_flag));
      if (ok) {
        tc_fence_after();
        const float m0 = xm[0 * BM + r], l0 = xm[1 * BM + r];
        const float m1 = xm[2 * BM + r], l1 = xm[3 * BM + r];
        // the groups with a tile: both from two on
        const bool has0 = cnt > 1 || (g0 & 1) == 0, has1 = cnt > 1 || (g0 & 1) == 1;
        const bool whole = s.whole != 0;
        const int h = s.h;
        float m_f = fmaxf(m0, m1);
        if (whole && a.sink) m_f = fmaxf(m_f, a.sink[h] * kLog2e);
        const float a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - m_f);
        const float a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - m_f);
        float lt = l0 * a0 + l1 * a1;
        float inv = 1.f;
        if (whole) {
          if (a.sink) lt += sink_weight(a.sink[h] * kLog2e, m_f);
          inv = lt > 0.f || lt != lt ? 1.f / lt : 0.f;  // a row that sees nothing: 0
        }
        const float f0 = a0 * inv, f1 = a1 * inv;
        const long row = (long)(s.t0 + r) * a.HQ + h;
        // each group writes half of the channels
        if (!idle) {
          // a NaN may be 0 * infinity or 0 * NaN of a masked value, an infinity a
          // sum that passed fp32 before its reference was raised
          bool bad = false;
#pragma unroll 1
          for (int cc = grp * (V / 2); cc < (grp + 1) * (V / 2); cc += 32) {
            uint32_t ov0[32], ov1[32];
            if (has0) tmem_ld32(tmem + lane_base + 256 + cc, ov0);
            if (has1) tmem_ld32(tmem + lane_base + 256 + V + cc, ov1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              // (a row whose weight is 0 had no key in the group: its O is 0)
              float x = has0 ? __uint_as_float(ov0[e]) * f0 : 0.f;
              if (has1) x = fmaf(__uint_as_float(ov1[e]), f1, x);
              bad |= !(fabsf(x) < INFINITY);
              ov0[e] = __float_as_uint(x);
            }
            if (row_ok) {
              if (whole) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * V + cc);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t pk[4];
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    pk[x] = pack_bf16x2(__uint_as_float(ov0[8 * e + 2 * x]),
                                        __uint_as_float(ov0[8 * e + 2 * x + 1]));
                  dst[e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
              } else {
                uint4* dst = reinterpret_cast<uint4*>(parts.o(cta, s.slot, V) + (size_t)r * V + cc);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  dst[e] = make_uint4(ov0[4 * e], ov0[4 * e + 1], ov0[4 * e + 2], ov0[4 * e + 3]);
              }
            }
          }
          tc_fence_before();
          if (bad && row_ok) flags.set(s.place, h, a.HQ);
        }
        if (grp == 0 && row_ok) {
          if (whole) {
            if (a.lse) a.lse[row] = lt == 0.f ? -INFINITY : (m_f + log2f(lt)) * kLn2;
          } else {
            float* pm = parts.ml(cta, s.slot, V) + r * 2;
            pm[0] = m_f;
            pm[1] = lt;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_OEMPTY));
      g0 += cnt;
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
// Qh = q * 2^(p + R_{page(i)} - R_I): rows of requests of n_min or more, a CTA a
// row at a time, eight channels a thread.  An exponent past +-kAnchorRange
// flags the row's unit; one above kRise marks it.
__global__ void __launch_bounds__(256) chunk_queries_kernel(AttnArgs a, __nv_bfloat16* qh,
                                                            UnitFlags flags) {
  start_next();
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
    if (t < r.t0 || t >= r.t0 + r.n || r.n < a.n_min || r.dead) continue;
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
      bool wide = false, rises = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        wide |= fabsf(pv[e]) > kAnchorRange;
        rises |= pv[e] > kRise;
        qv[e] *= exp2f(pv[e]);
      }
      if (rises) flags.mark(flags.place(r, b), off / a.K, a.HQ, UnitFlags::kRises);
      if (wide) flags.set(flags.place(r, b), off / a.K, a.HQ);
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
  return launch_behind(paged_chunk_kernel<KD>, parts.n_cta, kThreads, Smem<KD>::kAlloc, stream, tq, tk,
                       tv, a, parts, flags);
}

}  // namespace

namespace paged {

bool chunk_rows_supported(int dtype, int K, int V) {
  return dtype == WALL_BF16 && K == V && (K == 64 || K == 128);
}

int chunk_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, void* qh,
               cudaStream_t stream) {
  __nv_bfloat16* q16 = static_cast<__nv_bfloat16*>(qh);
  const int blocks = a.bt.T < kSms * 8 ? a.bt.T : kSms * 8;
  // In stream order: started while the decode kernel holds the SMs' shared
  // memory, it would run with the L1 that this leaves (an 8192-token prompt:
  // 416 us for the call against 406).
  chunk_queries_kernel<<<blocks, 256, 0, stream>>>(a, q16, flags);
  if (cudaGetLastError() != cudaSuccess) return WALL_ERR_CUDA;
  return a.K == 128 ? launch<128>(a, parts, flags, q16, stream)
                    : launch<64>(a, parts, flags, q16, stream);
}

}  // namespace paged
}  // namespace wall
