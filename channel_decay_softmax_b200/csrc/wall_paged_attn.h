// wall_paged_attn.h -- arguments and launchers of the paged attention kernels.
#pragma once

#include "wall_internal.h"
#include "wall_paged.cuh"

namespace wall {
namespace paged {

// CTAs that share the tiles of a batch, for each kind of kernel: one per SM
// for the kernels that fill an SM's shared memory, three for the general one.
constexpr int kSms = 148;
constexpr int kGeneralCtas = kSms * 3;
constexpr int kGeneralRows = 32;  // query rows of a general unit, keys of a tile
constexpr int kChunkRows = 128;   // the same of the tensor-core kernel
constexpr int kShortRows = 8;     // rows of a request that the decode kernel can take

struct AttnArgs {
  const void* q;        // [T, HQ, K]
  const float* p;       // [T, HQ, K]
  Batch bt;
  const int* table;     // [N, MP]
  int MP, NP, shift;
  int H, HQ, K, V;
  const void *kp, *vp;
  const int* rp;
  const float* sink;
  float scale_log2;     // scale * log2(e)
  int window;           // 0: none
  int max_new;
  int n_min;            // requests of so many rows on are the chunk (or general) kernel's
  void* o;              // [T, HQ, V]
  float* lse;           // [T, HQ] or null
  int* status;
};

// A kernel's partial results: CTA c's unit that an earlier CTA began (slot 0)
// and the one that it begins and a later CTA ends (slot 1), each `rows` rows
// of V sums followed by their (max, sum) pairs, in the log2 domain.
struct Parts {
  PartDesc* desc;  // one per CTA
  float* data;
  int rows;
  int n_cta;
  // floats of one part: whole 16-byte vectors, whatever the number of rows
  __host__ __device__ static size_t stride_of(int rows, int V) {
    return ((size_t)rows * (V + 2) + 3) & ~size_t(3);
  }
  __device__ __forceinline__ size_t stride(int V) const { return stride_of(rows, V); }
  __device__ __forceinline__ float* o(int cta, int slot, int V) const {
    return data + ((size_t)cta * 2 + slot) * stride(V);
  }
  __device__ __forceinline__ float* ml(int cta, int slot, int V) const {
    return o(cta, slot, V) + (size_t)rows * V;
  }
};

// What the tensor-core kernel's units are: a word for each (128-row block, head),
// cleared by every call, and one more that says whether any is to be computed
// again by the general kernel.  Block b of request i has place t0 / 128 + i + b, which
// no two share (a request of n rows starting at t0 ends before place
// (t0 + n) / 128 + i + 1).
struct UnitFlags {
  static constexpr int kAgain = 1;  // the general kernel computes the unit again
  static constexpr int kRises = 2;  // see kRise (wall_paged_chunk_sm100.cu)
  int* f;
  __host__ __device__ static long places(int N, int T) { return (long)T / kChunkRows + N; }
  __host__ __device__ static long count(int N, int T, int HQ) { return places(N, T) * HQ + 1; }
  int places_n;
  long total;  // count(N, T, HQ); 0: the call has none
  __device__ __forceinline__ int* any(int HQ) const { return f + (long)places_n * HQ; }
  __device__ __forceinline__ long place(const Request& r, int b) const {
    return (long)r.t0 / kChunkRows + r.i + b;
  }
  // (64 bits: 2^20 requests of 4096 heads have more words than an int counts)
  __device__ __forceinline__ int* at(long place, int h, int HQ) const { return f + place * HQ + h; }
  __device__ __forceinline__ bool has(long place, int h, int HQ, int bit) const {
    return (*reinterpret_cast<volatile int*>(at(place, h, HQ)) & bit) != 0;
  }
  __device__ __forceinline__ void mark(long place, int h, int HQ, int bit) const {
    if (!has(place, h, HQ, bit)) atomicOr(at(place, h, HQ), bit);
  }
  __device__ __forceinline__ void set(long place, int h, int HQ) const {
    mark(place, h, HQ, kAgain);
    set_flag(any(HQ));
  }
};

// rows of requests of n_min or more (wall_paged_chunk_sm100.cu): Parts of
// kChunkRows rows, kSms CTAs; qh: bf16 [T, HQ, K] of scratch
bool chunk_rows_supported(int dtype, int K, int V);
int chunk_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, void* qh,
               cudaStream_t stream);

// rows of requests of one, or of one to max_new where few_rows() says so
// (wall_paged_decode.cu): Parts of as many rows times HQ / H, kSms CTAs; it also
// clears the flags of the call's other units
inline bool few_rows(int max_new) { return max_new > 1 && max_new <= kShortRows; }
bool decode_rows_supported(int dtype, int H, int HQ, int K, int V);
int decode_rows(const AttnArgs& a, const Parts& parts, const UnitFlags& flags, cudaStream_t stream);

}  // namespace paged
}  // namespace wall
