// wall_paged_attn.h -- arguments and launchers of the paged attention kernels.
#pragma once

#include "wall_internal.h"
#include "wall_paged.cuh"

namespace wall {
namespace paged {

// CTAs that share the tiles of a batch, for each kind of kernel: one per SM
// for the kernels that fill an SM's shared memory, four for the general one.
constexpr int kSms = 148;
constexpr int kGeneralCtas = kSms * 4;
constexpr int kGeneralRows = 32;  // query rows of a general unit, keys of a tile

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

// single-token rows (wall_paged_decode.cu): Parts of HQ / H rows, kSms CTAs
bool decode_rows_supported(int dtype, int H, int HQ, int K, int V);
int decode_rows(const AttnArgs& a, const Parts& parts, cudaStream_t stream);

}  // namespace paged
}  // namespace wall
