// wall_paged_abi.cu -- the extern "C" entry points of the paged cache:
// argument checks and dispatch.  See include/wall_paged.h.
#include <math.h>

#include "wall_internal.h"
#include "wall_paged.h"

namespace wall {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok_ptr(const void* p, unsigned n) { return p != nullptr && aligned(p, n); }

constexpr int kMaxRequests = 1 << 20;

// log2 of a supported page size, or -1
int page_shift(int page_size) {
  return page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

// Shapes shared by the append and the attention.
int check_cache(int dtype, int n_req, int n_tokens, int H, int HQ, int K, int V, int page_size,
                int num_pages) {
  if (dtype != WALL_BF16 && dtype != WALL_FP32) return WALL_ERR_INVALID_ARG;
  if (n_req < 0 || n_tokens < 0 || H < 1 || HQ < 1 || HQ % H != 0 || num_pages < 1)
    return WALL_ERR_INVALID_ARG;
  if (K < 8 || K > 128 || K % 8 != 0 || V < 8 || V > 128 || V % 8 != 0) return WALL_ERR_UNSUPPORTED;
  if (page_shift(page_size) < 0 || n_req > kMaxRequests || HQ > 4096) return WALL_ERR_UNSUPPORTED;
  // rows of the pools are indexed by 32-bit TMA coordinates
  if ((long)num_pages * page_size * HQ >= (1l << 31)) return WALL_ERR_UNSUPPORTED;
  return WALL_OK;
}

}  // namespace
}  // namespace wall

using namespace wall;

extern "C" {

int wall_paged_plan(const int32_t* new_lens, const int32_t* lens, int32_t* block_table,
                    const int32_t* free_list, const int32_t* free_count, int n_req, int max_pages,
                    int num_pages, int page_size, int n_tokens, int32_t* cu_q, int32_t* kv_lens,
                    int64_t* slot_map, int32_t* admitted, int32_t* lens_out,
                    int32_t* free_count_out, wall_stream_t stream) {
  const TraceRange trace(__func__);
  if (n_req < 0 || max_pages < 1 || num_pages < 1 || n_tokens < 0) return WALL_ERR_INVALID_ARG;
  const int shift = page_shift(page_size);
  if (shift < 0 || n_req > kMaxRequests || (long)max_pages * page_size >= (1l << 31))
    return WALL_ERR_UNSUPPORTED;
  if (!ok_ptr(free_list, 4) || !ok_ptr(free_count, 4) || !ok_ptr(cu_q, 4) ||
      !ok_ptr(free_count_out, 4))
    return WALL_ERR_INVALID_ARG;
  if (n_req > 0 && (!ok_ptr(new_lens, 4) || !ok_ptr(lens, 4) || !ok_ptr(block_table, 4) ||
                    !ok_ptr(kv_lens, 4) || !ok_ptr(admitted, 4) || !ok_ptr(lens_out, 4)))
    return WALL_ERR_INVALID_ARG;
  if (n_tokens > 0 && !ok_ptr(slot_map, 8)) return WALL_ERR_INVALID_ARG;
  return paged_plan(new_lens, lens, block_table, free_list, free_count, n_req, max_pages,
                    num_pages, shift, n_tokens, cu_q, kv_lens, slot_map, admitted, lens_out,
                    free_count_out, reinterpret_cast<cudaStream_t>(stream));
}

int wall_paged_release(const int32_t* finished, int32_t* lens, int32_t* block_table,
                       int32_t* free_list, int32_t* free_count, int n_req, int max_pages,
                       int num_pages, int page_size, wall_stream_t stream) {
  const TraceRange trace(__func__);
  if (n_req < 0 || max_pages < 1 || num_pages < 1) return WALL_ERR_INVALID_ARG;
  const int shift = page_shift(page_size);
  if (shift < 0 || n_req > kMaxRequests || (long)max_pages * page_size >= (1l << 31))
    return WALL_ERR_UNSUPPORTED;
  if (!ok_ptr(free_list, 4) || !ok_ptr(free_count, 4)) return WALL_ERR_INVALID_ARG;
  if (n_req > 0 && (!ok_ptr(finished, 4) || !ok_ptr(lens, 4) || !ok_ptr(block_table, 4)))
    return WALL_ERR_INVALID_ARG;
  return paged_release(finished, lens, block_table, free_list, free_count, n_req, max_pages,
                       num_pages, shift, reinterpret_cast<cudaStream_t>(stream));
}

size_t wall_paged_append_workspace(int n_req, int n_tokens, int max_new, int HQ, int K,
                                   int page_size) {
  const int shift = page_shift(page_size);
  if (shift < 0 || n_req < 1 || n_tokens < 1 || HQ < 1 || K < 1 || max_new < 0) return 0;
  return paged_append_ws(n_req, n_tokens, HQ, K, shift,
                         max_new > 0 && max_new < n_tokens ? max_new : n_tokens);
}

int wall_paged_append(const void* k, const void* v, const void* g, int dtype, const int32_t* cu_q,
                      const int32_t* kv_lens, const int64_t* slot_map, int n_req, int n_tokens,
                      int max_new, int H, int HQ, int K, int V, int page_size, int num_pages,
                      void* k_pages, void* v_pages, int32_t* r_pages, const int64_t* carry_in,
                      int64_t* carry_out, float* p, void* workspace, size_t workspace_bytes,
                      wall_stream_t stream) {
  const TraceRange trace(__func__);
  int rc = check_cache(dtype, n_req, n_tokens, H, HQ, K, V, page_size, num_pages);
  if (rc) return rc;
  if (max_new < 0) return WALL_ERR_INVALID_ARG;
  if (n_req == 0) return WALL_OK;
  if (!ok_ptr(cu_q, 4) || !ok_ptr(kv_lens, 4) || !ok_ptr(carry_in, 16) || !ok_ptr(carry_out, 16) ||
      !ok_ptr(k_pages, 16) || !ok_ptr(v_pages, 16) || !ok_ptr(r_pages, 16))
    return WALL_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!ok_ptr(k, 16) || !ok_ptr(v, 16) || !ok_ptr(g, 16) || !ok_ptr(p, 16) ||
                       !ok_ptr(slot_map, 8)))
    return WALL_ERR_INVALID_ARG;
  PagedAppendProblem pb;
  pb.k = k; pb.v = v; pb.g = g; pb.dtype = dtype;
  pb.cu = cu_q; pb.kv = kv_lens; pb.slots = slot_map;
  pb.N = n_req; pb.T = n_tokens;
  pb.max_new = max_new > 0 && max_new < n_tokens ? max_new : n_tokens;
  pb.H = H; pb.HQ = HQ; pb.K = K; pb.V = V;
  pb.shift = page_shift(page_size);
  pb.NP = num_pages;
  pb.k_pages = k_pages; pb.v_pages = v_pages; pb.r_pages = r_pages;
  pb.carry_in = carry_in; pb.carry_out = carry_out; pb.p = p;
  const size_t need = paged_append_ws(n_req, n_tokens, HQ, K, pb.shift, pb.max_new);
  if (need > 0 && (workspace_bytes < need || !ok_ptr(workspace, 16))) return WALL_ERR_INVALID_ARG;
  return paged_append(pb, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t wall_paged_attn_workspace(int dtype, int n_req, int n_tokens, int max_new, int H, int HQ,
                                 int K, int V) {
  if (check_cache(dtype, n_req, n_tokens, H, HQ, K, V, 64, 1) != WALL_OK || max_new < 0 ||
      n_req == 0 || n_tokens == 0)
    return 0;
  return paged_attn_ws(dtype, n_req, n_tokens, max_new > 0 && max_new < n_tokens ? max_new : n_tokens,
                       H, HQ, K, V);
}

int wall_paged_attn(const void* q, const float* p, int dtype, const int32_t* cu_q,
                    const int32_t* kv_lens, const int32_t* block_table, int n_req, int n_tokens,
                    int max_new, int max_pages, int H, int HQ, int K, int V, int page_size,
                    int num_pages, const void* k_pages, const void* v_pages,
                    const int32_t* r_pages, const float* sink_bias, float scale, int window_size,
                    void* o, float* lse, void* workspace, size_t workspace_bytes,
                    wall_stream_t stream) {
  const TraceRange trace(__func__);
  int rc = check_cache(dtype, n_req, n_tokens, H, HQ, K, V, page_size, num_pages);
  if (rc) return rc;
  if (max_new < 0 || max_pages < 1) return WALL_ERR_INVALID_ARG;
  if ((long)max_pages * page_size >= (1l << 31)) return WALL_ERR_UNSUPPORTED;
  if (n_req == 0 || n_tokens == 0) return WALL_OK;
  if (!ok_ptr(q, 16) || !ok_ptr(p, 16) || !ok_ptr(cu_q, 4) || !ok_ptr(kv_lens, 4) ||
      !ok_ptr(block_table, 4) || !ok_ptr(k_pages, 16) || !ok_ptr(v_pages, 16) ||
      !ok_ptr(r_pages, 16) || !ok_ptr(o, 16) || !aligned(sink_bias, 4) || !aligned(lse, 4))
    return WALL_ERR_INVALID_ARG;
  PagedAttnProblem pb;
  pb.q = q; pb.p = p; pb.dtype = dtype;
  pb.cu = cu_q; pb.kv = kv_lens; pb.table = block_table;
  pb.N = n_req; pb.T = n_tokens; pb.MP = max_pages;
  pb.max_new = max_new > 0 && max_new < n_tokens ? max_new : n_tokens;
  pb.H = H; pb.HQ = HQ; pb.K = K; pb.V = V;
  pb.shift = page_shift(page_size);
  pb.NP = num_pages;
  pb.k_pages = k_pages; pb.v_pages = v_pages; pb.r_pages = r_pages;
  pb.sink = sink_bias;
  pb.scale = scale > 0.f ? scale : 1.f / sqrtf((float)K);
  pb.window = window_size > 0 ? window_size : 0;
  pb.o = o; pb.lse = lse;
  const size_t need = paged_attn_ws(dtype, n_req, n_tokens, pb.max_new, H, HQ, K, V);
  if (need > 0 && (workspace_bytes < need || !ok_ptr(workspace, 16))) return WALL_ERR_INVALID_ARG;
  return paged_attn(pb, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
