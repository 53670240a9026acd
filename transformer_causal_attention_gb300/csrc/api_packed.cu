// api_packed.cu - the exported C ABI of the steps that add several tokens per request over a
// paged cache (see include/attn_packed.h): argument checks and launches.  Nothing is allocated.
#include <limits.h>
#include <math.h>

#include "attn_packed.h"
#include "api.h"

using namespace attn;

namespace attn {
namespace {

// The sizes of an attention call, filled into *a (everything that the workspace depends on).
int check_sizes(int T, int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks,
                attn_dtype_t dtype, PackedArgs* a, bool* bf16, bool* half) {
  if (T <= 0 || B <= 0 || n_h <= 0 || n_kv <= 0 || n_h % n_kv || D_qk <= 0 || D_v <= 0) return ATTN_ERR_ARG;
  if (!parse_dtype(dtype, bf16, half)) return ATTN_ERR_ARG;
  int shift = 0;
  if (int rc = check_pages(n_pages, page_size, max_blocks, &shift)) return rc;
  if (static_cast<long long>(T) * n_h > INT_MAX || static_cast<long long>(B) * n_h > INT_MAX) return ATTN_ERR_ARG;
  if (D_qk % 8 || D_v % 8 || D_qk > 640 || D_v > 512 || n_kv > 65535) return ATTN_ERR_UNSUPPORTED;
  a->T = T;
  a->B = B;
  a->n_h = n_h;
  a->n_kv = n_kv;
  a->D_qk = D_qk;
  a->D_v = D_v;
  a->n_pages = n_pages;
  a->page_shift = shift;
  a->max_blocks = max_blocks;
  return ATTN_OK;
}

// Scratch of either path (which one a call takes also depends on its RoPE span); never 0, so that a
// workspace is always a pointer.
size_t workspace_of(const PackedArgs& a, bool bf16) {
  size_t n = packed_workspace(a);
  if (packed_tc_supported(a, bf16, 0, 0, false, false) && packed_tc_workspace(a) > n) n = packed_tc_workspace(a);
  return n > 16 ? n : 16;
}

int attend(const void* q, const void* k_pages, const void* v_pages, int v_token_stride, const int* block_table,
           const int* cu_new, const int* seqlens, const int* positions, const int* visible, int words, void* out,
           float* lse, int T, int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks,
           float rope_base, int rope_offset, int rope_dims, float scale, attn_dtype_t dtype, void* workspace,
           size_t workspace_bytes, void* stream) {
  if (!q || !k_pages || !v_pages || !block_table || !cu_new || !seqlens || !out || !workspace) return ATTN_ERR_ARG;
  PackedArgs a{};
  bool bf16 = false, half = false;
  if (int rc = check_sizes(T, B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, dtype, &a, &bf16, &half))
    return rc;
  if (v_token_stride < 0) return ATTN_ERR_ARG;
  const long long ldv = v_token_stride ? v_token_stride : static_cast<long long>(n_kv) * D_v;
  if (ldv < static_cast<long long>(n_kv) * D_v && v_pages != k_pages) return ATTN_ERR_ARG;
  if (ldv % 8) return ATTN_ERR_UNSUPPORTED;
  const bool rope = rope_base > 0.f;
  if (rope && (rope_offset < 0 || rope_dims <= 0 || rope_dims % 2 || rope_offset % 2 ||
               rope_offset > D_qk - rope_dims))
    return ATTN_ERR_ARG;
  if (rope && rope_dims / 2 > kMaxRopePairs) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned16(workspace) ||
      !aligned4(block_table) || !aligned4(cu_new) || !aligned4(seqlens) || !aligned4(positions) ||
      !aligned4(visible) || !aligned4(lse))
    return ATTN_ERR_ALIGN;
  const size_t e = bf16 ? 2 : 4, i4 = sizeof(int), rows = static_cast<size_t>(T) * n_h;
  const size_t slots = static_cast<size_t>(n_pages) << a.page_shift, need = workspace_of(a, bf16);
  if (workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  const Extent in[] = {{q, rows * D_qk * e},
                       {k_pages, slots * n_kv * D_qk * e},
                       {v_pages, ((slots - 1) * ldv + static_cast<size_t>(n_kv) * D_v) * e},
                       {block_table, static_cast<size_t>(B) * max_blocks * i4},
                       {cu_new, (static_cast<size_t>(B) + 1) * i4},
                       {seqlens, static_cast<size_t>(B) * i4},
                       {positions, static_cast<size_t>(T) * i4},
                       {visible, static_cast<size_t>(T) * words * i4}};
  const Extent outs[] = {{out, rows * D_v * e}, {lse, rows * sizeof(float)}, {workspace, need}};
  if (overlaps(outs, 3, in, 8)) return ATTN_ERR_ARG;

  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(D_qk));
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.v_token_stride = ldv;
  a.block_table = block_table;
  a.cu_new = cu_new;
  a.seqlens = seqlens;
  a.positions = positions;
  a.visible = visible;
  a.words = words;
  a.out = out;
  a.lse = lse;
  a.rope_offset = rope ? rope_offset : 0;
  a.scale_log2 = sc * kLog2e;
  a.workspace = workspace;
  a.status = dev.status;
  a.wait_limit_ns = wait_limit_ns();
  const RopeFreq rf = make_rope(rope_base, rope ? rope_dims : 0, half);
  int launches = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (packed_tc_supported(a, bf16, rope_offset, rope_dims, rope, half))
    return finish(launch_packed_tc(a, rf, dev.sms, st, &launches), launches);
  return finish(launch_packed(a, rf, bf16, st, &launches), launches);
}

}  // namespace
}  // namespace attn

extern "C" {

size_t attn_packed_workspace_size(int T, int B, int n_h, int n_kv, int D_qk, int D_v, int page_size, int max_blocks,
                                  attn_dtype_t dtype) {
  PackedArgs a{};
  bool bf16 = false, half = false;
  if (check_sizes(T, B, n_h, n_kv, D_qk, D_v, 1, page_size, max_blocks, dtype, &a, &bf16, &half))
    return static_cast<size_t>(-1);
  return workspace_of(a, bf16);
}

int attn_prefill_paged(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                       const int* block_table, const int* cu_new, const int* seqlens, const int* positions, void* out,
                       float* lse, int T, int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages, int page_size,
                       int max_blocks, float rope_base, int rope_offset, int rope_dims, float scale,
                       attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return attend(q, k_pages, v_pages, v_token_stride, block_table, cu_new, seqlens, positions, nullptr, 0, out, lse, T,
                B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, rope_base, rope_offset, rope_dims, scale,
                dtype, workspace, workspace_bytes, stream);
}

int attn_decode_tree(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                     const int* block_table, const int* cu_new, const int* seqlens, const int* positions,
                     const int* visible, int words, void* out, float* lse, int T, int B, int n_h, int n_kv, int D_qk,
                     int D_v, int n_pages, int page_size, int max_blocks, float rope_base, int rope_offset,
                     int rope_dims, float scale, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (!visible || words < 1 || words > kMaxDrafts / 32) return ATTN_ERR_ARG;
  return attend(q, k_pages, v_pages, v_token_stride, block_table, cu_new, seqlens, positions, visible, words, out, lse,
                T, B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, rope_base, rope_offset, rope_dims, scale,
                dtype, workspace, workspace_bytes, stream);
}

int attn_draft_plan(const int* places, const int* cu_new, const int* parents, int* positions, int* visible, int T,
                    int B, int words, void* stream) {
  if (!places || !cu_new || !parents || !positions || !visible) return ATTN_ERR_ARG;
  if (T <= 0 || B <= 0 || words < 1 || words > kMaxDrafts / 32) return ATTN_ERR_ARG;
  if (B > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  const size_t t = static_cast<size_t>(T) * sizeof(int);
  const Extent in[] = {{places, t}, {cu_new, (static_cast<size_t>(B) + 1) * sizeof(int)}, {parents, t}};
  const Extent outs[] = {{positions, t}, {visible, t * words}};
  for (const Extent& x : in)
    if (!aligned4(x.p)) return ATTN_ERR_ALIGN;
  for (const Extent& x : outs)
    if (!aligned4(x.p)) return ATTN_ERR_ALIGN;
  if (overlaps(outs, 2, in, 3)) return ATTN_ERR_ARG;
  int launches = 0;
  const cudaError_t err = launch_draft_plan(DraftPlanArgs{places, cu_new, parents, positions, visible, T, B, words},
                                            static_cast<cudaStream_t>(stream), &launches);
  return finish(err, launches);
}

int attn_draft_commit(void* k_pages, void* v_pages, int v_token_stride, const int* block_table, const int* lens,
                      const int* seqlens, const int* path, const int* n_path, int* new_lens, int* free_pages,
                      const int* n_free, int* n_left, int B, int max_path, int n_kv, int D_qk, int D_v, int n_pages,
                      int page_size, int max_blocks, int free_cap, attn_dtype_t dtype, void* stream) {
  if (!k_pages || !block_table || !lens || !seqlens || !path || !n_path || !new_lens) return ATTN_ERR_ARG;
  const bool stack = free_pages != nullptr;
  if (stack != (n_free != nullptr) || stack != (n_left != nullptr)) return ATTN_ERR_ARG;
  if (B <= 0 || max_path <= 0 || n_kv <= 0 || D_qk <= 0 || D_v <= 0 || v_token_stride < 0 || (stack && free_cap <= 0))
    return ATTN_ERR_ARG;
  bool bf16 = false, half = false;
  if (!parse_dtype(dtype, &bf16, &half)) return ATTN_ERR_ARG;
  int shift = 0;
  if (int rc = check_pages(n_pages, page_size, max_blocks, &shift)) return rc;
  if (stack && free_cap > n_pages) return ATTN_ERR_ARG;
  if (D_qk % 8 || D_v % 8 || B > kMaxPlanRequests || max_path > kMaxDrafts) return ATTN_ERR_UNSUPPORTED;
  const long long ldv = v_token_stride ? v_token_stride : static_cast<long long>(n_kv) * D_v;
  if (v_pages && ldv < static_cast<long long>(n_kv) * D_v) return ATTN_ERR_ARG;  // slots would overlap
  if (v_pages && ldv % 8) return ATTN_ERR_UNSUPPORTED;
  const size_t e = bf16 ? 2 : 4, i4 = sizeof(int), b = static_cast<size_t>(B), slots = static_cast<size_t>(n_pages) << shift;
  DraftCommitArgs a{};
  a.k_row = static_cast<long long>(n_kv) * D_qk * e / 16;
  a.v_row = v_pages ? static_cast<long long>(n_kv) * D_v * e / 16 : 0;
  if (B * ((a.k_row + a.v_row + 255) / 256) > INT_MAX - 1) return ATTN_ERR_UNSUPPORTED;
  const Extent in[] = {{block_table, b * max_blocks * i4}, {lens, b * i4},   {seqlens, b * i4},
                       {path, b * max_path * i4},          {n_path, b * i4}, {n_free, i4}};
  const Extent outs[] = {{k_pages, slots * n_kv * D_qk * e},
                         {v_pages, ((slots - 1) * ldv + static_cast<size_t>(n_kv) * D_v) * e},
                         {new_lens, b * i4},
                         {free_pages, static_cast<size_t>(free_cap) * i4},
                         {n_left, i4}};
  for (const Extent& x : in)
    if (!aligned4(x.p)) return ATTN_ERR_ALIGN;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned4(new_lens) || !aligned4(free_pages) || !aligned4(n_left))
    return ATTN_ERR_ALIGN;
  if (overlaps(outs, 5, in, 6)) return ATTN_ERR_ARG;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.v_stride = ldv * static_cast<long long>(e);
  a.block_table = block_table;
  a.lens = lens;
  a.seqlens = seqlens;
  a.path = path;
  a.n_path = n_path;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.n_left = n_left;
  a.B = B;
  a.max_path = max_path;
  a.n_pages = n_pages;
  a.page_shift = shift;
  a.max_blocks = max_blocks;
  a.free_cap = free_cap;
  int launches = 0;
  const cudaError_t err = launch_draft_commit(a, static_cast<cudaStream_t>(stream), &launches);
  return finish(err, launches);
}

}  // extern "C"
