// api_paged.cu - the exported C ABI of the paged cache (see include/attn_paged.h):
// argument checks, tensor maps and launches.  Nothing is allocated.
#include <limits.h>
#include <math.h>

#include "attn_paged.h"
#include "api.h"

using namespace attn;

namespace attn {
namespace {

// log2 of a supported page size, or -1.
int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Tokens of a table row: 32-bit positions with room for a few tiles or chunks more, which loops over keys step past.
constexpr long long kMaxRequestTokens = (1LL << 31) - (1 << 16);

}  // namespace

// The sizes of a paged cache and of a table over it.
int check_pages(int n_pages, int page_size, int max_blocks, int* shift) {
  if (n_pages <= 0 || page_size <= 0 || max_blocks <= 0) return ATTN_ERR_ARG;
  *shift = page_shift_of(page_size);
  if (*shift < 0) return ATTN_ERR_UNSUPPORTED;
  if ((static_cast<long long>(n_pages) << *shift) > INT_MAX ||
      (static_cast<long long>(max_blocks) << *shift) > kMaxRequestTokens)
    return ATTN_ERR_ARG;
  return ATTN_OK;
}

namespace {

// The sizes of a decode call, filled into *a (everything that the workspace depends on).
int check_sizes(int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks,
                int prefix_len, attn_dtype_t dtype, PagedDecodeArgs* a, bool* bf16, bool* half) {
  if (B <= 0 || n_h <= 0 || n_kv <= 0 || n_h % n_kv || D_qk <= 0 || D_v <= 0 || prefix_len < 0) return ATTN_ERR_ARG;
  if (!parse_dtype(dtype, bf16, half)) return ATTN_ERR_ARG;
  int shift = 0;
  if (int rc = check_pages(n_pages, page_size, max_blocks, &shift)) return rc;
  if (prefix_len % page_size || prefix_len > (max_blocks << shift)) return ATTN_ERR_ARG;
  if (static_cast<long long>(B) * n_h > INT_MAX) return ATTN_ERR_ARG;
  if (D_qk % 8 || D_v % 8 || D_qk > 640 || D_v > 512) return ATTN_ERR_UNSUPPORTED;
  a->B = B;
  a->n_h = n_h;
  a->n_kv = n_kv;
  a->D_qk = D_qk;
  a->D_v = D_v;
  a->n_pages = n_pages;
  a->page_shift = shift;
  a->max_blocks = max_blocks;
  a->prefix_len = prefix_len;
  return ATTN_OK;
}

// The MLA-absorbed shape on the tensor cores (decode_mla.cu), its partials: outputs, then log-sum-exps.
bool mla_shape(const PagedDecodeArgs& a, bool bf16) {
  const long long keys = static_cast<long long>(a.max_blocks) << a.page_shift;
  return decode_mla_supported(a.B, a.n_h, a.n_kv, a.D_qk, a.D_v, a.D_qk, true, bf16) && keys * a.B <= INT_MAX;
}
size_t mla_slots(const PagedDecodeArgs& a) { return static_cast<size_t>(kMlaMaxPairs + a.B) * a.n_h; }

// Scratch of every path (which one a call takes also depends on its RoPE span and where its values lie).
size_t workspace_of(const PagedDecodeArgs& a, bool bf16) {
  size_t n = decode_paged_workspace(a);
  if (mla_shape(a, bf16)) {
    const size_t mla = mla_slots(a) * (a.D_v + 1) * sizeof(float);
    if (mla > n) n = mla;
  }
  if (!decode_paged_tc_supported(a, bf16, 0, 0, false)) return n;
  const size_t tc = decode_paged_tc_workspace(a);
  return tc > n ? tc : n;
}

int decode_impl(const void* q, const void* k_pages, const void* v_pages, int v_token_stride, const int* prefix_pages,
                int prefix_len, const int* block_table, const int* seqlens, void* out, float* lse, int B, int n_h,
                int n_kv, int D_qk, int D_v, int n_pages, int page_size, int max_blocks, float rope_base,
                int rope_offset, int rope_dims, float scale, attn_dtype_t dtype, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!q || !k_pages || !v_pages || !block_table || !seqlens || !out || !workspace) return ATTN_ERR_ARG;
  PagedDecodeArgs a{};
  bool bf16 = false, half = false;
  if (int rc = check_sizes(B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, prefix_len, dtype, &a, &bf16,
                           &half))
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
      !aligned4(block_table) || !aligned4(seqlens) || !aligned4(prefix_pages) || !aligned4(lse))
    return ATTN_ERR_ALIGN;
  if (workspace_bytes < workspace_of(a, bf16)) return ATTN_ERR_WORKSPACE;

  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(D_qk));
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.v_token_stride = ldv;
  a.prefix_pages = prefix_pages;
  a.block_table = block_table;
  a.seqlens = seqlens;
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
  if (mla_shape(a, bf16) && v_pages == k_pages && ldv == D_qk &&
      (!rope || decode_mla_rope_ok(rope_offset, rope_dims, half))) {
    float* const ws_o = static_cast<float*>(workspace);
    const DecodeArgs da{q, k_pages, v_pages, ldv, seqlens, out, lse, B, n_h, n_kv, D_qk, D_v, max_blocks << a.page_shift,
                        a.rope_offset, a.scale_log2, ws_o, ws_o + mla_slots(a) * D_v, decode_mla_pairs(dev.sms), 0,
                        dev.status, a.wait_limit_ns, 0, 0, nullptr};
    const MlaPages pages{block_table, prefix_pages, a.page_shift, max_blocks, prefix_len};
    CUtensorMap maps[2];
    const unsigned long long row = static_cast<unsigned long long>(D_qk) * 2;
    if (!make_map3(&maps[0], q, D_qk, n_h, B, row, row * n_h, 64) ||
        !make_map3(&maps[1], k_pages, D_qk, page_size, n_pages, row, row * page_size, page_size < 128 ? page_size : 128))
      return finish(cudaErrorInvalidValue, launches);
    return finish(launch_decode_mla_paged(da, rf, pages, maps, st, &launches), launches);
  }
  if (!decode_paged_tc_supported(a, bf16, rope_offset, rope_dims, rope))
    return finish(launch_decode_paged(a, rf, bf16, st, &launches), launches);
  return finish(launch_decode_paged_tc(a, rf, dev.sms, st, &launches), launches);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_page_plan(const int* lens, const int* n_new, int* block_table, const int* free_pages, const int* n_free,
                   int* seqlens, int* cu_new, int* slots, int* positions, int* n_left, int B, int max_blocks,
                   int page_size, int n_pages, int free_cap, int max_tokens, void* stream) {
  if (!lens || !n_new || !block_table || !free_pages || !n_free || !seqlens || !cu_new || !slots || !positions ||
      !n_left)
    return ATTN_ERR_ARG;
  int shift = 0;
  if (B <= 0 || free_cap <= 0 || max_tokens <= 0) return ATTN_ERR_ARG;
  if (int rc = check_pages(n_pages, page_size, max_blocks, &shift)) return rc;
  if (free_cap > n_pages) return ATTN_ERR_ARG;
  if (B > kMaxPlanRequests) return ATTN_ERR_UNSUPPORTED;
  struct Buf {
    const void* p;
    size_t bytes;
  };
  const size_t e = sizeof(int), b = static_cast<size_t>(B);
  const Buf in[4] = {{lens, b * e}, {n_new, b * e}, {free_pages, static_cast<size_t>(free_cap) * e}, {n_free, e}};
  const Buf out[6] = {{block_table, b * max_blocks * e},
                      {seqlens, b * e},
                      {cu_new, (b + 1) * e},
                      {slots, static_cast<size_t>(max_tokens) * e},
                      {positions, static_cast<size_t>(max_tokens) * e},
                      {n_left, e}};
  for (const Buf& x : in)
    if (!aligned4(x.p)) return ATTN_ERR_ALIGN;
  for (const Buf& x : out)
    if (!aligned4(x.p)) return ATTN_ERR_ALIGN;
  for (int i = 0; i < 6; ++i) {
    for (const Buf& x : in)
      if (overlap(out[i].p, out[i].bytes, x.p, x.bytes)) return ATTN_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return ATTN_ERR_ARG;
  }
  const PagePlanArgs a{lens,  n_new,      block_table, free_pages, n_free,  seqlens,  cu_new,    slots,
                       positions, n_left, B,           max_blocks, shift,   n_pages,  free_cap,  max_tokens};
  int launches = 0;
  const cudaError_t err = launch_page_plan(a, static_cast<cudaStream_t>(stream), &launches);
  return finish(err, launches);
}

int attn_kv_append_paged(const void* k_new, const void* v_new, void* k_pages, void* v_pages, int v_token_stride,
                         const int* slots, const int* positions, int T, int n_kv, int D_qk, int D_v, int n_pages,
                         int page_size, float rope_base, int rope_offset, int rope_dims, attn_dtype_t dtype,
                         void* stream) {
  const bool rope = rope_base > 0.f;
  if (!k_new || !k_pages || !slots || (v_new && !v_pages) || (rope && !positions)) return ATTN_ERR_ARG;
  if (T <= 0 || n_kv <= 0 || D_qk <= 0 || D_v <= 0 || v_token_stride < 0) return ATTN_ERR_ARG;
  bool bf16 = false, half = false;
  if (!parse_dtype(dtype, &bf16, &half)) return ATTN_ERR_ARG;
  int shift = 0;
  if (int rc = check_pages(n_pages, page_size, 1, &shift)) return rc;
  if (D_qk % 8 || D_v % 8) return ATTN_ERR_ARG;
  if (rope && (rope_offset < 0 || rope_dims <= 0 || rope_offset % 8 || rope_dims % (half ? 16 : 8) ||
               rope_offset > D_qk - rope_dims))
    return ATTN_ERR_ARG;
  if (rope && rope_dims / 2 > kMaxRopePairs) return ATTN_ERR_UNSUPPORTED;
  const long long ldv = v_token_stride ? v_token_stride : static_cast<long long>(n_kv) * D_v;
  if (v_new && ldv < static_cast<long long>(n_kv) * D_v) return ATTN_ERR_ARG;  // slots would overlap
  if (v_new && ldv % 8) return ATTN_ERR_UNSUPPORTED;
  const size_t slots_all = static_cast<size_t>(n_pages) << shift, e = bf16 ? 2 : 4;
  if (v_new && overlap(k_pages, slots_all * n_kv * D_qk * e, v_pages, slots_all * ldv * e)) return ATTN_ERR_ARG;
  if (!aligned16(k_new) || !aligned16(k_pages) || (v_new && (!aligned16(v_new) || !aligned16(v_pages))) ||
      !aligned4(slots) || !aligned4(positions))
    return ATTN_ERR_ALIGN;
  KvAppendArgs a{};
  a.k_new = k_new;
  a.v_new = v_new;
  a.kcache = k_pages;
  a.vcache = v_pages;
  a.v_token_stride = ldv;
  a.B = 1;
  a.C = T;
  a.n_kv = n_kv;
  a.D_qk = D_qk;
  a.D_v = D_v;
  a.rope_offset = rope ? rope_offset : 0;
  a.slots = slots;
  a.positions = positions;
  a.n_slots = n_pages << shift;
  int launches = 0;
  const cudaError_t err = launch_kv_append_paged(a, make_rope(rope_base, rope ? rope_dims : 0, half), bf16,
                                                 static_cast<cudaStream_t>(stream), &launches);
  return finish(err, launches);
}

size_t attn_decode_paged_workspace_size(int B, int n_h, int n_kv, int D_qk, int D_v, int page_size, int max_blocks,
                                        int prefix_len, attn_dtype_t dtype) {
  PagedDecodeArgs a{};
  bool bf16 = false, half = false;
  if (check_sizes(B, n_h, n_kv, D_qk, D_v, 1, page_size, max_blocks, prefix_len, dtype, &a, &bf16, &half))
    return static_cast<size_t>(-1);
  return workspace_of(a, bf16);
}

int attn_decode_paged(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                      const int* block_table, const int* seqlens, void* out, float* lse, int B, int n_h, int n_kv,
                      int D_qk, int D_v, int n_pages, int page_size, int max_blocks, float rope_base, int rope_offset,
                      int rope_dims, float scale, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return decode_impl(q, k_pages, v_pages, v_token_stride, nullptr, 0, block_table, seqlens, out, lse, B, n_h, n_kv,
                     D_qk, D_v, n_pages, page_size, max_blocks, rope_base, rope_offset, rope_dims, scale, dtype,
                     workspace, workspace_bytes, stream);
}

int attn_decode_shared(const void* q, const void* k_pages, const void* v_pages, int v_token_stride,
                       const int* prefix_pages, int prefix_len, const int* block_table, const int* seqlens, void* out,
                       float* lse, int B, int n_h, int n_kv, int D_qk, int D_v, int n_pages, int page_size,
                       int max_blocks, float rope_base, int rope_offset, int rope_dims, float scale,
                       attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!prefix_pages || prefix_len <= 0) return ATTN_ERR_ARG;
  return decode_impl(q, k_pages, v_pages, v_token_stride, prefix_pages, prefix_len, block_table, seqlens, out, lse, B,
                     n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, rope_base, rope_offset, rope_dims, scale,
                     dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
