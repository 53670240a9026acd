// api.h - host helpers shared by the exported entry points (api.cu, api_paged.cu, api_packed.cu):
// per-device facts, argument checks, the RoPE table, tensor maps and the launch
// counter.  Defined in api.cu; nothing here is exported.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "attn.h"
#include "kernels.h"

namespace attn {

struct DeviceInfo {
  bool ready;
  int sms;
  int l2_bytes;
  unsigned int* status;
};
// Facts of the current device, fetched once per device with that device current.
int device_info(DeviceInfo* out);

// 4-D tensor map over a bf16 tensor indexed (d, head, position, batch); see api.cu.
bool make_map4(CUtensorMap* map, const void* base, int D, int heads, int rows, int B, unsigned long long head_stride,
               unsigned long long row_stride, unsigned long long batch_stride, int box_rows);

// 4-D tensor map over bf16 rows indexed (d, i1, i2, i3), boxes of 64 dims x box1 x box2 x box3; see api.cu.
bool make_map_box(CUtensorMap* map, const void* base, int D, int n1, int n2, int n3, unsigned long long s1,
                  unsigned long long s2, unsigned long long s3, int box1, int box2, int box3, bool promote_256);

// 3-D tensor map over a bf16 tensor indexed (d, row, batch); see api.cu.
bool make_map3(CUtensorMap* map, const void* base, int D, int rows, int B, unsigned long long row_stride,
               unsigned long long batch_stride, int box_rows);

// The dtype argument: element type in the low byte, ATTN_ROPE_HALF optionally OR'd in.
bool parse_dtype(attn_dtype_t dtype, bool* bf16, bool* half);

// theta_i = base^(-2i/dims) expressed in turns per position, split hi + lo.
RopeFreq make_rope(float base, int dims, bool half);

unsigned long long wait_limit_ns();

// Adds the enqueued kernels to the launch counter and maps a launch error to a return code.
int finish(cudaError_t e, int launches);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A buffer's extent; p null: none.
struct Extent {
  const void* p;
  size_t bytes;
};
// Whether an output overlaps an input or another output.
inline bool overlaps(const Extent* outs, int n_outs, const Extent* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    if (!outs[i].p) continue;
    for (int j = 0; j < n_ins; ++j)
      if (ins[j].p && overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (outs[j].p && overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

// The sizes of a paged cache and of a table over it; *shift: log2 of the page size (api_paged.cu).
int check_pages(int n_pages, int page_size, int max_blocks, int* shift);

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace attn
