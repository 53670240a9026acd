// draft.cu - what a step of drafted tokens needs around its attention: positions and
// visibility bits from the drafts' parents, and the move of the accepted ones to
// consecutive places of the paged cache.
#include "kernels.h"

namespace attn {
namespace {

// One block per request, a thread per drafted token: thread i walks from token i to its root (parents
// have smaller indices, so the walk ends), setting a bit and counting a level at each step.  The parents
// are in shared memory, 4 bytes each.  Blocks behind the requests' clear the rows that belong to none.
// Bound by its launch: 59 requests of 32 drafts move 38 KB.
__global__ void __launch_bounds__(kMaxDrafts) draft_plan_kernel(const __grid_constant__ DraftPlanArgs a) {
  __shared__ int parent[kMaxDrafts];
  const int i = threadIdx.x;
  if (blockIdx.x >= a.B) {
    const int stride = (gridDim.x - a.B) * kMaxDrafts;
    for (long long t = min(max(a.cu_new[a.B], 0), a.T) + (blockIdx.x - a.B) * kMaxDrafts + i; t < a.T; t += stride) {
      a.positions[t] = -1;
      for (int w = 0; w < a.words; ++w) a.visible[t * a.words + w] = 0;
    }
    return;
  }
  const int b = blockIdx.x;
  const int first = min(max(a.cu_new[b], 0), a.T), end = min(max(a.cu_new[b + 1], 0), a.T);
  const int n = end - first;
  const int most = 32 * a.words;
  int place = -1;
  if (i < n) {
    parent[i] = a.parents[first + i];
    place = a.places[first + i];
  }
  __syncthreads();
  for (int t = i; t < n; t += kMaxDrafts) {
    uint32_t bits[4] = {0u, 0u, 0u, 0u};
    int position = -1;
    if (t < most && place >= 0) {  // t = i: most <= kMaxDrafts
      int j = t, depth = -1;
      for (;;) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (j >> 5 == w) bits[w] |= 1u << (j & 31);
        ++depth;
        const int p = parent[j];
        if (p < 0 || p >= j) {
          if (p == -1) position = place - t + depth;
          break;
        }
        j = p;
      }
    }
    const long long row = first + static_cast<long long>(t);
    a.positions[row] = position;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (w < a.words) a.visible[row * a.words + w] = position >= 0 ? static_cast<int>(bits[w]) : 0;
  }
}

// Accepted drafts of request b: the entries of its path before the first that does not rise or that the
// request does not have.  By a warp, 32 entries at a time; all lanes get the count.
__device__ __forceinline__ int accepted(const DraftCommitArgs& a, int b, int lane, int held, int len) {
  const int most = min(max(a.n_path[b], 0), a.max_path);
  const int* const path = a.path + static_cast<long long>(b) * a.max_path;
  for (int i0 = 0; i0 < most; i0 += 32) {
    const int i = i0 + lane;
    bool good = false;
    if (i < most) {
      const int p = path[i], before = i > 0 ? path[i - 1] : -1;
      good = p > before && p < len - held;  // held >= 0: no overflow
    }
    const uint32_t bad = __ballot_sync(0xffffffffu, i < most && !good);
    if (bad) return i0 + __ffs(bad) - 1;
  }
  return most;
}
// The same by one thread, eight entries in flight.
__device__ __forceinline__ int accepted_alone(const DraftCommitArgs& a, int b, int held, int len) {
  const int most = min(max(a.n_path[b], 0), a.max_path);
  const int* const path = a.path + static_cast<long long>(b) * a.max_path;
  int before = -1;
  for (int i0 = 0; i0 < most; i0 += 8) {
    int p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = i0 + e < most ? path[i0 + e] : -1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (i0 + e < most && !(p[e] > before && p[e] < len - held)) return i0 + e;
      before = p[e];
    }
  }
  return most;
}

constexpr int kCommitThreads = 256, kCommitBatch = 8;
constexpr int kAlone = 32;  // entries of a row that a thread walks by itself

// Blocks (request, 256 pieces of 16 bytes of a token): each thread moves its piece of the accepted tokens,
// one after the other in batches of kCommitBatch loads.  Token i comes from index path[i] >= i, and later
// ones from higher indices still, so no store hits what is loaded later; a batch is loaded before it is
// stored.  The first block puts the pages that fall free on the stack: a thread counts a request's (a warp those of one with
// more than kAlone entries), a scan over kCommitThreads requests at a time gives their places.  (A warp per request, one
// after the other, took 35 us for 512.)
__global__ void __launch_bounds__(kCommitThreads) draft_commit_kernel(const __grid_constant__ DraftCommitArgs a,
                                                                      int slices) {
  __shared__ long long src[kMaxDrafts], dst[kMaxDrafts];
  __shared__ int shared_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int limit = a.max_blocks << a.page_shift;
  const auto held_of = [&](int b) { return max(a.lens[b], 0); };
  const auto len_of = [&](int b) { return min(max(a.seqlens[b], 0), limit); };
  const int stack = a.free_pages != nullptr;
  if (static_cast<int>(blockIdx.x) >= stack) {
    const int b = (blockIdx.x - stack) / slices, slice = blockIdx.x - stack - b * slices;
    const int held = held_of(b);
    if (warp == 0) {
      const int n = accepted(a, b, lane, held, len_of(b));
      if (lane == 0) shared_n = n;
    }
    __syncthreads();
    const int n = shared_n;
    if (slice == 0 && threadIdx.x == 0) a.new_lens[b] = held + n;
    if (threadIdx.x < n) {
      const int i = threadIdx.x;
      const int from = held + a.path[static_cast<long long>(b) * a.max_path + i], to = held + i;
      const int* const table = a.block_table + static_cast<long long>(b) * a.max_blocks;
      const int mask = (1 << a.page_shift) - 1;
      const int p = table[from >> a.page_shift], q = table[to >> a.page_shift];
      const bool real = from != to && p >= 0 && p < a.n_pages && q >= 0 && q < a.n_pages;
      src[i] = real ? (static_cast<long long>(p) << a.page_shift) + (from & mask) : -1;
      dst[i] = real ? (static_cast<long long>(q) << a.page_shift) + (to & mask) : -1;
    }
    __syncthreads();
    const long long piece = static_cast<long long>(slice) * kCommitThreads + threadIdx.x;
    const bool is_v = piece >= a.k_row;
    if (piece >= a.k_row + a.v_row) return;
    char* const base = is_v ? static_cast<char*>(a.v_pages) + (piece - a.k_row) * 16
                            : static_cast<char*>(a.k_pages) + piece * 16;
    const long long stride = is_v ? a.v_stride : a.k_row * 16;
    for (int i0 = 0; i0 < n; i0 += kCommitBatch) {
      uint4 x[kCommitBatch];
#pragma unroll
      for (int e = 0; e < kCommitBatch; ++e)
        if (i0 + e < n && src[i0 + e] >= 0) x[e] = *reinterpret_cast<const uint4*>(base + src[i0 + e] * stride);
#pragma unroll
      for (int e = 0; e < kCommitBatch; ++e)
        if (i0 + e < n && src[i0 + e] >= 0) *reinterpret_cast<uint4*>(base + dst[i0 + e] * stride) = x[e];
    }
    return;
  }
  // the stack: of each row's surplus entries those that are pages of the cache
  __shared__ long long warp_sum[kCommitThreads / 32];
  const int page = 1 << a.page_shift;
  const auto is_page = [&](int id) { return id >= 0 && id < a.n_pages; };
  long long at = min(max(*a.n_free, 0), a.free_cap);
  for (int b0 = 0; b0 < a.B; b0 += kCommitThreads) {
    const int b = b0 + threadIdx.x;
    int first = 0, mine = 0;
    if (b < a.B) {
      const int held = held_of(b), len = len_of(b), kept = held + accepted_alone(a, b, held, len);
      first = (kept >> a.page_shift) + ((kept & (page - 1)) != 0);
      mine = max((len >> a.page_shift) + ((len & (page - 1)) != 0) - first, 0);
    }
    const int* const entries = a.block_table + static_cast<long long>(b < a.B ? b : 0) * a.max_blocks + first;
    const uint32_t many = __ballot_sync(0xffffffffu, mine > kAlone);  // requests whose entries the warp walks together
    // f(l, n, row): the request of lane l, with n entries from `row` on
    const auto each_of_many = [&](auto f) {
      for (uint32_t left = many; left; left &= left - 1) {
        const int l = __ffs(left) - 1;
        f(l, __shfl_sync(0xffffffffu, mine, l),
          reinterpret_cast<const int*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(entries), l)));
      }
    };
    int real = 0;
    if (mine <= kAlone)
      for (int j = 0; j < mine; ++j) real += is_page(entries[j]);
    each_of_many([&](int l, int n, const int* row) {
      int sum = 0;
#pragma unroll 4
      for (int j = lane; j < n; j += 32) sum += is_page(row[j]);
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == l) real = sum;
    });
    long long before = real;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    long long sum = 0, ahead = 0;
#pragma unroll
    for (int w = 0; w < kCommitThreads / 32; ++w) {
      if (w < warp) ahead += warp_sum[w];
      sum += warp_sum[w];
    }
    const long long to = at + ahead + before - real;
    if (mine <= kAlone) {
      long long put = to;
      for (int j = 0; j < mine && put < a.free_cap; ++j) {
        const int id = entries[j];
        if (is_page(id)) a.free_pages[put++] = id;
      }
    }
    each_of_many([&](int l, int n, const int* row) {
      long long put = __shfl_sync(0xffffffffu, to, l);
      for (int j0 = 0; j0 < n && put < a.free_cap; j0 += 32) {
        const int id = j0 + lane < n ? row[j0 + lane] : -1;
        const uint32_t some = __ballot_sync(0xffffffffu, is_page(id));
        const long long mine_at = put + __popc(some & ((1u << lane) - 1u));
        if (is_page(id) && mine_at < a.free_cap) a.free_pages[mine_at] = id;
        put += __popc(some);
      }
    });
    at += sum;
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.n_left = static_cast<int>(at < a.free_cap ? at : a.free_cap);
}

}  // namespace

cudaError_t launch_draft_plan(const DraftPlanArgs& a, cudaStream_t st, int* launches) {
  // blocks behind the requests' for the rows behind the last one
  const int rest = a.T < 16 * kMaxDrafts ? (a.T + kMaxDrafts - 1) / kMaxDrafts : 16;
  draft_plan_kernel<<<a.B + rest, kMaxDrafts, 0, st>>>(a);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_draft_commit(const DraftCommitArgs& a, cudaStream_t st, int* launches) {
  const int slices = static_cast<int>((a.k_row + a.v_row + kCommitThreads - 1) / kCommitThreads);
  draft_commit_kernel<<<static_cast<unsigned>(a.B) * slices + (a.free_pages ? 1 : 0), kCommitThreads, 0, st>>>(a, slices);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace attn
