// page_plan.cu - block tables, slots and positions of a step's new tokens.
//
// Request b holds len tokens and adds n.  With pages of P tokens it owns
// ceil(len / P) pages and comes to need(b) = ceil((len + n) / P) - ceil(len / P)
// more.  Two exclusive prefix sums over the requests order everything: cu of n
// (the packed rows of the new tokens) and pc of need (which pages of the free
// stack are whose).  Token i of request b then has position len + i in block
// (len + i) / P, and that block's page is either already in the table (the
// partly filled last page) or page pc[b] + block - ceil(len / P) from the top of
// the stack - so no token waits for the table to be written.
//
// Every block of threads computes both sums over all requests on its own (8
// bytes per request, from L2) and keeps them in shared memory, then takes its
// share of the tokens and of the taken pages; each finds its request by binary
// search.  That needs no second kernel and no exchange between blocks.  The
// work is a few bytes per token: what bounds it is the chain launch - lengths -
// sums - page - slot, so a step of single tokens runs as one block: 4.2 us for 59
// requests of one token, 9.1 us for 512 requests of up to 255.
#include <limits.h>

#include "kernels.h"

namespace attn {
namespace {

constexpr unsigned kRefused = 0x80000000u;  // in cu: the request's own lengths rule it out

// Inclusive sum over the block's threads; wsum holds one value per warp.
__device__ __forceinline__ long long block_scan(long long v, long long* wsum, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the previous use of wsum is over
  if (lane == 31) wsum[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < n_warps; ++w) {
    const long long x = wsum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

__device__ __forceinline__ int saturate(long long x) { return static_cast<int>(min(x, static_cast<long long>(INT_MAX))); }

// The last request whose sum (flag bit cleared) is at most t.
__device__ __forceinline__ int owner(const unsigned* sum, int B, unsigned t) {
  int lo = 0, hi = B;  // sum[lo] <= t, and t < sum[hi] or hi == B
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((sum[mid] & ~kRefused) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) page_plan_kernel(PagePlanArgs a) {
  extern __shared__ unsigned sums[];
  unsigned* const cu = sums;               // [B + 1] packed row of each request's first token | kRefused
  unsigned* const pc = sums + a.B + 1;     // [B + 1] place of its first new page, counted from the stack's top
  __shared__ long long wsum[32];
  const int page = 1 << a.page_shift;
  const long long room = static_cast<long long>(a.max_blocks) << a.page_shift;
  const int n_free = min(max(*a.n_free, 0), a.free_cap);

  long long t0 = 0, p0 = 0;
  for (int base = 0; base < a.B; base += blockDim.x) {
    const int b = base + threadIdx.x;
    const long long len = b < a.B ? max(a.lens[b], 0) : 0;
    const long long n = b < a.B ? max(a.n_new[b], 0) : 0;
    long long all;
    const long long end = t0 + block_scan(n, wsum, &all);
    t0 += all;
    const bool fits = len + n <= room && end <= a.max_tokens;
    const long long need = fits ? ((len + n + page - 1) >> a.page_shift) - ((len + page - 1) >> a.page_shift) : 0;
    const long long pend = p0 + block_scan(need, wsum, &all);
    p0 += all;
    if (b < a.B) {
      cu[b] = static_cast<unsigned>(saturate(end - n)) | (fits ? 0u : kRefused);
      pc[b] = static_cast<unsigned>(saturate(pend - need));
    }
  }
  if (threadIdx.x == 0) {
    cu[a.B] = static_cast<unsigned>(saturate(t0));
    pc[a.B] = static_cast<unsigned>(saturate(p0));
  }
  __syncthreads();

  // granted: not ruled out, and the stack reaches to its last new page
  auto granted = [&](int b) {
    return !(cu[b] & kRefused) && (pc[b + 1] == pc[b] || pc[b + 1] <= static_cast<unsigned>(n_free));
  };
  // unsigned: the last step past max_tokens must not overflow
  const unsigned first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;

  for (unsigned t = first; t < static_cast<unsigned>(a.max_tokens); t += step) {
    int slot = -1, pos = -1;
    if (t < cu[a.B]) {
      const int b = owner(cu, a.B, t);
      if (granted(b)) {
        const int len = max(a.lens[b], 0);
        pos = len + static_cast<int>(t - cu[b]);
        const int block = pos >> a.page_shift;
        const int fresh = block - static_cast<int>((static_cast<unsigned>(len) + page - 1) >> a.page_shift);
        const int id = fresh < 0 ? a.block_table[static_cast<long long>(b) * a.max_blocks + block]
                                 : a.free_pages[n_free - 1 - static_cast<int>(pc[b]) - fresh];
        if (id >= 0 && id < a.n_pages) slot = (id << a.page_shift) + (pos & (page - 1));
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }

  const unsigned n_taken = min(pc[a.B], static_cast<unsigned>(n_free));  // pages that may be taken
  for (unsigned j = first; j < n_taken; j += step) {
    const int b = owner(pc, a.B, j);
    if (!granted(b)) continue;  // the request that the stack does not reach
    const int have = static_cast<int>((static_cast<unsigned>(max(a.lens[b], 0)) + page - 1) >> a.page_shift);
    a.block_table[static_cast<long long>(b) * a.max_blocks + have + static_cast<int>(j - pc[b])] =
        a.free_pages[n_free - 1 - static_cast<int>(j)];
  }

  for (int b = static_cast<int>(first); b < a.B; b += static_cast<int>(step)) {
    const int len = max(a.lens[b], 0);
    const bool ok = granted(b);
    a.seqlens[b] = ok ? len + max(a.n_new[b], 0) : len;
    a.cu_new[b] = static_cast<int>(cu[b] & ~kRefused);
    // the last granted request that takes pages is the one behind which the sum first passes the stack,
    // or the last one of all: it says what is left
    if (ok && pc[b + 1] > pc[b] && (pc[b + 1] == pc[a.B] || !granted(owner(pc, a.B, pc[b + 1]))))
      *a.n_left = n_free - static_cast<int>(pc[b + 1]);
  }
  if (first == 0) {
    a.cu_new[a.B] = static_cast<int>(cu[a.B]);
    if (pc[a.B] == 0u || !granted(owner(pc, a.B, 0u))) *a.n_left = n_free;  // no page is taken
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t st, int* launches) {
  const size_t smem = 2 * sizeof(unsigned) * (static_cast<size_t>(a.B) + 1);
  if (smem > 48 * 1024) {  // above the default: opt in
    const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * static_cast<int>(sizeof(unsigned)) * (kMaxPlanRequests + 1));
    if (e != cudaSuccess) return e;
  }
  const int threads = a.B <= 256 && a.max_tokens <= 1024 ? 256 : 1024;
  long long blocks = (static_cast<long long>(a.max_tokens) + 2 * threads - 1) / (2 * threads);
  if (a.max_tokens <= 1024) blocks = 1;
  if (blocks > 152) blocks = 152;
  page_plan_kernel<<<static_cast<unsigned>(blocks), threads, smem, st>>>(a);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace attn
