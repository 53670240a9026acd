// decode_paged.cu - single-token decode over a paged KV cache on CUDA cores: any
// head dims, fp32 and bf16, alone or behind a prefix that the batch shares; and
// the combine of the partial results.
//
// The keys of a request are its prefix [0, P) (P = prefix_len, the same pages for
// the whole batch; 0 without one) and its own [P, L).  softmax(q K^T) V over a
// union of key ranges is the weighted mean of the ranges' results,
//   lse = log2 sum_j 2^lse_j,   O = sum_j 2^(lse_j - lse) O_j
// ("Transformer架构完全深度解析" §13's running sum, written for whole ranges), so
// the prefix is computed once: its rows are the B * G query rows of a KV head
// (G = n_h / n_kv, row r = request r / G, head r mod G of the group), each group
// of HG rows sharing the key rows that it loads.  A request's own keys are
// computed for HG heads of its group at a time.
//
// One block per (HG rows, KV head, chunk of kChunk keys): a half-warp covers one
// key row with 16-byte loads, NB rows per step; the scores are reduced across the
// half-warp by shuffles and folded into a running maximum and sum per row (fp32
// throughout); the 16 half-warps merge in shared memory and the block writes one
// normalised partial per row.  The chunk's page indices are staged in shared
// memory, so that a key row costs no dependent load from the table.
// This is the path of the shapes the tensor cores do not take; it is bound by HBM
// (few rows) or the fp32 pipes (many rows behind a prefix).
#include <math.h>

#include "kernels.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kMinPageShift = 4;
constexpr int kMaxChunk = 4096;

// How the call is cut: chunk keys per block, slots of partials per row.
struct Plan {
  int chunk, n_pre, n_own;  // n_pre chunks of the prefix, then n_own of a request's own keys
  __host__ __device__ int slots() const { return n_pre + n_own; }
};

// 8 consecutive elements as stored, and their fp32 values.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float* f) const { bf16x8_to_f32(u, f); }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void unpack(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// NQC / NVC: 128-dim column groups of the keys / values; HG rows per block; PREFIX: the shared part.
template <typename T, int NQC, int NVC, int HG, int NB, bool PREFIX>
__global__ void __launch_bounds__(kThreads) paged_split_kernel(PagedDecodeArgs a, RopeFreq f, Plan plan) {
  extern __shared__ float smem[];
  float* q_s = smem;                                   // [HG][NQC*128]
  float* red_o = q_s + HG * NQC * 128;                 // [16][HG][NVC*128]
  float* red_m = red_o + kHalfWarps * HG * NVC * 128;  // [16][HG]
  float* red_l = red_m + kHalfWarps * HG;              // [16][HG]
  __shared__ int pages[kMaxChunk >> kMinPageShift];

  const int G = a.n_h / a.n_kv;
  const int n_rows = PREFIX ? a.B * G : G;  // rows of a KV head that see these keys
  const int n_hg = (n_rows + HG - 1) / HG;
  // the chunk varies slowest: blocks that run together share a KV head's keys in L2
  long long u = blockIdx.x;
  const int r0 = static_cast<int>(u % n_hg) * HG;
  u /= n_hg;
  const int g = static_cast<int>(u % a.n_kv);
  u /= a.n_kv;
  const int b0 = PREFIX ? 0 : static_cast<int>(u % a.B);
  const int split = static_cast<int>(PREFIX ? u : u / a.B);
  // keys [start, end): of the prefix, or of request b0's own
  const int lo = PREFIX ? 0 : a.prefix_len, hi = PREFIX ? a.prefix_len : paged_len(a, b0);
  const long long start_ll = lo + static_cast<long long>(split) * plan.chunk;
  if (start_ll >= hi) return;  // nothing here: the combine pass never reads this partial
  const int start = static_cast<int>(start_ll);
  const int end = static_cast<int>(min(static_cast<long long>(hi), start_ll + plan.chunk));
  const int* table = PREFIX ? a.prefix_pages : a.block_table + static_cast<long long>(b0) * a.max_blocks;
  const int page0 = start >> a.page_shift;  // start is the first token of a page
  for (int i = threadIdx.x; i < ((end - 1) >> a.page_shift) - page0 + 1; i += kThreads) pages[i] = table[page0 + i];

  auto row_b = [&](int i) { return PREFIX ? (r0 + i) / G : b0; };
  auto row_h = [&](int i) { return g * G + (PREFIX ? (r0 + i) % G : r0 + i); };

  // rotated, pre-scaled queries of the rows, at each row's own position
  for (int idx = threadIdx.x; idx < HG * (NQC * 64); idx += kThreads) {
    const int i = idx / (NQC * 64), p = idx % (NQC * 64);
    const int j = p - a.rope_offset / 2;
    const bool rot = j >= 0 && j < f.n_pairs;
    int2 d = make_int2(2 * p, 2 * p + 1);
    if (rot) {
      d = rope_pair_dims(f, j);
      d.x += a.rope_offset;
      d.y += a.rope_offset;
    }
    float x0 = 0.f, x1 = 0.f;
    if (2 * p < a.D_qk && r0 + i < n_rows) {
      const int b = row_b(i);
      const T* qr = static_cast<const T*>(a.q) + (static_cast<long long>(b) * a.n_h + row_h(i)) * a.D_qk;
      x0 = to_f32(qr[d.x]);
      x1 = to_f32(qr[d.y]);
      if (rot) {
        float s, c;
        rope_sincos(max(paged_len(a, b), 1) - 1, f.hi[j], f.lo[j], &s, &c);
        rotate_pair(x0, x1, s, c);
      }
    }
    q_s[i * NQC * 128 + d.x] = x0 * a.scale_log2;
    q_s[i * NQC * 128 + d.y] = x1 * a.scale_log2;
  }
  __syncthreads();

  const int hw = threadIdx.x >> 4, hl = threadIdx.x & 15;
  float qr[HG][NQC][8];
#pragma unroll
  for (int i = 0; i < HG; ++i)
#pragma unroll
    for (int c = 0; c < NQC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) qr[i][c][e] = q_s[i * NQC * 128 + c * 128 + hl * 8 + e];

  float o[HG][NVC][8];
  float m_run[HG], l_run[HG];
#pragma unroll
  for (int i = 0; i < HG; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NVC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[i][c][e] = 0.f;
  }

  const long long k_tok = static_cast<long long>(a.n_kv) * a.D_qk;
  const T* kb = static_cast<const T*>(a.k_pages) + static_cast<long long>(g) * a.D_qk;
  const T* vb = static_cast<const T*>(a.v_pages) + static_cast<long long>(g) * a.D_v;
  const int row_mask = (1 << a.page_shift) - 1;

  // A warp takes 2*NB consecutive keys per step (NB per half-warp); the trip count is uniform
  // across the warp so the full-mask shuffles are legal.
  const int warp = threadIdx.x >> 5;
  for (int base = start + warp * 2 * NB; base < end; base += (kThreads / 32) * 2 * NB) {
    const int key0 = base + (hw & 1) * NB;
    Raw8<T> kr[NB][NQC], vr[NB][NVC];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int key = key0 + j;
      int page = -1;
      if (key < end) page = pages[(key >> a.page_shift) - page0];
      const bool ok = page >= 0 && page < a.n_pages;  // keys of a page outside the cache read as zero
      const long long slot = (static_cast<long long>(page) << a.page_shift) + (key & row_mask);
#pragma unroll
      for (int c = 0; c < NQC; ++c) {
        const int d = c * 128 + hl * 8;
        if (ok && d < a.D_qk) kr[j][c].load(kb + slot * k_tok + d);
        else kr[j][c].zero();
      }
#pragma unroll
      for (int c = 0; c < NVC; ++c) {
        const int d = c * 128 + hl * 8;
        if (ok && d < a.D_v) vr[j][c].load(vb + slot * a.v_token_stride + d);
        else vr[j][c].zero();
      }
    }
    float s[NB][HG];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int i = 0; i < HG; ++i) s[j][i] = 0.f;
#pragma unroll
      for (int c = 0; c < NQC; ++c) {
        float kf[8];
        kr[j][c].unpack(kf);
#pragma unroll
        for (int i = 0; i < HG; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[j][i] = fmaf(qr[i][c][e], kf[e], s[j][i]);
      }
#pragma unroll
      for (int i = 0; i < HG; ++i) {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) s[j][i] += __shfl_xor_sync(0xffffffffu, s[j][i], off);
        if (key0 + j >= end) s[j][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < HG; ++i) {
      float mx = s[0][i];
#pragma unroll
      for (int j = 1; j < NB; ++j) mx = fmaxf(mx, s[j][i]);
      const float m_new = fmaxf(m_run[i], mx);
      // -inf only while this half-warp has seen no key: weights stay 0
      const float m_ref = (m_new == -INFINITY) ? 0.f : m_new;
      const float alpha = fast_exp2(m_run[i] - m_ref);
      float psum = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        s[j][i] = fast_exp2(s[j][i] - m_ref);
        psum += s[j][i];
      }
      l_run[i] = l_run[i] * alpha + psum;
      m_run[i] = m_new;
#pragma unroll
      for (int c = 0; c < NVC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][c][e] *= alpha;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int c = 0; c < NVC; ++c) {
        float vf[8];
        vr[j][c].unpack(vf);
#pragma unroll
        for (int i = 0; i < HG; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[i][c][e] = fmaf(s[j][i], vf[e], o[i][c][e]);
      }
    }
  }

  // merge the 16 half-warps
#pragma unroll
  for (int i = 0; i < HG; ++i) {
    if (hl == 0) {
      red_m[hw * HG + i] = m_run[i];
      red_l[hw * HG + i] = l_run[i];
    }
#pragma unroll
    for (int c = 0; c < NVC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) red_o[(hw * HG + i) * NVC * 128 + c * 128 + hl * 8 + e] = o[i][c][e];
  }
  __syncthreads();
  const int ns = plan.slots();
  float* const ws_o = static_cast<float*>(a.workspace);
  float* const ws_lse = ws_o + static_cast<long long>(a.B) * a.n_h * ns * a.D_v;
  for (int idx = threadIdx.x; idx < HG * a.D_v; idx += kThreads) {
    const int i = idx / a.D_v, d = idx % a.D_v;
    if (r0 + i >= n_rows) continue;
    float M = -INFINITY;
    for (int w = 0; w < kHalfWarps; ++w) M = fmaxf(M, red_m[w * HG + i]);
    float num = 0.f, den = 0.f;
    for (int w = 0; w < kHalfWarps; ++w) {
      const float mw = red_m[w * HG + i];
      if (mw == -INFINITY) continue;  // this half-warp saw no key
      const float sc = fast_exp2(mw - M);
      num = fmaf(red_o[(w * HG + i) * NVC * 128 + d], sc, num);
      den = fmaf(red_l[w * HG + i], sc, den);
    }
    const long long slot = (static_cast<long long>(row_b(i)) * a.n_h + row_h(i)) * ns +
                           (PREFIX ? split : plan.n_pre + split);
    ws_o[slot * a.D_v + d] = den > 0.f ? num / den : 0.f;  // den = 0: every score is -inf, the weight is 0
    if (d == 0) ws_lse[slot] = M + log2f(den);
  }
}

// Four consecutive fp32 values stored as T.
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// One warp per (request b, head h): the written partials are the prefix's n_pre chunks and the
// first ceil((L - P) / chunk) of its own.  D_v <= 512, a multiple of 8: dims 4 lane + 128 c.
constexpr int kCombineWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kCombineWarps * 32) paged_combine_kernel(PagedDecodeArgs a, Plan plan) {
  const int lane = threadIdx.x & 31;
  const long long bh = static_cast<long long>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  if (bh >= static_cast<long long>(a.B) * a.n_h) return;  // whole warps only
  const int L = paged_len(a, static_cast<int>(bh / a.n_h));
  T* const out = static_cast<T*>(a.out) + bh * a.D_v;
  if (L <= a.prefix_len) {  // an empty place of the batch
    for (int d0 = 4 * lane; d0 < a.D_v; d0 += 128) store4<T>(out + d0, make_float4(0.f, 0.f, 0.f, 0.f));
    if (a.lse != nullptr && lane == 0) a.lse[bh] = -INFINITY;
    return;
  }
  const int ns = plan.slots();
  const int n = plan.n_pre + static_cast<int>((static_cast<long long>(L) - a.prefix_len + plan.chunk - 1) / plan.chunk);
  const float* const po = static_cast<const float*>(a.workspace) + bh * ns * a.D_v;
  const float* const lse = static_cast<const float*>(a.workspace) + static_cast<long long>(a.B) * a.n_h * ns * a.D_v +
                           bh * ns;
  float M = -INFINITY;
  for (int j = lane; j < n; j += 32) M = fmaxf(M, lse[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += 32) {
    const float wl = j0 + lane < n ? exp2f(lse[j0 + lane] - M) : 0.f;
    den += wl;
    const int nj = min(32, n - j0);
    for (int jj = 0; jj < nj; ++jj) {
      const float w = __shfl_sync(0xffffffffu, wl, jj);
      const float* pj = po + static_cast<long long>(j0 + jj) * a.D_v;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d0 = 4 * lane + 128 * c;
        if (d0 < a.D_v) {
          const float4 v = *reinterpret_cast<const float4*>(pj + d0);
          acc[c].x = fmaf(w, v.x, acc[c].x);
          acc[c].y = fmaf(w, v.y, acc[c].y);
          acc[c].z = fmaf(w, v.z, acc[c].z);
          acc[c].w = fmaf(w, v.w, acc[c].w);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  const float inv = 1.f / den;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int d0 = 4 * lane + 128 * c;
    if (d0 < a.D_v)
      store4<T>(out + d0, make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv));
  }
  if (a.lse != nullptr && lane == 0) a.lse[bh] = (M + log2f(den)) * 0.69314718055994530942f;
}

// Rows per block: more rows share each loaded K/V row, but every row costs registers for its
// query slice and output slice (as in decode.cu).
int pick_hg(int rows, int D_qk, int D_v) {
  if (D_qk > 256 || D_v > 256) return 1;
  if (D_qk <= 128 && D_v <= 128 && rows >= 3) return 4;
  return rows >= 2 ? 2 : 1;
}

// Keys per block: the smallest power of two from 256 that keeps the grid near 8192 blocks, at
// most kMaxChunk (the staged page indices).
Plan make_plan(const PagedDecodeArgs& a) {
  const int G = a.n_h / a.n_kv;
  const int hg = pick_hg(G, a.D_qk, a.D_v);
  const long long own = (static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len;  // keys at most
  const long long units = static_cast<long long>(a.B) * a.n_kv * ((G + hg - 1) / hg);
  Plan p;
  p.chunk = 256;
  while (p.chunk < kMaxChunk && p.chunk < own && units * ((own + p.chunk - 1) / p.chunk) > 8192) p.chunk *= 2;
  p.n_pre = (a.prefix_len + p.chunk - 1) / p.chunk;
  p.n_own = static_cast<int>((own + p.chunk - 1) / p.chunk);
  return p;
}

template <typename T, int NQC, int NVC, int HG, bool PREFIX>
cudaError_t launch_split(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st,
                         int* launches) {
  constexpr int NB = (NQC + NVC > 4) ? 2 : 4;
  const size_t smem = sizeof(float) * (HG * NQC * 128 + kHalfWarps * HG * NVC * 128 + 2 * kHalfWarps * HG);
  auto kern = paged_split_kernel<T, NQC, NVC, HG, NB, PREFIX>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int G = a.n_h / a.n_kv;
  const long long rows = PREFIX ? static_cast<long long>(a.B) * G : G;
  const long long grid = (rows + HG - 1) / HG * a.n_kv * (PREFIX ? plan.n_pre : static_cast<long long>(a.B) * plan.n_own);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a, f, plan);
  *launches += 1;
  return cudaGetLastError();
}

template <typename T, int NQC, int NVC, bool PREFIX>
cudaError_t launch_hg(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st, int* launches) {
  const int G = a.n_h / a.n_kv;
  const int hg = pick_hg(PREFIX ? (a.B < 4 ? a.B * G : 4) : G, a.D_qk, a.D_v);
  if constexpr (NQC + NVC <= 2) {
    if (hg == 4) return launch_split<T, NQC, NVC, 4, PREFIX>(a, f, plan, st, launches);
  }
  if constexpr (NQC + NVC <= 4) {
    if (hg >= 2) return launch_split<T, NQC, NVC, 2, PREFIX>(a, f, plan, st, launches);
  }
  return launch_split<T, NQC, NVC, 1, PREFIX>(a, f, plan, st, launches);
}

template <typename T, bool PREFIX>
cudaError_t launch_part(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st,
                        int* launches) {
  const int nq = (a.D_qk + 127) / 128, nv = (a.D_v + 127) / 128;
  if (nq == 1 && nv == 1) return launch_hg<T, 1, 1, PREFIX>(a, f, plan, st, launches);
  if (nq <= 2 && nv <= 2) return launch_hg<T, 2, 2, PREFIX>(a, f, plan, st, launches);
  return launch_hg<T, 5, 4, PREFIX>(a, f, plan, st, launches);
}

template <typename T>
cudaError_t launch_all(const PagedDecodeArgs& a, const RopeFreq& f, cudaStream_t st, int* launches) {
  const Plan plan = make_plan(a);
  if (a.prefix_len > 0) {
    const cudaError_t e = launch_part<T, true>(a, f, plan, st, launches);
    if (e != cudaSuccess) return e;
  }
  if (plan.n_own > 0) {  // none where the table has no block behind the prefix
    const cudaError_t e = launch_part<T, false>(a, f, plan, st, launches);
    if (e != cudaSuccess) return e;
  }
  const long long grid = (static_cast<long long>(a.B) * a.n_h + kCombineWarps - 1) / kCombineWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  paged_combine_kernel<T><<<static_cast<unsigned>(grid), kCombineWarps * 32, 0, st>>>(a, plan);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace

size_t decode_paged_workspace(const PagedDecodeArgs& a) {
  return sizeof(float) * static_cast<size_t>(a.B) * a.n_h * make_plan(a).slots() * (static_cast<size_t>(a.D_v) + 1);
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& a, const RopeFreq& rope, bool bf16, cudaStream_t st,
                                int* launches) {
  return bf16 ? launch_all<__nv_bfloat16>(a, rope, st, launches) : launch_all<float>(a, rope, st, launches);
}

}  // namespace attn
