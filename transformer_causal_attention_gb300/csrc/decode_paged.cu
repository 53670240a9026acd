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
// A block takes HG rows of a KV head and a run of keys: a half-warp covers one
// key row with 16-byte loads, NB rows per step; the scores are reduced across the
// half-warp by shuffles and folded into a running maximum and sum per row (fp32
// throughout); the 16 half-warps merge in shared memory and the block writes one
// normalised partial per row.  The run's page indices are staged in shared
// memory, so that a key row costs no dependent load from the table.
// The requests' own keys lie on one line of 64-key tiles, request after request,
// that is cut into equal parts, one per block (of each HG rows and KV head): the
// blocks find their parts from the lengths, so that neither the work's balance nor
// the number of partials depends on the table's width.  (Cut by the width, fp32, 8
// requests of up to 1024 keys took 11.1 us with a table of 1024 tokens and 19.6
// with one of 65536, now 10.9 and 11.3; and 1024 requests with tables of 131072
// tokens needed 541 MB for partials, now 18.)  A step to the next piece of a block's part raises the block's
// index or the request's, so their sum numbers the partials.
// Behind a prefix with 16 rows or more (and head dims up to 128) the shared part is a
// matrix product for the fp32 pipes instead: see paged_prefix_tile_kernel.
// This is the path of the shapes the tensor cores do not take.  fp32, 12 heads of
// 64 dims: 8 requests of up to 1024 keys 10.9 us, 6 behind 1024 shared tokens 17.5 us
// (two and three launches and their chains of dependent loads); 59 requests of 4096
// to 8192 keys, 32 heads over 8, D = 128: 592 us in fp32 (5.0 TB/s), 380 in bf16 with
// D = 96; 256 requests behind 2048 tokens, 40 heads over 8, D = 128: 535 us.
#include <math.h>

#include "kernels.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kMinPageShift = 4;
constexpr int kMaxRun = 4096;  // keys whose page indices are staged at a time (whole pages)

constexpr int kMinLineShift = 6;  // log2 of the line's tiles, in keys

// How the call is cut, and where its partials lie.
struct Plan {
  int pre_chunk, n_pre;    // the prefix: n_pre runs of pre_chunk keys
  int line_shift;          // own keys: log2 of the line's tiles (more keys only where 32 bits could not count tiles)
  int parts;               // parts of the line
  int blocks;              // blocks per (HG rows, KV head): parts that a table of this size can have
  // float offsets into the workspace: partial outputs and log-sum-exps of the prefix [B, n_h, n_pre] and of the
  // pieces [blocks + B, n_h], then (int) B + 1 sums of tiles
  long long own_o, pre_l, own_l, sums, end;
};

// Tiles of request b's own keys.
__device__ __forceinline__ int line_tiles(const PagedDecodeArgs& a, const Plan& p, int b) {
  const int own = paged_len(a, b) - a.prefix_len;
  return own > 0 ? ((own - 1) >> p.line_shift) + 1 : 0;
}

// Tiles of a part of a line of `total`.
__device__ __forceinline__ int part_tiles(const Plan& p, int total) {
  const unsigned n = p.parts;
  return max(1, static_cast<int>((static_cast<unsigned>(total) + n - 1u) / n));
}

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

// Part w of the line: the request and tile that it begins with, and its tiles (0: the line is shorter).  Every warp
// finds it for itself, without a barrier; the publishing block leaves the sums for the combine kernel.
struct Part {
  int b, t, left;
};
__device__ __forceinline__ Part find_part(const PagedDecodeArgs& a, const Plan& plan, int w, bool publish) {
  const int lane = threadIdx.x & 31;
  // lane i sums the tiles of requests [i s, (i + 1) s)
  const int strip = (a.B - 1) / 32 + 1;
  const int b_lo = static_cast<int>(min(static_cast<long long>(a.B), static_cast<long long>(lane) * strip));
  const int b_hi = b_lo + min(a.B - b_lo, strip);
  int mine = 0;
#pragma unroll 8
  for (int b = b_lo; b < b_hi; ++b) mine += line_tiles(a, plan, b);
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  const int part = part_tiles(plan, total);
  const long long x = static_cast<long long>(w) * part;
  int at_b = b_lo, at_t = 0;
  const bool here = x >= before && x < before + static_cast<long long>(mine);
  if (here) {
    at_t = static_cast<int>(x) - before;
    for (int n; at_b < b_hi - 1 && at_t >= (n = line_tiles(a, plan, at_b)); ++at_b) at_t -= n;
  }
  const int from = max(__ffs(__ballot_sync(0xffffffffu, here)) - 1, 0);
  at_b = __shfl_sync(0xffffffffu, at_b, from);
  at_t = __shfl_sync(0xffffffffu, at_t, from);
  if (publish && threadIdx.x < 32) {
    int* const sums = reinterpret_cast<int*>(static_cast<float*>(a.workspace) + plan.sums);
    for (int b = b_lo; b < b_hi; ++b) {
      sums[b] = before;
      before += line_tiles(a, plan, b);
    }
    if (lane == 0) sums[a.B] = total;
  }
  return Part{at_b, at_t, x < total ? static_cast<int>(min(static_cast<long long>(part), total - x)) : 0};
}

// The first request from b on that has own keys, a.B without one; every warp finds it for itself.
__device__ __forceinline__ int next_live(const PagedDecodeArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  for (; b < a.B; b += 32) {
    const uint32_t live = __ballot_sync(0xffffffffu, b + lane < a.B && paged_len(a, b + lane) > a.prefix_len);
    if (live) return b + __ffs(live) - 1;
  }
  return a.B;
}

// A later run's normalised result and log-sum-exp (base 2), merged with those of the runs before.
__device__ __forceinline__ float merge_weights(float lse_before, float* lse, float* w_before) {
  const float m = fmaxf(lse_before, *lse), m_ref = m == -INFINITY ? 0.f : m;
  const float x = exp2f(lse_before - m_ref), y = exp2f(*lse - m_ref), sum = x + y;
  const float inv = sum > 0.f ? 1.f / sum : sum;  // 0: every score is -inf; NaN stays
  *lse = m_ref + log2f(sum);
  *w_before = x * inv;
  return y * inv;
}
__device__ __forceinline__ void merge_partial(float before, float lse_before, float* out, float* lse) {
  float x;
  const float y = merge_weights(lse_before, lse, &x);
  *out = fmaf(x, before, y * *out);
}

// NQC / NVC: 128-dim column groups of the keys / values; HG rows per block; PREFIX: the shared part.
template <typename T, int NQC, int NVC, int HG, int NB, bool PREFIX>
__global__ void __launch_bounds__(kThreads) paged_split_kernel(PagedDecodeArgs a, RopeFreq f, Plan plan) {
  extern __shared__ float smem[];
  float* q_s = smem;                                   // [HG][NQC*128]
  float* red_o = q_s + HG * NQC * 128;                 // [16][HG][NVC*128]
  float* red_m = red_o + kHalfWarps * HG * NVC * 128;  // [16][HG]
  float* red_l = red_m + kHalfWarps * HG;              // [16][HG]
  __shared__ int pages[(kMaxRun >> kMinPageShift) + 1];

  const int G = a.n_h / a.n_kv;
  const int n_rows = PREFIX ? a.B * G : G;  // rows of a KV head that see these keys
  const int n_hg = (n_rows + HG - 1) / HG;
  // the run of keys varies slowest: blocks that run together share a KV head's keys in L2
  const int r0 = static_cast<int>(blockIdx.x % n_hg) * HG;
  const int g = static_cast<int>(blockIdx.x / n_hg % a.n_kv);
  const int w = static_cast<int>(blockIdx.x / n_hg / a.n_kv);
  Part part{0, 0, 0};
  if (!PREFIX) {
    part = find_part(a, plan, w, blockIdx.x == 0);
    if (part.left == 0) return;
  }
  // A piece is a run of the prefix, or what a request has in this part of the line.  More than kMaxRun keys of it are
  // computed that many at a time, so that no fp32 sum gets long, and merged with what was computed before.
  __shared__ float run_lse[2][HG];
  int at = 0, n_run = 0;  // the piece's next key, and which run of it begins there
  if (PREFIX) at = w * plan.pre_chunk;
  else at = a.prefix_len + (part.t << plan.line_shift);
  for (;;) {
    const int b0 = PREFIX ? 0 : part.b;
    int stop;  // the piece's end
    if (PREFIX) {
      stop = w * plan.pre_chunk + min(a.prefix_len - w * plan.pre_chunk, plan.pre_chunk);
    } else {
      const long long x = (static_cast<long long>(part.t) + part.left) << plan.line_shift;
      stop = a.prefix_len + static_cast<int>(min(static_cast<long long>(paged_len(a, b0) - a.prefix_len), x));
    }
    const int start = at, end = start + min(stop - start, kMaxRun);
    const int* table = PREFIX ? a.prefix_pages : a.block_table + static_cast<long long>(b0) * a.max_blocks;
    const int page0 = start >> a.page_shift;
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
          const int pos = max(paged_len(a, b), 1) - 1;
          float s, c;
          if (rope_is_far(pos)) rope_sincos_far(pos, f.hi[j], f.lo[j], &s, &c);
          else rope_sincos(pos, f.hi[j], f.lo[j], &s, &c);
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
    float* const ws = static_cast<float*>(a.workspace);
    for (int idx = threadIdx.x; idx < HG * a.D_v; idx += kThreads) {
      const int i = idx / a.D_v, d = idx % a.D_v;
      if (r0 + i >= n_rows) continue;
      float M = -INFINITY;
      for (int hw = 0; hw < kHalfWarps; ++hw) M = fmaxf(M, red_m[hw * HG + i]);
      const float m_ref = M == -INFINITY ? 0.f : M;
      float num = 0.f, den = 0.f;
      for (int hw = 0; hw < kHalfWarps; ++hw) {
        // 0 for a half-warp that saw no key; NaN in its sums stays
        const float sc = fast_exp2(red_m[hw * HG + i] - m_ref);
        num = fmaf(red_o[(hw * HG + i) * NVC * 128 + d], sc, num);
        den = fmaf(red_l[hw * HG + i], sc, den);
      }
      const long long slot = PREFIX ? (static_cast<long long>(row_b(i)) * a.n_h + row_h(i)) * plan.n_pre + w
                                    : (static_cast<long long>(w) + b0) * a.n_h + row_h(i);
      float* const o_out = ws + (PREFIX ? 0 : plan.own_o) + slot * a.D_v + d;
      float out = den > 0.f ? num / den : den;  // 0: every score is -inf, the weight is 0; NaN stays
      float lse = M + log2f(den);
      if (n_run > 0) merge_partial(*o_out, run_lse[(n_run - 1) & 1][i], &out, &lse);
      *o_out = out;
      if (d == 0) {
        ws[(PREFIX ? plan.pre_l : plan.own_l) + slot] = lse;
        run_lse[n_run & 1][i] = lse;
      }
    }
    if (end < stop) {
      at = end;
      ++n_run;
      continue;
    }
    if (PREFIX) return;
    part.left -= line_tiles(a, plan, b0) - part.t;
    if (part.left <= 0) return;
    part.b = next_live(a, b0 + 1);
    if (part.b == a.B) return;
    part.t = n_run = 0;
    at = a.prefix_len;
  }
}

// The shared part for many rows: one block per (64 rows of a KV head, chunk of keys), 64 keys at a time
// through shared memory.  S = Q K^T and O += P V are register tiles of 4 x 4 and 4 x (DM / 16) per
// thread, fed by 16-byte loads of transposed tiles (Q^T and K^T by dim, P^T by key), with packed fp32
// FMAs; a row's 16 threads sit in one half-warp, so its maximum takes four shuffles.  K and V take turns
// in one buffer, which lets two blocks share an SM and cover each other's loads.  Bound by the loads from
// shared memory (two thirds of their rate; warps wait for them more than for anything else, the FMA pipes are
// 39% busy): 256 requests behind 16384 tokens, 32 heads over 8, D = 128, take 2256 us, 30 TFLOP/s; the split
// kernel above, with a shuffle per 8 FMAs and a load of every key per 4 rows, took 5275.
constexpr int kTile = 64;           // rows and keys
constexpr int kPad = kTile + 4;     // row stride of the transposed tiles, in floats
constexpr int kTileMinRows = 16;    // below, the split kernel's 4 rows per block waste less

template <int DM> constexpr int prefix_tile_smem() {
  constexpr int kv = DM * kPad > kTile * (DM + 4) ? DM * kPad : kTile * (DM + 4);
  return (DM * kPad + kv + kTile * kPad) * static_cast<int>(sizeof(float));
}

template <typename T, int DM>
__global__ void __launch_bounds__(kThreads, 2)
    paged_prefix_tile_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ RopeFreq f, Plan plan) {
  constexpr int VD = DM / 16;  // value dims per thread
  extern __shared__ float smem[];
  float* const q_t = smem;                                  // [DM][kPad]: rotated, scaled queries by dim
  float* const kv = q_t + DM * kPad;                        // K^T [DM][kPad], then V [64][DM + 4]
  float* const p_t = kv + (DM * kPad > kTile * (DM + 4) ? DM * kPad : kTile * (DM + 4));  // P^T [64 keys][kPad]
  __shared__ int pages[(kMaxRun >> kMinPageShift) + 1];

  const int G = a.n_h / a.n_kv, n_rows = a.B * G;
  const int n_rt = (n_rows + kTile - 1) / kTile;
  const int rt = blockIdx.x % n_rt, g = blockIdx.x / n_rt % a.n_kv, split = blockIdx.x / n_rt / a.n_kv;
  const int r0 = rt * kTile;
  const int first = split * plan.pre_chunk, last = min(a.prefix_len - first, plan.pre_chunk) + first;

  for (int idx = threadIdx.x; idx < kTile * (DM / 2); idx += kThreads) {
    const int i = idx % kTile, p = idx / kTile;
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
      const int b = (r0 + i) / G, h = g * G + r0 + i - b * G;
      const T* qr = static_cast<const T*>(a.q) + (static_cast<long long>(b) * a.n_h + h) * a.D_qk;
      x0 = to_f32(qr[d.x]);
      x1 = to_f32(qr[d.y]);
      if (rot) {
        const int pos = max(paged_len(a, b), 1) - 1;
        float s, c;
        if (rope_is_far(pos)) rope_sincos_far(pos, f.hi[j], f.lo[j], &s, &c);
        else rope_sincos(pos, f.hi[j], f.lo[j], &s, &c);
        rotate_pair(x0, x1, s, c);
      }
    }
    q_t[d.x * kPad + i] = x0 * a.scale_log2;
    q_t[d.y * kPad + i] = x1 * a.scale_log2;
  }

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // keys 4 tx .. and dims VD tx .. of rows 4 ty ..
  const long long k_tok = static_cast<long long>(a.n_kv) * a.D_qk;
  const T* const kb = static_cast<const T*>(a.k_pages) + static_cast<long long>(g) * a.D_qk;
  const T* const vb = static_cast<const T*>(a.v_pages) + static_cast<long long>(g) * a.D_v;
  const int row_mask = (1 << a.page_shift) - 1;
  float lse_before[4];
  // more than kMaxRun keys in runs, each merged with those before (as in the split kernel)
  for (int start = first, end; start < last; start = end) {
    end = start + min(last - start, kMaxRun);
    const int page0 = start >> a.page_shift;
    // (the run before has read its last page indices before its last barrier)
    for (int i = threadIdx.x; i < ((end - 1) >> a.page_shift) - page0 + 1; i += kThreads)
      pages[i] = a.prefix_pages[page0 + i];
    auto slot_of = [&](int key) -> long long {  // -1: behind the run, or in a page outside the cache (zeros)
      if (key >= end) return -1;
      const int page = pages[(key >> a.page_shift) - page0];
      return page >= 0 && page < a.n_pages ? (static_cast<long long>(page) << a.page_shift) + (key & row_mask) : -1;
    };

    float2 o[4][VD / 2];
    float m_run[4], l_part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m_run[i] = -INFINITY;
      l_part[i] = 0.f;
#pragma unroll
      for (int e = 0; e < VD / 2; ++e) o[i][e] = make_float2(0.f, 0.f);
    }
    for (int k0 = start; k0 < end; k0 += kTile) {
      __syncthreads();  // the tile before has been read (and, the first time, the pages and queries are there)
#pragma unroll 2
      for (int idx = threadIdx.x; idx < kTile * (DM / 8); idx += kThreads) {
        const int key = idx % kTile, c = idx / kTile;
        const long long slot = slot_of(k0 + key);
        Raw8<T> raw;
        if (slot >= 0 && c * 8 < a.D_qk) raw.load(kb + slot * k_tok + c * 8);
        else raw.zero();
        float x[8];
        raw.unpack(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) kv[(c * 8 + e) * kPad + key] = x[e];
      }
      __syncthreads();
      float2 s2[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) s2[i][0] = s2[i][1] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < DM; ++d) {
        const float4 q4 = *reinterpret_cast<const float4*>(q_t + d * kPad + 4 * ty);
        const float4 k4 = *reinterpret_cast<const float4*>(kv + d * kPad + 4 * tx);
        const float2 ka = make_float2(k4.x, k4.y), kc = make_float2(k4.z, k4.w);
        const float q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 qq = make_float2(q[i], q[i]);
          s2[i][0] = __ffma2_rn(qq, ka, s2[i][0]);
          s2[i][1] = __ffma2_rn(qq, kc, s2[i][1]);
        }
      }
      float p[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i][0] = s2[i][0].x;
        p[i][1] = s2[i][0].y;
        p[i][2] = s2[i][1].x;
        p[i][3] = s2[i][1].y;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k0 + 4 * tx + e >= end) p[i][e] = -INFINITY;
        float mx = fmaxf(fmaxf(p[i][0], p[i][1]), fmaxf(p[i][2], p[i][3]));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float m_new = fmaxf(m_run[i], mx);
        const float m_ref = m_new == -INFINITY ? 0.f : m_new;  // every score so far is -inf: weights 0
        const float alpha = fast_exp2(m_run[i] - m_ref);
        m_run[i] = m_new;
        l_part[i] *= alpha;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[i][e] = fast_exp2(p[i][e] - m_ref);
          l_part[i] += p[i][e];
        }
#pragma unroll
        for (int e = 0; e < VD / 2; ++e) o[i][e] = make_float2(o[i][e].x * alpha, o[i][e].y * alpha);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(p_t + (4 * tx + e) * kPad + 4 * ty) =
            make_float4(p[0][e], p[1][e], p[2][e], p[3][e]);
      __syncthreads();  // K^T has been read, P^T is whole
#pragma unroll 2
      for (int idx = threadIdx.x; idx < kTile * (DM / 8); idx += kThreads) {
        const int key = idx / (DM / 8), c = idx % (DM / 8);
        const long long slot = slot_of(k0 + key);
        Raw8<T> raw;
        if (slot >= 0 && c * 8 < a.D_v) raw.load(vb + slot * a.v_token_stride + c * 8);
        else raw.zero();
        float x[8];
        raw.unpack(x);
        float4* const dst = reinterpret_cast<float4*>(kv + key * (DM + 4) + c * 8);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
      __syncthreads();
#pragma unroll 4
      for (int j = 0; j < kTile; ++j) {
        const float4 p4 = *reinterpret_cast<const float4*>(p_t + j * kPad + 4 * ty);
        const float pj[4] = {p4.x, p4.y, p4.z, p4.w};
        float2 v[VD / 2];
#pragma unroll
        for (int e = 0; e < VD / 4; ++e) {
          const float4 x = *reinterpret_cast<const float4*>(kv + j * (DM + 4) + VD * tx + 4 * e);
          v[2 * e] = make_float2(x.x, x.y);
          v[2 * e + 1] = make_float2(x.z, x.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 pp = make_float2(pj[i], pj[i]);
#pragma unroll
          for (int e = 0; e < VD / 2; ++e) o[i][e] = __ffma2_rn(pp, v[e], o[i][e]);
        }
      }
    }

    float* const ws = static_cast<float*>(a.workspace);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float l = l_part[i];
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const int r = r0 + 4 * ty + i;
      if (r >= n_rows) continue;
      const int b = r / G, h = g * G + r - b * G;
      const long long slot = (static_cast<long long>(b) * a.n_h + h) * plan.n_pre + split;
      float inv = l > 0.f ? 1.f / l : l;  // 0: every score is -inf, the weight is 0; NaN stays
      float lse = m_run[i] + log2f(l), x = 0.f;
      if (start > first) inv *= merge_weights(lse_before[i], &lse, &x);
      lse_before[i] = lse;
#pragma unroll
      for (int e = 0; e < VD / 2; ++e) {
        const int d = VD * tx + 2 * e;
        if (d >= a.D_v) continue;
        float2* const p = reinterpret_cast<float2*>(ws + slot * a.D_v + d);
        float2 v = make_float2(o[i][e].x * inv, o[i][e].y * inv);
        if (start > first) v = make_float2(fmaf(x, p->x, v.x), fmaf(x, p->y, v.y));
        *p = v;
      }
      if (tx == 0) ws[plan.pre_l + slot] = lse;
    }
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

// The partials of a (request b, head h) are the prefix's n_pre runs and the pieces of the parts of the line that
// hold its own tiles.  A warp per row takes them kBatch at a time, its lanes four dims
// at 4 lane + 128 c (D_v <= 512, a multiple of 8); SPLIT: the eight warps of a block take every eighth
// partial of one row each and merge in shared memory, for rows in many partials.
constexpr int kCombineWarps = 8;
constexpr int kBatch = 4;

template <typename T, bool SPLIT>
__global__ void __launch_bounds__(kCombineWarps * 32) paged_combine_kernel(PagedDecodeArgs a, Plan plan) {
  __shared__ float red_o[SPLIT ? kCombineWarps * 512 : 1];
  __shared__ float red_m[kCombineWarps], red_l[kCombineWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long bh = SPLIT ? blockIdx.x : static_cast<long long>(blockIdx.x) * kCombineWarps + warp;
  if (bh >= static_cast<long long>(a.B) * a.n_h) return;  // whole warps only
  const int b = static_cast<int>(bh / a.n_h);
  const float* const ws = static_cast<const float*>(a.workspace);
  const int* const sums = reinterpret_cast<const int*>(ws + plan.sums);
  // (loaded beside the length; not written, nor used, where no request can have own keys)
  const int t_all = sums[a.B], t0 = sums[b], t1 = sums[b + 1];
  const int L = paged_len(a, b);
  T* const out = static_cast<T*>(a.out) + bh * a.D_v;
  if (L <= a.prefix_len) {  // an empty place of the batch
    if (SPLIT && warp > 0) return;
    for (int d0 = 4 * lane; d0 < a.D_v; d0 += 128) store4<T>(out + d0, make_float4(0.f, 0.f, 0.f, 0.f));
    if (a.lse != nullptr && lane == 0) a.lse[bh] = -INFINITY;
    return;
  }
  const unsigned part = part_tiles(plan, t_all);
  const int w0 = static_cast<int>(static_cast<unsigned>(t0) / part);
  const int w1 = static_cast<int>((static_cast<unsigned>(t1) - 1u) / part);
  const int n = plan.n_pre + w1 - w0 + 1;
  const long long pre = bh * plan.n_pre, own = static_cast<long long>(w0 + b) * a.n_h + bh % a.n_h;
  auto slot = [&](int j) { return j < plan.n_pre ? pre + j : own + static_cast<long long>(j - plan.n_pre) * a.n_h; };
  const bool shared = SPLIT && n > kBatch;  // one warp takes a few partials at once
  if (SPLIT && !shared && warp > 0) return;
  const int step = shared ? kCombineWarps : 1;
  float M = -INFINITY, den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = SPLIT ? warp : 0; j0 < n; j0 += kBatch * step) {
    float l[kBatch];
    float4 v[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = j0 + k * step;
      l[k] = j < n ? ws[(j < plan.n_pre ? plan.pre_l : plan.own_l) + slot(j)] : -INFINITY;
      const float* const o = ws + (j < plan.n_pre ? 0 : plan.own_o) + slot(j) * a.D_v;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d0 = 4 * lane + 128 * c;
        v[k][c] = j < n && d0 < a.D_v ? *reinterpret_cast<const float4*>(o + d0)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) m = fmaxf(m, l[k]);
    const float m_ref = m == -INFINITY ? 0.f : m;  // every score so far is -inf: weights 0
    const float alpha = exp2f(M - m_ref);
    M = m;
    den *= alpha;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(acc[c].x * alpha, acc[c].y * alpha, acc[c].z * alpha, acc[c].w * alpha);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = exp2f(l[k] - m_ref);
      den += w;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[c] = make_float4(fmaf(w, v[k][c].x, acc[c].x), fmaf(w, v[k][c].y, acc[c].y), fmaf(w, v[k][c].z, acc[c].z),
                             fmaf(w, v[k][c].w, acc[c].w));
    }
  }
  if (shared) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(red_o + warp * 512 + 4 * lane + 128 * c) = acc[c];
    if (lane == 0) {
      red_m[warp] = M;
      red_l[warp] = den;
    }
    __syncthreads();
    if (warp > 0) return;
    M = -INFINITY;
    den = 0.f;
    for (int w = 0; w < kCombineWarps; ++w) M = fmaxf(M, red_m[w]);
    const float m_ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < kCombineWarps; ++w) {
      const float x = exp2f(red_m[w] - m_ref);
      den = fmaf(red_l[w], x, den);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(red_o + w * 512 + 4 * lane + 128 * c);
        acc[c] = make_float4(fmaf(x, v.x, acc[c].x), fmaf(x, v.y, acc[c].y), fmaf(x, v.z, acc[c].z), fmaf(x, v.w, acc[c].w));
      }
    }
  }
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

// Whether the shared part runs as 64 x 64 tiles.
bool prefix_tiles(const PagedDecodeArgs& a) {
  return a.D_qk <= 128 && a.D_v <= 128 && static_cast<long long>(a.B) * (a.n_h / a.n_kv) >= kTileMinRows;
}

// Rows per block of the prefix's split kernel.
int prefix_hg(const PagedDecodeArgs& a) {
  const long long rows = static_cast<long long>(a.B) * (a.n_h / a.n_kv);
  return pick_hg(rows < 4 ? static_cast<int>(rows) : 4, a.D_qk, a.D_v);
}

constexpr long long kWave = 304;  // two blocks per SM

// Cuts the prefix into runs of whole 64-key tiles for `units` blocks each: as short as a tile while that makes no more
// than `fill` blocks; runs of 256 keys and more as many as fill up to eight waves best.
int pick_runs(long long units, long long keys, int fill, int* run) {
  const auto up = [](long long x, long long y) { return (x + y - 1) / y; };
  const long long tiles = up(keys, kTile);
  long long best = kTile * up(tiles, up(fill, units));
  if (best >= 256) {
    best = kTile * tiles;
    double use = 0;
    for (int waves = 1; waves <= 8; ++waves) {
      long long n = waves * kWave / units;
      if (n > up(keys, 256)) n = up(keys, 256);
      if (n < 1) continue;
      const long long r = kTile * up(tiles, n);
      const double busy = static_cast<double>(units * tiles) / (up(units * up(keys, r), kWave) * kWave * r);
      if (busy > use) {
        use = busy;
        best = r;
      }
    }
  }
  *run = static_cast<int>(best < keys ? best : keys);
  return static_cast<int>(up(keys, *run));
}

// Parts of the line of own keys, for `columns` blocks each: one wave of blocks where that is nine tenths full, else
// two to four.  Equal parts need no more than one wave, and pieces cost less in few parts: fp32, 59 requests of 4096 to
// 8192 keys, 32 heads over 8: 592 us, 595 in two waves, 626 in six, 678 in twelve, 714 in runs of 512 keys; 64 of up to
// 1024 keys, 12 heads: 50, 53, 64 and 57.
int pick_parts(long long columns) {
  int best = 1;
  double use = 0;
  for (int waves = 1; waves <= 4 && use < 0.9; ++waves) {
    const long long n = waves * kWave / columns;
    const double busy = static_cast<double>(n * columns) / (waves * kWave);
    if (n > 0 && busy > use) {
      use = busy;
      best = static_cast<int>(n);
    }
  }
  return best;
}

Plan make_plan(const PagedDecodeArgs& a) {
  const int G = a.n_h / a.n_kv;
  const int hg = pick_hg(G, a.D_qk, a.D_v);
  const long long own = (static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len;  // keys at most
  const long long rows = static_cast<long long>(a.B) * G, heads = static_cast<long long>(a.B) * a.n_h;
  Plan p{};
  if (a.prefix_len > 0) {
    const bool tile = prefix_tiles(a);
    const int per_block = tile ? kTile : prefix_hg(a);
    p.n_pre = pick_runs((rows + per_block - 1) / per_block * a.n_kv, a.prefix_len, tile ? 152 : 304, &p.pre_chunk);
  }
  const long long columns = static_cast<long long>(a.n_kv) * ((G + hg - 1) / hg);
  p.parts = pick_parts(columns);
  // no more blocks than the table has tiles; which parts there are does not depend on it
  p.line_shift = kMinLineShift;
  auto tiles = [&] { return ((own + (1LL << p.line_shift) - 1) >> p.line_shift) * a.B; };
  while (tiles() > 0x7fffffffLL) ++p.line_shift;
  p.blocks = static_cast<int>(tiles() < p.parts ? tiles() : p.parts);
  const long long pieces = (static_cast<long long>(p.blocks) + a.B) * a.n_h;
  p.own_o = heads * p.n_pre * a.D_v;
  p.pre_l = p.own_o + pieces * a.D_v;
  p.own_l = p.pre_l + heads * p.n_pre;
  p.sums = p.own_l + pieces;
  p.end = p.sums + a.B + 1;
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
  const long long grid = (rows + HG - 1) / HG * a.n_kv * (PREFIX ? plan.n_pre : plan.blocks);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a, f, plan);
  *launches += 1;
  return cudaGetLastError();
}

template <typename T, int NQC, int NVC, bool PREFIX>
cudaError_t launch_hg(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st, int* launches) {
  const int G = a.n_h / a.n_kv;
  const int hg = PREFIX ? prefix_hg(a) : pick_hg(G, a.D_qk, a.D_v);
  if constexpr (NQC + NVC <= 2) {
    if (hg == 4) return launch_split<T, NQC, NVC, 4, PREFIX>(a, f, plan, st, launches);
  }
  if constexpr (NQC + NVC <= 4) {
    if (hg >= 2) return launch_split<T, NQC, NVC, 2, PREFIX>(a, f, plan, st, launches);
  }
  return launch_split<T, NQC, NVC, 1, PREFIX>(a, f, plan, st, launches);
}

template <typename T, int DM>
cudaError_t launch_prefix_tile(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st,
                               int* launches) {
  auto kern = paged_prefix_tile_kernel<T, DM>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, prefix_tile_smem<DM>());
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.B) * (a.n_h / a.n_kv);
  const long long grid = (rows + kTile - 1) / kTile * a.n_kv * plan.n_pre;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<static_cast<unsigned>(grid), kThreads, prefix_tile_smem<DM>(), st>>>(a, f, plan);
  *launches += 1;
  return cudaGetLastError();
}

template <typename T, bool PREFIX>
cudaError_t launch_part(const PagedDecodeArgs& a, const RopeFreq& f, const Plan& plan, cudaStream_t st,
                        int* launches) {
  if constexpr (PREFIX) {
    if (prefix_tiles(a))
      return a.D_qk <= 64 && a.D_v <= 64 ? launch_prefix_tile<T, 64>(a, f, plan, st, launches)
                                         : launch_prefix_tile<T, 128>(a, f, plan, st, launches);
  }
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
  if (plan.blocks > 0) {  // none where the table has no block behind the prefix
    const cudaError_t e = launch_part<T, false>(a, f, plan, st, launches);
    if (e != cudaSuccess) return e;
  }
  // eight warps per row where rows are few and may have many partials
  const long long rows = static_cast<long long>(a.B) * a.n_h;
  const bool split = rows <= 2432;
  const long long grid = split ? rows : (rows + kCombineWarps - 1) / kCombineWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (split)
    paged_combine_kernel<T, true><<<static_cast<unsigned>(grid), kCombineWarps * 32, 0, st>>>(a, plan);
  else
    paged_combine_kernel<T, false><<<static_cast<unsigned>(grid), kCombineWarps * 32, 0, st>>>(a, plan);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace

size_t decode_paged_workspace(const PagedDecodeArgs& a) {
  return sizeof(float) * static_cast<size_t>(make_plan(a).end);
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& a, const RopeFreq& rope, bool bf16, cudaStream_t st,
                                int* launches) {
  return bf16 ? launch_all<__nv_bfloat16>(a, rope, st, launches) : launch_all<float>(a, rope, st, launches);
}

}  // namespace attn
