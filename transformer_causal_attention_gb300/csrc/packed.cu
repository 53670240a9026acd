// packed.cu - attention of packed new tokens over a paged KV cache on CUDA cores: causal, or
// by visibility bits among drafted tokens (any head dims up to 640 / 512, bf16 or fp32).
//
// The rows of a KV head in request b are its n_b * G (token, head of the group) pairs, token
// after token; a block takes 64 of them against 64 keys at a time: S = Q K^T with 4 x 4 scores
// per thread, an online softmax over the rows ("Transformer架构完全深度解析" §13), O += P V with
// 4 rows x 4 dims per thread and 64 dims.  Everything is fp32; Q stays in shared memory
// (dim-major), K passes through it 32 dims at a time, P once per tile, V 64 dims at a time.
// Bound by the FMA pipe and the shared-memory reads that feed it (8 floats per 16 FMAs): bf16, D = 96, 3 prompts of
// 300 to 900 tokens, 32 heads over 8: 338 us, 23 TFLOP/s.
//
// Tiles are numbered without a table: request b's start at floor(cu_new[b] * G / 64) + b, which
// leaves each request at least as many numbers as it has tiles, so a block finds its request by
// bisection and a number that nobody uses ends at once.  Blocks start with the last tiles, which see the most keys,
// of all heads (head by head, one fp32 prompt of 2000 tokens of 8 heads took 293 us instead of 215).  With few tiles the keys
// of each are cut into equal parts and a second kernel joins the parts of a row by their log-sum-exps.
//
// fp32 with head dims up to 128 has a kernel of its own, packed_f32_kernel: the same tiles, but K and V in
// shared memory as they lie in the cache, copied asynchronously, and packed pairs of FMAs.  Where there is room, K and V have
// two stages, and a tile one barrier: 64 dims in two blocks per SM, 128 in one (with values of 64 dims or fewer and keys of
// more, one stage: K of the next tile comes while this one's P V runs, V while the next scores do).  8 prompts of up to 500
// tokens, 12 heads of 64 dims: 73 us, 17 TFLOP/s; 4 x 128 tokens behind 2000, 32 heads over 8 of 128 dims: 553 us, 31 TFLOP/s
// (one stage: 573).  A tile of 64 keys takes a block some 7 us, whether it has an SM for itself or shares it: its chain of
// shared-memory reads, FMAs and shuffles has too few warps to hide behind.  (Three blocks per SM spill; 8 x 4 scores per
// thread of 128 threads, and weights twice in shared memory so that they are read as pairs, were not faster.)
#include <math.h>

#include "kernels.h"

namespace attn {
namespace {

constexpr int R = 64;         // rows per tile
constexpr int KT = 64;        // keys per tile
constexpr int DC = 32;        // dims of K in shared memory at a time
constexpr int kPad = 4;       // floats behind a row of 64: float4 rows on other banks
constexpr int LD = 64 + kPad;
constexpr int kThreads = 256;
constexpr float kMasked = -1.f;  // stands for the weight of a key that the row does not see (weights are >= 0)

// 8 consecutive elements as floats.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ long long tile_start(const PackedArgs& a, int b, int G) {
  return static_cast<long long>(packed_first(a, b)) * G / R + b;
}

// A block's rows: the request, its rows row0 .. row0 + here - 1, and the keys [k_lo, k_hi) of this split.
struct Tile {
  int b, here;
  PackedRequest rq;
  long long row0;
  int k_lo, k_hi;
  int first_place;  // of its first row, -1 or more
  bool whole;       // one part: the rows go to the output
};
// Keys that a tile's last row may see, and keys in each of its parts.
__device__ __forceinline__ int keys_of(const PackedArgs& a, const PackedRequest& rq, long long last_row, int G) {
  const int last = rq.base + static_cast<int>(last_row / G);
  return a.visible != nullptr ? rq.len : min(max(last, -1) + 1, rq.len);
}
__device__ __forceinline__ int part_of(int keys, int n_split) {
  const int part = static_cast<int>((static_cast<long long>(keys) + n_split - 1) / n_split);
  return max((part + KT - 1) / KT, 1) * KT;
}
// Finds a block's tile and part (here = 0: none), and clears its share of the rows behind the last request's.  Blocks
// count from the last tile, which sees the most keys of its request, the KV heads of a tile side by side.
template <typename T>
__device__ __forceinline__ Tile find_tile(const PackedArgs& a, int g, int n_split) {
  const int tid = threadIdx.x, G = a.n_h / a.n_kv, split = blockIdx.y;
  const long long numbers = gridDim.x / a.n_kv, number = numbers - 1 - blockIdx.x / a.n_kv;
  if (split == 0) {
    const long long per = static_cast<long long>(G) * a.D_v;  // of a KV head and row
    const long long from = packed_first(a, a.B) * per, to = a.T * per;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long i = from + 4LL * (number * kThreads + tid); i < to; i += 4LL * numbers * kThreads) {
      const long long row = i / per, at = i - row * per, head = row * a.n_h + static_cast<long long>(g) * G;
      store4(static_cast<T*>(a.out) + head * a.D_v + at, zero);
      if (a.lse != nullptr && at % a.D_v == 0) a.lse[head + at / a.D_v] = -INFINITY;
    }
  }
  Tile t;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start(a, mid, G) <= number) lo = mid;
    else hi = mid - 1;
  }
  t.b = lo;
  t.rq = packed_request(a, lo);
  t.row0 = (number - tile_start(a, lo, G)) * R;
  const long long n_rows = static_cast<long long>(t.rq.rows) * G;
  t.here = t.row0 < 0 || t.row0 >= n_rows ? 0 : static_cast<int>(n_rows - t.row0 < R ? n_rows - t.row0 : R);
  if (t.here == 0) return t;
  const int keys = keys_of(a, t.rq, t.row0 + t.here - 1, G), part = part_of(keys, n_split);
  const long long k_lo = static_cast<long long>(split) * part;
  if (k_lo >= keys && split > 0) t.here = 0;
  t.whole = keys <= part;
  t.k_hi = static_cast<int>(k_lo + part < keys ? k_lo + part : keys);
  t.k_lo = static_cast<int>(k_lo < t.k_hi ? k_lo : t.k_hi);
  t.first_place = max(t.rq.base + static_cast<int>(t.row0 / G), -1);
  return t;
}
// A row of the tile: which (token, head) of q and out it is, the position at which it is rotated, and what it sees - its
// place (-1: nothing, and no rotation) and bits.  (Once per row: divisions by G at each use were a third of a tile's time.)
struct Rows {
  int at[R], pos[R], place[R];
  uint32_t vis[R][4];
};
__device__ __forceinline__ void load_row(const PackedArgs& a, const Tile& t, int g, int r, Rows* rows) {
  rows->place[r] = -1;
  if (r >= t.here) return;
  const int G = a.n_h / a.n_kv;
  const int i = static_cast<int>((t.row0 + r) / G), row = t.rq.first + i;
  rows->at[r] = row * a.n_h + g * G + static_cast<int>(t.row0 + r - static_cast<long long>(i) * G);
  const int place = t.rq.base + i, pos = a.positions != nullptr ? a.positions[row] : place;
  rows->pos[r] = pos;
  rows->place[r] = pos < 0 ? -1 : place;
  for (int w = 0; w < 4; ++w) rows->vis[r][w] = w < a.words ? static_cast<uint32_t>(a.visible[static_cast<long long>(row) * a.words + w]) : 0u;
}
__device__ __forceinline__ bool sees(const PackedArgs& a, const Tile& t, int place, const uint32_t* vis, int key) {
  if (a.visible == nullptr) return key < t.k_hi && key <= place;
  const int draft = key - t.rq.base;  // base may be below 0: key - base <= len - base = n
  return key < t.k_hi && place >= 0 && (draft < 0 || (draft < 32 * a.words && ((vis[draft >> 5] >> (draft & 31)) & 1u)));
}
// Whether some row of the tile does not see some of the 64 keys from k0 on.
__device__ __forceinline__ bool partly_seen(const PackedArgs& a, const Tile& t, int k0) {
  return a.visible != nullptr ? k0 + KT > t.rq.base : k0 + KT - 1 > t.first_place || k0 + KT > t.k_hi;
}
// The slot of a key of the tile's request, -1: none.
__device__ __forceinline__ long long slot_of(const PackedArgs& a, const int* table, int key, int k_hi) {
  if (key >= k_hi) return -1;
  const int page = table[key >> a.page_shift];
  if (page < 0 || page >= a.n_pages) return -1;
  return (static_cast<long long>(page) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}
// Dims d .. d + 3 of the output row `at` (normalised) and, for put_lse, its log-sum-exp: to the output, or to this part's
// scratch.
template <typename T>
__device__ __forceinline__ void put_row(const PackedArgs& a, bool whole, long long at, int d, const float* o) {
  if (whole) store4(static_cast<T*>(a.out) + at * a.D_v + d, o);
  else store4(static_cast<float*>(a.workspace) + (static_cast<long long>(blockIdx.y) * a.T * a.n_h + at) * a.D_v + d, o);
}
__device__ __forceinline__ void put_lse(const PackedArgs& a, bool whole, long long at, float lse2, int n_split) {
  if (whole) {
    if (a.lse != nullptr) a.lse[at] = lse2 * 0.69314718055994530942f;
  } else {
    static_cast<float*>(a.workspace)[static_cast<long long>(n_split) * a.T * a.n_h * a.D_v +
                                     static_cast<long long>(blockIdx.y) * a.T * a.n_h + at] = lse2;
  }
}

// fp32, D_qk <= 128, NV blocks of 64 value dims.  Thread (tx, ty) has the scores of rows 4 ty + i with keys tx + 16 j, and
// dims 4 tx + 64 v of the same rows' outputs.  Rows of K, V, Q and P end 4 floats behind a multiple of 32, so that the
// 16-byte reads of eight lanes fall on different banks.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {  // zeros where there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all_but_last() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <int NV, int ST>
__global__ void __launch_bounds__(kThreads, NV == 2 ? 1 : 2)
    packed_f32_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ RopeFreq f, int n_split) {
  extern __shared__ float4 smem4[];
  constexpr int VLD = NV * 64 + kPad;
  const int QLD = a.D_qk + (a.D_qk % 32 ? 36 - a.D_qk % 32 : 4);  // 4 behind a multiple of 32
  float* const Qs = reinterpret_cast<float*>(smem4);
  float* const Ks = Qs + R * QLD;
  float* const Vs = Ks + ST * KT * QLD;
  float* const Ps = Vs + ST * KT * VLD;  // [R][LD]; a warp reads what it wrote itself
  __shared__ long long slot[2][KT];
  __shared__ Rows rows;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int g = blockIdx.x % a.n_kv;
  const Tile t = find_tile<float>(a, g, n_split);
  if (t.here == 0) return;
  const int* const table = a.block_table + static_cast<long long>(t.b) * a.max_blocks;
  const float* const kp = static_cast<const float*>(a.k_pages) + g * a.D_qk;
  const float* const vp = static_cast<const float*>(a.v_pages) + g * a.D_v;
  const int kc = a.D_qk / 4, vc = a.D_v / 4;
  const long long k_row = static_cast<long long>(a.n_kv) * a.D_qk;
  // 16-byte pieces of 64 keys, a thread's first one and the step to its next (no divisions in the loop over tiles)
  const int k_key = tid / kc, k_c = tid - k_key * kc, k_step = kThreads / kc, k_rest = kThreads - k_step * kc;
  const int v_key = tid / vc, v_c = tid - v_key * vc, v_step = kThreads / vc, v_rest = kThreads - v_step * vc;
  const auto fetch_k = [&](int s) {
    for (int key = k_key, c = k_c; key < KT;) {
      const long long at = slot[s][key];
      copy16(Ks + ((ST - 1) * s * KT + key) * QLD + c * 4, kp + (at < 0 ? 0 : at) * k_row + c * 4, at >= 0);
      key += k_step;
      if ((c += k_rest) >= kc) c -= kc, ++key;
    }
    copy_commit();
  };
  const auto fetch_v = [&](int s) {
    for (int key = v_key, c = v_c; key < KT;) {
      const long long at = slot[s][key];
      copy16(Vs + ((ST - 1) * s * KT + key) * VLD + c * 4, vp + (at < 0 ? 0 : at) * a.v_token_stride + c * 4, at >= 0);
      key += v_step;
      if ((c += v_rest) >= vc) c -= vc, ++key;
    }
    copy_commit();
  };
  if (tid < 2 * KT) slot[tid >> 6][tid & 63] = slot_of(a, table, t.k_lo + tid, t.k_hi);
  if (tid < R) load_row(a, t, g, tid, &rows);
  for (int i = tid; i < ST * KT * (NV * 16 - vc); i += kThreads) {  // value dims behind the last stay 0
    const int n = NV * 16 - vc, key = i / n;
    *reinterpret_cast<float4*>(Vs + key * VLD + (vc + i - key * n) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  fetch_k(0);
  fetch_v(0);
  for (int r = k_key, c = k_c; r < R;) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < t.here) x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + static_cast<long long>(rows.at[r]) * a.D_qk + c * 4);
    *reinterpret_cast<float4*>(Qs + r * QLD + c * 4) = x;
    r += k_step;
    if ((c += k_rest) >= kc) c -= kc, ++r;
  }
  if (f.n_pairs) __syncthreads();
  for (int i = tid; i < t.here * f.n_pairs; i += kThreads) {
    const int r = i / f.n_pairs, p = i - r * f.n_pairs, pos = rows.pos[r];
    if (pos < 0) continue;
    float sn, cs;
    with_angles<true, false>(pos, [&](auto angle) { angle(f.hi[p], f.lo[p], &sn, &cs); });
    const int2 d = rope_pair_dims(f, p);
    rotate_pair(Qs[r * QLD + a.rope_offset + d.x], Qs[r * QLD + a.rope_offset + d.y], sn, cs);
  }
  float m[4], l[4];
  float2 acc[NV][4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v][i][0] = acc[v][i][1] = make_float2(0.f, 0.f);
  }
  const bool active = (tid >> 5) * 8 < t.here;  // this warp has rows (eight of them)
  int cur = 0;
  for (int k0 = t.k_lo; k0 < t.k_hi; k0 += KT, cur ^= 1) {  // k_hi <= 2^31 - 2^16: no overflow
    if constexpr (ST == 2) copy_wait_all();
    else copy_wait_all_but_last();
    __syncthreads();  // K (two stages: and V), and before the first tile Q, are there; the stage before is free
    long long next_slot = -1;  // of the tile behind the next one, which takes this one's place
    const auto look = [&] {
      const long long next = static_cast<long long>(k0) + 2 * KT + tid;
      if (tid < KT && next < t.k_hi) next_slot = slot_of(a, table, static_cast<int>(next), t.k_hi);
    };
    if (ST == 2) look();
    if (ST == 2 && k0 + KT < t.k_hi) {
      fetch_k(cur ^ 1);
      fetch_v(cur ^ 1);
    }
    const float* const Kt = Ks + (ST - 1) * cur * KT * QLD;
    const float* const Vt = Vs + (ST - 1) * cur * KT * VLD;
    float2 s2[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; active && d < a.D_qk; d += 4) {
      float4 q4[4], k4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q4[i] = *reinterpret_cast<const float4*>(Qs + (ty * 4 + i) * QLD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(Kt + (tx + 16 * j) * QLD + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i][j] = __ffma2_rn(make_float2(q4[i].x, q4[i].y), make_float2(k4[j].x, k4[j].y), s2[i][j]);
          s2[i][j] = __ffma2_rn(make_float2(q4[i].z, q4[i].w), make_float2(k4[j].z, k4[j].w), s2[i][j]);
        }
    }
    if constexpr (ST == 1) {
      __syncthreads();
      fetch_k(cur ^ 1);
    }
    const bool masked = partly_seen(a, t, k0);
    const auto weights = [&](auto with_mask) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        float s[4], mx = -INFINITY;
        bool seen[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] = s2[i][j].x + s2[i][j].y;
          seen[j] = !with_mask() || sees(a, t, rows.place[r], rows.vis[r], k0 + tx + 16 * j);
          if (seen[j]) mx = fmaxf(mx, s[j]);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m[i], mx * a.scale_log2), m_ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = fast_exp2(m[i] - m_ref);
        m[i] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = fast_exp2(fmaf(s[j], a.scale_log2, -m_ref));
          if (seen[j]) sum += p;
          Ps[r * LD + tx + 16 * j] = seen[j] ? p : kMasked;
        }
        l[i] = fmaf(l[i], alpha, sum);  // of this thread's keys
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            acc[v][i][j].x *= alpha;
            acc[v][i][j].y *= alpha;
          }
      }
    };
    if (active) {
      if (masked) weights([] { return true; });
      else weights([] { return false; });
    }
    if constexpr (ST == 1) {
      look();
      copy_wait_all_but_last();
      __syncthreads();  // V and P are there
    } else {
      __syncwarp();
    }
    const auto add = [&](auto with_mask) {
#pragma unroll 4
      for (int k = 0; k < KT; k += 4) {
        float p4[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(Ps + (ty * 4 + i) * LD + k);
          p4[i][0] = x.x; p4[i][1] = x.y; p4[i][2] = x.z; p4[i][3] = x.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const float4 x = *reinterpret_cast<const float4*>(Vt + (k + kk) * VLD + v * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a value that the row does not see may be anything
              if (with_mask() && p4[i][kk] == kMasked) continue;
              const float2 p = make_float2(p4[i][kk], p4[i][kk]);
              acc[v][i][0] = __ffma2_rn(p, make_float2(x.x, x.y), acc[v][i][0]);
              acc[v][i][1] = __ffma2_rn(p, make_float2(x.z, x.w), acc[v][i][1]);
            }
          }
      }
    };
    if (active) {
      if (masked) add([] { return true; });
      else add([] { return false; });
    }
    if constexpr (ST == 1) {
      __syncthreads();
      fetch_v(cur ^ 1);
    }
    if (tid < KT) slot[cur][tid] = next_slot;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    if (r >= t.here) continue;
    if (rows.place[r] < 0) l[i] = 0.f;  // an empty row: tiles that are seen whole do not ask
    const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];  // 0: no key with a weight; NaN stays
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = v * 64 + tx * 4;
      if (d >= a.D_v) continue;
      float o[4] = {acc[v][i][0].x * inv, acc[v][i][0].y * inv, acc[v][i][1].x * inv, acc[v][i][1].y * inv};
      if (rows.place[r] < 0 || (t.whole && l[i] == 0.f)) o[0] = o[1] = o[2] = o[3] = 0.f;
      put_row<float>(a, t.whole, rows.at[r], d, o);
    }
    if (tx == 0) put_lse(a, t.whole, rows.at[r], l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]), n_split);
  }
}

// NV: blocks of 64 value dims.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads)
    packed_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ RopeFreq f, int n_split) {
  extern __shared__ float4 smem4[];
  float* const Qs = reinterpret_cast<float*>(smem4);  // [D_qk][LD]
  float* const Ks = Qs + a.D_qk * LD;                 // [DC][LD], then V: [KT][LD]
  float* const Ps = Ks + KT * LD;                     // [KT keys][LD rows]
  __shared__ long long slot[KT];                      // slots of the tile's keys, -1: none
  __shared__ Rows rows;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int g = blockIdx.x % a.n_kv;
  const Tile t = find_tile<T>(a, g, n_split);
  if (t.here == 0) return;
  const int* const table = a.block_table + static_cast<long long>(t.b) * a.max_blocks;
  if (tid < R) load_row(a, t, g, tid, &rows);
  __syncthreads();
  for (int i = tid; i < R * (a.D_qk / 8); i += kThreads) {
    const int r = i & (R - 1), d = (i >> 6) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < t.here) load8(static_cast<const T*>(a.q) + static_cast<long long>(rows.at[r]) * a.D_qk + d, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) Qs[(d + e) * LD + r] = x[e];
  }
  __syncthreads();
  if (f.n_pairs) {
    for (int i = tid; i < t.here * f.n_pairs; i += kThreads) {
      const int r = i % t.here, p = i / t.here, pos = rows.pos[r];
      if (pos < 0) continue;
      float sn, cs;
      with_angles<true, false>(pos, [&](auto angle) { angle(f.hi[p], f.lo[p], &sn, &cs); });
      const int2 d = rope_pair_dims(f, p);
      rotate_pair(Qs[(a.rope_offset + d.x) * LD + r], Qs[(a.rope_offset + d.y) * LD + r], sn, cs);
    }
  }
  float m[4], l[4], acc[NV][4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[v][i][j] = 0.f;
  }
  for (int k0 = t.k_lo; k0 < t.k_hi; k0 += KT) {
    __syncthreads();
    if (tid < KT) slot[tid] = slot_of(a, table, k0 + tid, t.k_hi);
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int d0 = 0; d0 < a.D_qk; d0 += DC) {
      __syncthreads();
      {  // 64 keys x 32 dims, 8 dims of a key per thread
        const int key = tid >> 2, d = d0 + (tid & 3) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (d < a.D_qk && slot[key] >= 0)
          load8(static_cast<const T*>(a.k_pages) + (slot[key] * a.n_kv + g) * a.D_qk + d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) Ks[(d - d0 + e) * LD + key] = x[e];
      }
      __syncthreads();
      const int dn = min(DC, a.D_qk - d0);
#pragma unroll 8
      for (int d = 0; d < dn; ++d) {
        const float4 qv = *reinterpret_cast<const float4*>(Qs + (d0 + d) * LD + ty * 4);
        const float4 kv = *reinterpret_cast<const float4*>(Ks + d * LD + tx * 4);
        const float q4[4] = {qv.x, qv.y, qv.z, qv.w}, k4[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = fmaf(q4[i], k4[j], s[i][j]);
      }
    }
    const bool masked = partly_seen(a, t, k0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, place = rows.place[r];
      bool seen[4];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        seen[j] = sees(a, t, place, rows.vis[r], k0 + tx * 4 + j);
        s[i][j] *= a.scale_log2;
        if (seen[j]) mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m[i], mx);
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m[i] - m_ref);
      m[i] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - m_ref);
        s[i][j] = seen[j] ? p : kMasked;
        if (seen[j]) sum += p;
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[v][i][j] *= alpha;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(Ps + (tx * 4 + j) * LD + ty * 4) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      __syncthreads();
      for (int i = tid; i < KT * 8; i += kThreads) {
        const int key = i >> 3, d = v * 64 + (i & 7) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (d < a.D_v && slot[key] >= 0)
          load8(static_cast<const T*>(a.v_pages) + slot[key] * a.v_token_stride + g * a.D_v + d, x);
        *reinterpret_cast<float4*>(Ks + key * LD + (i & 7) * 8) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(Ks + key * LD + (i & 7) * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
      }
      __syncthreads();
      const auto add = [&](auto with_mask) {
#pragma unroll 8
        for (int k = 0; k < KT; ++k) {
          const float4 pv = *reinterpret_cast<const float4*>(Ps + k * LD + ty * 4);
          const float4 vv = *reinterpret_cast<const float4*>(Ks + k * LD + tx * 4);
          const float p4[4] = {pv.x, pv.y, pv.z, pv.w}, v4[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a value that the row does not see may be anything
            if (with_mask() && p4[i] == kMasked) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[v][i][j] = fmaf(p4[i], v4[j], acc[v][i][j]);
          }
        }
      };
      if (masked) add([] { return true; });
      else add([] { return false; });
    }
  }
  // out, or this split's normalised part (of no weight: 0, or beside values that are not finite NaN, as 0 times these is)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= t.here) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];  // 0: no key with a weight; NaN stays
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = v * 64 + tx * 4;
      if (d >= a.D_v) continue;
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = rows.place[r] < 0 || (t.whole && l[i] == 0.f) ? 0.f : acc[v][i][j] * inv;
      put_row<T>(a, t.whole, rows.at[r], d, o);
    }
    if (tx == 0) put_lse(a, t.whole, rows.at[r], l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]), n_split);
  }
}

// A warp per row whose keys were cut: out = sum_j 2^(lse_j - lse) out_j over the parts.
template <typename T>
__global__ void __launch_bounds__(kThreads) packed_combine_kernel(const __grid_constant__ PackedArgs a, int n_split) {
  const int lane = threadIdx.x & 31;
  const long long at = blockIdx.x * static_cast<long long>(kThreads / 32) + (threadIdx.x >> 5);
  const long long rows = static_cast<long long>(a.T) * a.n_h;
  if (at >= rows || at >= static_cast<long long>(packed_first(a, a.B)) * a.n_h) return;  // those behind are written
  const float* const ws = static_cast<const float*>(a.workspace);
  const float* const lses = ws + n_split * rows * a.D_v + at;
  const int t = static_cast<int>(at / a.n_h), G = a.n_h / a.n_kv;
  int lo = 0, hi = a.B - 1;  // the row's request: the last one that starts at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (packed_first(a, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const PackedRequest rq = packed_request(a, lo);
  const long long n_rows = static_cast<long long>(rq.rows) * G;
  long long end = (static_cast<long long>(t - rq.first) * G + (at - static_cast<long long>(t) * a.n_h) % G) / R * R + R;  // of its tile
  end = end < n_rows ? end : n_rows;
  const int keys = keys_of(a, rq, end - 1, G), part = part_of(keys, n_split);
  if (keys <= part) return;
  const int parts = static_cast<int>((static_cast<long long>(keys) + part - 1) / part);
  float m = -INFINITY, den = 0.f;
  for (int j = 0; j < parts; ++j) m = fmaxf(m, lses[j * rows]);
  const float m_ref = m == -INFINITY ? 0.f : m;
  for (int j = 0; j < parts; ++j) den += exp2f(lses[j * rows] - m_ref);
  const float inv = den > 0.f ? 1.f / den : den;
  for (int d = lane * 4; d < a.D_v; d += 128) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < parts; ++j) {
      const float w = exp2f(lses[j * rows] - m_ref) * inv;
      const float4 x = *reinterpret_cast<const float4*>(ws + (j * rows + at) * a.D_v + d);
      o[0] = fmaf(w, x.x, o[0]);
      o[1] = fmaf(w, x.y, o[1]);
      o[2] = fmaf(w, x.z, o[2]);
      o[3] = fmaf(w, x.w, o[3]);
    }
    if (den == 0.f) o[0] = o[1] = o[2] = o[3] = 0.f;
    store4(static_cast<T*>(a.out) + at * a.D_v + d, o);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[at] = den == 0.f ? -INFINITY : (m + log2f(den)) * 0.69314718055994530942f;
}

// Numbers of tiles: an upper bound of the tiles.
long long tile_numbers(const PackedArgs& a) {
  return static_cast<long long>(a.T) * (a.n_h / a.n_kv) / R + a.B;
}
// Parts of a tile's keys, at most: as many as make two blocks per SM of a GB300 (152; a constant, as the workspace is sized
// by it).  With fp32 heads of up to 64 value dims, and in packed_kernel up to 256 value and some 270 query dims, these all run
// at once.  (A second wave costs as much as the first: with half as many parts again, 6 requests of up to 16 drafts took half
// as long again.)  Where shared memory or registers leave room for one block per SM - packed_f32_kernel<2, 2>, and
// packed_kernel with more dims, as MLA's 576 - they run in two waves of parts half as long.  (Two to four parts of
// 256 keys or more where there are one to four waves made 8 prompts of up to 500 tokens, 12 heads, up to 14% slower, and 4 x
// 128 tokens behind 2000, 32 heads, 7% to 11%.  Not by the table's width: tables are as wide as a request may grow.)
int splits(const PackedArgs& a) {
  const long long n = 2 * 152 / (tile_numbers(a) * a.n_kv);
  return static_cast<int>(n < 1 ? 1 : n > 64 ? 64 : n);
}
size_t smem_bytes(const PackedArgs& a) { return static_cast<size_t>(a.D_qk + 2 * KT) * LD * sizeof(float); }

// Behind a kernel's launch: the one that joins its splits.
template <typename T>
cudaError_t join(const PackedArgs& a, int n_split, cudaStream_t st, int* launches) {
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || n_split == 1) return err;
  const long long rows = static_cast<long long>(a.T) * a.n_h;
  packed_combine_kernel<T><<<static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, st>>>(a, n_split);
  *launches += 1;
  return cudaGetLastError();
}
template <typename T, int NV>
cudaError_t launch(const PackedArgs& a, const RopeFreq& rope, int n_split, cudaStream_t st, int* launches) {
  const size_t smem = smem_bytes(a);
  const cudaError_t e = cudaFuncSetAttribute(packed_kernel<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>((640 + 2 * KT) * LD * sizeof(float)));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(tile_numbers(a) * a.n_kv), n_split);
  packed_kernel<T, NV><<<grid, kThreads, smem, st>>>(a, rope, n_split);
  *launches += 1;
  return join<T>(a, n_split, st, launches);
}
template <int NV, int ST>
cudaError_t launch_f32(const PackedArgs& a, const RopeFreq& rope, int n_split, cudaStream_t st, int* launches) {
  const int qld = a.D_qk + (a.D_qk % 32 ? 36 - a.D_qk % 32 : 4);
  const size_t smem = ((1 + ST) * 64 * qld + ST * 64 * (NV * 64 + kPad) + 64 * LD) * sizeof(float);
  constexpr int kMost = ((1 + ST) * 64 * ((NV == 1 && ST == 2 ? 64 : 128) + kPad) + ST * 64 * (NV * 64 + kPad) + 64 * LD) * static_cast<int>(sizeof(float));
  const cudaError_t e = cudaFuncSetAttribute(packed_f32_kernel<NV, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(tile_numbers(a) * a.n_kv), n_split);
  packed_f32_kernel<NV, ST><<<grid, kThreads, smem, st>>>(a, rope, n_split);
  *launches += 1;
  return join<float>(a, n_split, st, launches);
}
template <typename T>
cudaError_t launch_dims(const PackedArgs& a, const RopeFreq& rope, int n_split, cudaStream_t st, int* launches) {
  if constexpr (sizeof(T) == 4) {
    if (a.D_qk <= 128 && a.D_v <= 128)
      return a.D_v > 64    ? launch_f32<2, 2>(a, rope, n_split, st, launches)
             : a.D_qk > 64 ? launch_f32<1, 1>(a, rope, n_split, st, launches)
                           : launch_f32<1, 2>(a, rope, n_split, st, launches);
  }
  if (a.D_v <= 64) return launch<T, 1>(a, rope, n_split, st, launches);
  if (a.D_v <= 128) return launch<T, 2>(a, rope, n_split, st, launches);
  if (a.D_v <= 256) return launch<T, 4>(a, rope, n_split, st, launches);
  return launch<T, 8>(a, rope, n_split, st, launches);
}

}  // namespace

size_t packed_workspace(const PackedArgs& a) {
  const int n = splits(a);
  return n == 1 ? 0 : static_cast<size_t>(n) * a.T * a.n_h * (a.D_v + 1) * sizeof(float);
}

cudaError_t launch_packed(const PackedArgs& a, const RopeFreq& rope, bool bf16, cudaStream_t st, int* launches) {
  const int n_split = splits(a);
  return bf16 ? launch_dims<__nv_bfloat16>(a, rope, n_split, st, launches) : launch_dims<float>(a, rope, n_split, st, launches);
}

}  // namespace attn
