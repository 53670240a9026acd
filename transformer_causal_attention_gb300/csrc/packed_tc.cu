// packed_tc.cu - attention of packed new tokens over a paged KV cache on the tensor cores (bf16,
// D_qk = D_v = 64 or 128): causal, or by visibility bits among drafted tokens.
//
// The query rows of a KV head in one request are its (token, head of the group) pairs, token after
// token; 128 / G tokens (G = n_h / n_kv) fill a row tile of an MMA.  Two row tiles that follow one
// another share each 128-key tile of K and V (a pair segment, 256 rows); what is left at a request's end,
// up to one row tile, is a single segment, whose key tiles the two softmax warpgroups take in turns.  So
// packed prompts, chunks behind a cache, trees of drafts and single tokens are one kernel:
//   S = Q K^T, online softmax over the rows ("Transformer架构完全深度解析" §13), O += P V.
//
// Work split.  The segments lie on one line, request by request, KV head by KV head, row tiles rising;
// a segment's length is its keys times a weight (pair or single) plus a lead for what starting it costs.
// The line is cut into equal parts, one per CTA (one persistent CTA per SM), at tile borders, also
// inside a segment: so SMs finish together whatever the lengths are, from one short prompt to two long
// documents with a few drafts each.  Lengths are on the device, so each CTA sums the line itself (a closed
// form per request) and finds its part by bisection.  Only a CTA's first and last piece can be a part of
// a segment: these leave a normalised partial and its log-sum-exp, which a second kernel joins; all other
// pieces write their rows of the output.
//
// Rounding.  Weights are rounded to bf16.  A rotated query is kept as the sum of two bf16 values, the
// second for kLoSteps of the D / 16 MMA steps (from the start of the rotated span on): one bf16 alone made the
// output's error 1.5 times that of its own rounding behind 2000 keys and 1.7 times behind 30000 (normally
// distributed inputs, against 64 bits), with five of eight steps it is at most 1.46 times.  The second part's
// MMAs use the K tile that is there anyway.  It is kept unswizzled, 16 bytes of a row after the other row's.
//
// What a row does not see.  Scores are masked by index.  A value whose weight is 0 still meets the MMA, so in
// the tiles that some row sees in part ("care" tiles: the last ones of a segment) warp 3 clears value rows
// behind the last key and replaces infinities and NaN by 0, noting their keys; the epilogue adds such
// values to the rows that do see them.  The rest of the tiles is seen whole by every row.
//
// A CTA (384 threads): warp 0 loads K tiles by TMA, warp 2 query rows and V (in quarters of 32 keys, so that
// the shared memory left by both parts of Q holds 1.75 V tiles), a lane per box; warp 1 issues the MMAs; warp 3
// walks the line, hands the pieces out through a queue in shared memory and treats care tiles; warps
// 4-7 and 8-11 are the softmax of row tiles 0 and 1 (or of alternate key tiles), a row per thread.
// TMEM: S/P of the two in columns [0, 128) and [128, 256), O behind them.
#include <math.h>

#include <atomic>

#include "api.h"
#include "paged_tc.cuh"

namespace attn {

struct PackedTcPlan {
  int ctas;
  int tile_toks;  // tokens per row tile: 128 / G
  int slot_rows;  // rows of a partial
  int lo_first;   // first MMA step with a second part of Q
  int n_pairs, half;  // of the rotation
  // float offsets into the workspace: partials [2 * ctas, slot_rows, D], their log-sum-exps, records, angles
  long long l, rec, angles, end;
};

namespace {

constexpr int BM = 128;  // rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kCare = 3;   // care tiles of a piece, at most: 256 tokens of a pair, or 128 drafts
constexpr int kQueue = 6;  // pieces in the queue; kAhead are handed out before warp 3 treats the first of them
constexpr int kAhead = 3;

// Points on the line per key of a segment, and the leads, in keys of the same weight.
constexpr int kPairWeight = 8, kSingleWeight = 6;
constexpr int kPairLead = 256, kSingleLead = 256;

// Register split as in prefill_tc.cu: a softmax thread holds a row of 128 scores.
constexpr int kLaunchRegs = 168;
constexpr int kRegsCtl = 152, kRegsSoftmax = 176;
constexpr int kRegsNeeded = 4 * 32 * kRegsCtl + 8 * 32 * kRegsSoftmax;
static_assert(kRegsNeeded <= kThreads * kLaunchRegs, "register split exceeds the launch's pool");

// A piece: tiles [t, t_end) of a segment.
enum : int { kNone = 0, kSingle = 1, kPair = 2 };
struct Piece {
  int kind, g, b;
  int row0, ntok;      // its tokens: rows row0 .. row0 + ntok - 1 of q
  int t, t_end;
  int kt0, kt;         // key tiles of the segment, for its first row tile and in all
  int place0;          // place of its first token
  int base, klim;      // place of the request's first new token; keys behind klim are not there
  int care_t;          // first care tile
  int slot;            // partial 0 or 1 of the CTA, -1: the whole segment
  uint32_t bad_any, bad[kCare][4];  // keys of care tiles with values that are not finite
};

// Tiles of a piece that worker w takes: first, first + step, ... (n of them).
struct Share {
  int n, first, step;
  __device__ __forceinline__ Share(const Piece& u, int w) {
    const int nv = u.t_end - u.t;
    if (u.kind == kPair) {
      first = u.t;
      step = 1;
      n = w ? nv : max(0, min(u.t_end, u.kt0) - u.t);
    } else {
      first = u.t + w;
      step = 2;
      n = (nv + 1 - w) >> 1;
    }
  }
};

template <int D, bool LO>
struct Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kBlocks = D / 64;                      // 64-dim column blocks of a tile
  static constexpr int kBlockBytes = BM * 128;                // one column block (128 rows x 128 bytes, swizzled)
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kSteps = D / 16;
  static constexpr int kLoSteps = LO ? D / 32 : 0;             // MMA steps with a second part of Q
  static constexpr int kLoBytes = kLoSteps * 2 * BM * 16;     // of a row tile
  static constexpr int kPLoSteps = LO ? 4 : 0;                // steps of 16 keys with a second part of P
  static constexpr int kKStages = D == 128 ? 2 : 4;
  static constexpr int kVStages = D == 128 ? 2 : 4;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kLoOff = kVOff + kVStages * kTileBytes;
  static constexpr int kMlOff = kLoOff + 2 * kLoBytes;         // worker 1's maximum and sum of each row
  static constexpr int kBarOff = kMlOff + BM * 8;
  static constexpr uint32_t kOCol = 256;                       // O of worker w at kOCol + w D
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, true);
};

template <typename C>
struct Bars {
  uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  uint64_t v_full[C::kVStages], v_empty[C::kVStages], v_fixed[C::kVStages];
  uint64_t q_full[2], q_ready[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t x_full, x_done;  // single pieces: worker 1's sums are there, have been read
  uint64_t piece_full[kQueue], piece_empty[kQueue], care_done[kQueue];
  uint64_t fin;
  Piece piece[kQueue];
  WaitCtl wc;
  long long warp_sum[kThreads / 32];
  long long start_off;
  int start_b;
  uint32_t tmem_base;
  int abort_flag;
};
template <typename C>
constexpr int smem_bytes() {
  static_assert(C::kBarOff + sizeof(Bars<C>) <= 227 * 1024, "shared memory per CTA");
  return C::kBarOff + static_cast<int>(sizeof(Bars<C>));
}

// What a CTA's partial in a slot is, for the kernel that joins them (kt = 0: nothing).
struct Record {
  int kind, g, row0, ntok, t, t_end, kt, pad;
};

// ------------------------------------------------------------------------------------- the line
// A request's segments in one KV head: np pairs of row tiles, then a last one of rem tokens (a pair if they
// fill more than a row tile).  Points are 64-bit: rows * keys / 128 * weight stays below 2^60.
struct Seg {
  PackedRequest r;
  int tt;        // tokens per row tile
  int np, rem;
  int keys;      // causal: keys in front of the request's new tokens; tree: of every segment
  bool tree;
  __device__ __forceinline__ Seg(const PackedArgs& a, const PackedTcPlan& pl, int b) : r(packed_request(a, b)), tt(pl.tile_toks) {
    tree = a.visible != nullptr;
    np = r.rows / (2 * tt);
    rem = r.rows - np * 2 * tt;
    keys = tree ? max(min(r.len, static_cast<int>(min(static_cast<long long>(r.base) + 32 * a.words, 0x7fffffffLL))), 1)
                : max(r.base, 0);
  }
  __device__ __forceinline__ bool last_is_pair() const { return rem > tt; }
  __device__ __forceinline__ bool is_pair(int p) const { return p < np || last_is_pair(); }
  __device__ __forceinline__ int weight(int p) const { return is_pair(p) ? kPairWeight : kSingleWeight; }
  __device__ __forceinline__ long long lead(int p) const {
    return is_pair(p) ? kPairLead * kPairWeight : kSingleLead * kSingleWeight;
  }
  __device__ __forceinline__ int count() const { return np + (rem > 0); }
  __device__ __forceinline__ long long keys_of(int p) const {  // for the length
    return tree ? keys : static_cast<long long>(keys) + min((p + 1) * 2 * tt, r.rows);
  }
  __device__ __forceinline__ long long length(int p) const { return lead(p) + keys_of(p) * weight(p); }
  // points in front of pair p <= np
  __device__ __forceinline__ long long before(int p) const {
    const long long q = p;
    return q * (kPairLead * kPairWeight) + kPairWeight * (q * keys + (tree ? 0 : tt * q * (q + 1)));
  }
  __device__ __forceinline__ long long own() const { return before(np) + (rem > 0 ? length(np) : 0); }
  // real keys of the segment's first n tokens, at least 1
  __device__ __forceinline__ int seen(int p, int n) const {
    return tree ? keys : max(min(r.len, r.base + p * 2 * tt + n), 1);
  }
};
__device__ __forceinline__ int tiles_of(int keys) { return static_cast<int>((static_cast<unsigned>(keys) + BN - 1) / BN); }
// The first tile that starts at or behind point x of a segment of kt tiles.
__device__ __forceinline__ int tile_at(long long x, long long lead, int weight, int kt) {
  const long long d = x - lead;
  if (d <= 0) return 0;
  const long long t = (d + BN * weight - 1) / (BN * weight);
  return t < kt ? static_cast<int>(t) : kt;
}
struct Cut {
  long long part;
  int extra;
  __device__ __forceinline__ Cut(long long total, int n) : part(total / n), extra(static_cast<int>(total % n)) {}
  __device__ __forceinline__ long long at(int k) const { return part * k + min(k, extra); }
};

// A walk along one CTA's part: the segment (b, g, p), its next tile, and the part's end from its first point.
struct Walk {
  int b, g, p, t;
  long long end;
  bool live;
};

__device__ __forceinline__ void next_request(const PackedArgs& a, Walk& w) {
  do ++w.b;
  while (w.b < a.B && packed_request(a, w.b).rows == 0);
  if (w.b >= a.B) w.live = false;
  w.g = w.p = w.t = 0;
}

// The next piece of a walk (kind kNone at its end).
__device__ __noinline__ void next_piece(const PackedArgs& a, const PackedTcPlan& pl, Walk& w, Piece* out) {
  out->kind = kNone;
  while (w.live && w.end > 0) {
    const Seg s(a, pl, w.b);
    const int p = w.p;
    const bool pair = s.is_pair(p);
    const int tok0 = p * 2 * s.tt, ntok = min(2 * s.tt, s.r.rows - tok0);
    const int klim = s.seen(p, ntok), kt = tiles_of(klim);
    const int t = w.t, t_end = tile_at(w.end, s.lead(p), s.weight(p), kt);
    if (t < t_end) {
      out->kind = pair ? kPair : kSingle;
      out->g = w.g;
      out->b = w.b;
      out->row0 = s.r.first + tok0;
      out->ntok = ntok;
      out->t = t;
      out->t_end = t_end;
      out->kt = kt;
      out->kt0 = pair ? tiles_of(s.seen(p, s.tt)) : kt;
      out->place0 = s.r.base + tok0;
      out->base = s.r.base;
      out->klim = klim;
      out->care_t = max(s.tree ? s.r.base : s.r.base + tok0 + 1, 0) / BN;
      out->slot = t > 0 ? 0 : t_end < kt ? 1 : -1;
      out->bad_any = 0;
    }
    w.t = t_end;
    if (t_end < kt) {  // the part ends here
      w.live = false;
    } else {
      w.t = 0;
      w.end -= s.length(p);
      if (++w.p == s.count()) {
        w.p = 0;
        if (++w.g == a.n_kv) next_request(a, w);
      }
    }
    if (t < t_end) return;
  }
  w.live = false;
}

// ------------------------------------------------------------------------------------- MMAs
// A unswizzled (the second part of Q: 16-byte chunks of 128 rows one after the other), B as all tiles.
constexpr uint32_t kLoHigh = (128u >> 4) | (1u << 14);  // 8-row groups 128 bytes apart, descriptor version, no swizzle
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kLoHigh), "n"(kDescHigh)
      : "memory");
}

// ------------------------------------------------------------------------------------- rows
// Rotate row r of a query tile by the cosines and sines at cs (a pair each): the rounded values in place, what the
// rounding left of chunks [lo_chunk0, lo_chunk0 + LO_CHUNKS) to the second part (0 for dims outside the span).
template <int LO_CHUNKS>
__device__ __noinline__ void rotate_row(uint8_t* tile, uint8_t* lo, int r, const float2* cs, int rope_offset, int n_pairs,
                                      bool half, int lo_chunk0) {
  auto chunk = [&](int c) { return reinterpret_cast<uint4*>(tile + (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
  auto rest = [&](int c, const float* x, uint4 rounded) {
    if (static_cast<unsigned>(c - lo_chunk0) >= static_cast<unsigned>(LO_CHUNKS)) return;
    float y[8];
    bf16x8_to_f32(rounded, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fabsf(y[e]) < INFINITY ? x[e] - y[e] : 0.f;  // 0 behind an infinity
    *reinterpret_cast<uint4*>(lo + (c - lo_chunk0) * (BM * 16) + r * 16) = f32_to_bf16x8(y);
  };
  const int c0 = rope_offset / 8, c1 = c0 + n_pairs / 4;
  if (c0 > lo_chunk0 || c1 < lo_chunk0 + LO_CHUNKS) {
    for (int c = 0; c < LO_CHUNKS; ++c)
      *reinterpret_cast<uint4*>(lo + c * (BM * 16) + r * 16) = make_uint4(0, 0, 0, 0);
  }
  const float4* const angles = reinterpret_cast<const float4*>(cs);  // two pairs each
  if (half) {
    const int hc = n_pairs / 8;
#pragma unroll 2
    for (int i = 0; i < hc; ++i) {
      float4 w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __ldg(angles + 4 * i + e);
      uint4* const p0 = chunk(c0 + i);
      uint4* const p1 = chunk(c0 + i + hc);
      float x0[8], x1[8];
      bf16x8_to_f32(*p0, x0);
      bf16x8_to_f32(*p1, x1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rotate_pair(x0[2 * e], x1[2 * e], w[e].y, w[e].x);
        rotate_pair(x0[2 * e + 1], x1[2 * e + 1], w[e].w, w[e].z);
      }
      const uint4 y0 = f32_to_bf16x8(x0), y1 = f32_to_bf16x8(x1);
      *p0 = y0;
      *p1 = y1;
      rest(c0 + i, x0, y0);
      rest(c0 + i + hc, x1, y1);
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < n_pairs / 4; ++i) {
      const float4 w0 = __ldg(angles + 2 * i), w1 = __ldg(angles + 2 * i + 1);
      uint4* const p = chunk(c0 + i);
      float x[8];
      bf16x8_to_f32(*p, x);
      rotate_pair(x[0], x[1], w0.y, w0.x);
      rotate_pair(x[2], x[3], w0.w, w0.z);
      rotate_pair(x[4], x[5], w1.y, w1.x);
      rotate_pair(x[6], x[7], w1.w, w1.z);
      const uint4 y = f32_to_bf16x8(x);
      *p = y;
      rest(c0 + i, x, y);
    }
  }
}

// Cosines and sines of the rows' rotations, float2 [T, n_pairs]: computed once for all heads (in the attention kernel,
// where all rows of a tile meet them at once, they took 3 us per piece).  A thread per (row, pair).
__global__ void __launch_bounds__(256) packed_angles_kernel(const __grid_constant__ PackedArgs a,
                                                            const __grid_constant__ RopeFreq f, float2* out) {
  asm volatile("griddepcontrol.launch_dependents;");  // the attention kernel starts, and waits where it reads these
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  const int t = static_cast<int>(i / f.n_pairs), p = static_cast<int>(i - static_cast<long long>(t) * f.n_pairs);
  if (t >= a.T) return;
  int pos;
  if (a.positions != nullptr) {
    pos = a.positions[t];
  } else {
    int lo = 0, hi = a.B - 1;  // the last request that starts at or before the row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (packed_first(a, mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    const PackedRequest r = packed_request(a, lo);
    pos = r.base + t - r.first;
  }
  float sn, cs;
  with_angles<true, false>(max(pos, 0), [&](auto angle) { angle(f.hi[p], f.lo[p], &sn, &cs); });
  out[i] = make_float2(cs, sn);
}

// Bits of the 128 keys from key0 on that a row sees: those below lim, or (tree) those below base and the drafts
// whose bits are set in w.
__device__ __forceinline__ void seen_below(int lim, int key0, uint32_t* m) {
  const int n = lim - key0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = n >= 32 * i + 32 ? 0xffffffffu : n > 32 * i ? (1u << (n - 32 * i)) - 1u : 0u;
}
__device__ __forceinline__ void seen_tree(const uint32_t* w, int base, int klim, int key0, uint32_t* m) {
  const int sh = key0 - base;  // draft of the tile's first key
  seen_below(klim, key0, m);   // keys that are there
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 32 keys from key0 + 32 i on: drafts d0 .. d0 + 31
    const int d0 = sh + 32 * i;
    uint32_t x;
    if (d0 <= -32) {
      x = 0xffffffffu;
    } else if (d0 >= 128) {
      x = 0u;
    } else {
      const int j = d0 >> 5, s = d0 & 31;  // j from -1 (all ones: in front of the drafts) to 3
      uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (j == k) lo = w[k];
        if (j + 1 == k) hi = w[k];
      }
      x = __funnelshift_r(lo, hi, s);
    }
    m[i] &= x;
  }
}

// This thread's row of a tile's scores become its weights P (see prefill_tc.cu): p = 2^(s * scale*log2e - m), m moves
// when the row maximum grew by more than the threshold.
// The first kLoKeys weights come as the sum of two bf16 values, the second ones behind all first ones.
template <int D, int kLoKeys>
__device__ __forceinline__ void softmax_row(uint32_t s_addr, uint32_t o_addr, bool masked, const uint32_t* mask,
                                            bool rescale, float scale_log2, float& m_run, float& l_run) {
  uint32_t sr[BN];
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_addr + c * 32, sr + c * 32);
  tmem_wait_ld();
  float s[BN];
#pragma unroll
  for (int c = 0; c < BN; ++c) s[c] = __uint_as_float(sr[c]);
  if (masked) {
#pragma unroll
    for (int c = 0; c < BN; ++c)
      if (!((mask[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
  }
  float m8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) m8[e] = s[e];
#pragma unroll
  for (int c = 8; c + 16 <= BN; c += 16)
#pragma unroll
    for (int e = 0; e < 8; ++e) m8[e] = fmax3(m8[e], s[c + e], s[c + 8 + e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], s[BN - 8 + e]);
  const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7])) * scale_log2;
  const bool need = mx > m_run + kRescaleThreshold;
  float alpha = 1.f;
  if (need) {
    if (m_run != -INFINITY) alpha = fast_exp2(m_run - mx);
    l_run *= alpha;
    m_run = mx;
  }
  uint32_t pr[BN / 2];
  const float2 sl2 = make_float2(scale_log2, scale_log2);
  const float m_ref = (m_run == -INFINITY) ? 0.f : m_run;  // every score so far is -inf: weights 0
  const float2 nm2 = make_float2(-m_ref, -m_ref);
  float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t pl[kLoKeys > 0 ? BN / 4 : 1];
#pragma unroll
  for (int c = 0; c < BN / 4; ++c) {
    const float2 x = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sl2, nm2);
    const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    acc[c & 3] = __fadd2_rn(acc[c & 3], pp);
    pr[c] = pack_bf16x2(pp.x, pp.y);
    if (2 * c < kLoKeys)
      pl[c] = pack_bf16x2(pp.x - __uint_as_float(pr[c] << 16), pp.y - __uint_as_float(pr[c] & 0xffff0000u));
  }
  tmem_st32(s_addr, pr);
  static_assert(kLoKeys == 0 || kLoKeys == BN / 2, "second parts fill 32 columns");
  if constexpr (kLoKeys > 0) tmem_st32(s_addr + 64, pl);
  if (__any_sync(0xffffffffu, need && rescale)) rescale_o<D>(o_addr, alpha);
#pragma unroll
  for (int c = BN / 4; c < BN / 2; ++c) {
    const float2 x = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sl2, nm2);
    const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    acc[c & 3] = __fadd2_rn(acc[c & 3], pp);
    pr[c] = pack_bf16x2(pp.x, pp.y);
  }
  acc[0] = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
  l_run += acc[0].x + acc[0].y;
  tmem_st32(s_addr + 32, pr + 32);
}

// The values that are not finite in care tiles, of dims [d, d + 32), added to the outputs of a row that sees them
// (tree: by the bits w, else below lim).
__device__ __noinline__ void add_bad(const PackedArgs& a, const Piece& u, int lim, const uint32_t* w, int d, float* o) {
  for (int i = 0; i < kCare; ++i) {
    const int key0 = (u.care_t + i) * BN;
    if (u.care_t + i >= u.t_end) break;
    if (u.care_t + i < u.t) continue;
    uint32_t m[4];
    if (a.visible != nullptr) seen_tree(w, u.base, u.klim, key0, m);
    else seen_below(lim, key0, m);
    for (int j = 0; j < 4; ++j) {
      for (uint32_t left = u.bad[i][j] & m[j]; left; left &= left - 1) {
        const int key = key0 + 32 * j + __ffs(left) - 1;
        const int page = a.block_table[static_cast<long long>(u.b) * a.max_blocks + (key >> a.page_shift)];
        const long long slot = (static_cast<long long>(page) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        const __nv_bfloat16* const v = static_cast<const __nv_bfloat16*>(a.v_pages) + slot * a.v_token_stride + u.g * a.D_v + d;
        for (int e = 0; e < 32; ++e) {
          const float x = __bfloat162float(v[e]);
          if (!(fabsf(x) < INFINITY)) o[e] += x;
        }
      }
    }
  }
}

template <int D, bool LO>
__global__ void __launch_bounds__(kThreads, 1)
    packed_tc_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ PackedTcPlan pl,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, LO>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // no room is left for aligning it here
    if (threadIdx.x == 0) atomicOr(a.status, STATUS_LAYOUT);
    return;
  }
  Bars<C>* bars = reinterpret_cast<Bars<C>*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_h / a.n_kv;
  asm volatile("griddepcontrol.launch_dependents;");  // the combine kernel may start to wait
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 2);  // the MMA issuer and warp 3, which passes every tile
      mbar_init(&bars->v_fixed[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars->q_full[w], 1);
      mbar_init(&bars->q_ready[w], 128);
      mbar_init(&bars->q_empty[w], 1);
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->p_full[w], 128);
      mbar_init(&bars->o_done[w], 1);
      mbar_init(&bars->o_empty[w], 128);
    }
    mbar_init(&bars->x_full, 128);
    mbar_init(&bars->x_done, 128);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&bars->piece_full[i], 1);
      mbar_init(&bars->piece_empty[i], 11);  // two producers, the MMA issuer, eight softmax warps
      mbar_init(&bars->care_done[i], 1);
    }
    mbar_init(&bars->fin, 1);
    bars->abort_flag = 0;
    bars->start_b = -1;
    bars->wc.abort_flag = &bars->abort_flag;
    bars->wc.status = a.status;
    bars->wc.limit_ns = a.wait_limit_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  // the line: thread i sums requests [i s, (i + 1) s)
  long long mine = 0, before, total = 0;
  const int strip = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, static_cast<int>(threadIdx.x) * strip), b_hi = min(a.B, b_lo + strip);
  for (int b = b_lo; b < b_hi; ++b) mine += Seg(a, pl, b).own() * a.n_kv;
  before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) bars->warp_sum[warp] = before;
  // rows behind the last request's
  {
    const long long row16 = static_cast<long long>(a.n_h) * D / 8;
    const long long from = packed_first(a, a.B) * row16, to = a.T * row16;
    for (long long i = from + blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < to; i += static_cast<long long>(gridDim.x) * kThreads) {
      static_cast<uint4*>(a.out)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse != nullptr && i % (D / 8) == 0) a.lse[i / (D / 8)] = -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  before -= mine;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += bars->warp_sum[w];
    total += bars->warp_sum[w];
  }
  const Cut cut(total, gridDim.x);
  const long long part_lo = cut.at(blockIdx.x), part_hi = cut.at(blockIdx.x + 1);
  if (part_lo < part_hi && part_lo >= before && part_lo < before + mine) {
    long long at = before;
    int b = b_lo;
    for (;; ++b) {
      const long long len = Seg(a, pl, b).own() * a.n_kv;
      if (part_lo < at + len) break;
      at += len;
    }
    bars->start_b = b;
    bars->start_off = part_lo - at;
  }
  __syncthreads();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl* const wc = &bars->wc;

  if (warp < 4) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ TMA producers
      const bool is_v = warp == 2;
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      uint8_t* const ring = smem + (is_v ? C::kVOff : C::kKOff);
      uint64_t* const full = is_v ? bars->v_full : bars->k_full;
      uint64_t* const empty = is_v ? bars->v_empty : bars->k_empty;
      const uint32_t n_stages = is_v ? C::kVStages : C::kKStages;
      if (lane == 0) tma_prefetch_desc(map);
      // rows per box: a page, or half of a 256-token page; a lane per box of a tile: block blk, rows from box_row on
      const int box_shift = min(a.page_shift, 7);
      const int boxes = BN >> box_shift;
      const int box = lane & (boxes - 1), blk = lane / boxes;
      const int box_row = box << box_shift;
      const bool loads = blk < C::kBlocks;
      const int page_mask = (1 << a.page_shift) - 1;
      Ring r;
      uint32_t q_ph = 0, q_used = 0;  // bits per worker: parity of its next query tile, whether one was loaded
      uint32_t issued = 0, last_ph = 0;
      bool ok = true;
      for (uint32_t n = 0;; ++n) {
        ok = warp_wait(&bars->piece_full[n % kQueue], (n / kQueue) & 1u, wc);
        if (!ok) break;
        const Piece* const pc = &bars->piece[n % kQueue];
        const int kind = pc->kind, g = pc->g, t_end = pc->t_end, klim = pc->klim;
        if (kind == kNone) break;
        const int* const table = a.block_table + static_cast<long long>(pc->b) * a.max_blocks;
        auto fetch = [&](int t) -> int {
          const int key = t * BN + box_row;  // t * BN < 2^31 - 2^16
          return loads && t < t_end && key < klim ? table[key >> a.page_shift] : -1;
        };
        int t = pc->t;
        int id = fetch(t);
        if (is_v) {
          for (int w = 0; w < 2; ++w) {
            if (Share(*pc, w).n == 0) continue;
            if (!warp_wait(&bars->q_empty[w], ((q_ph >> w) & 1u) ^ 1u, wc)) { ok = false; break; }
            if (lane == 0) {
              const int row = pc->row0 + (kind == kPair && w ? pl.tile_toks : 0);
              mbar_arrive_expect_tx(&bars->q_full[w], static_cast<uint32_t>(pl.tile_toks * G) * 128u * C::kBlocks);
              for (int d = 0; d < C::kBlocks; ++d)
                tma_load_4d(smem + C::kQOff + w * C::kTileBytes + d * C::kBlockBytes, &tm_q, &bars->q_full[w], d * 64, 0, g, row);
            }
            __syncwarp();
            q_ph ^= 1u << w;
            q_used |= 1u << w;
          }
          if (!ok) break;
        }
        for (; t < t_end; ++t) {
          if (!(ok = warp_wait(&empty[r.st], r.ph ^ 1u, wc))) break;
          const int n_boxes = (min(klim - t * BN, BN) + (1 << box_shift) - 1) >> box_shift;  // others hold no key
          if (lane == 0)
            mbar_arrive_expect_tx(&full[r.st], static_cast<uint32_t>(n_boxes * C::kBlocks) << (box_shift + 7));
          __syncwarp();
          if (loads && box < n_boxes)
            tma_load_4d(ring + r.st * C::kTileBytes + blk * C::kBlockBytes + box_row * 128, map, &full[r.st], blk * 64, g,
                        (t * BN + box_row) & page_mask, id);
          issued |= 1u << r.st;
          last_ph = (last_ph & ~(1u << r.st)) | (r.ph << r.st);
          r.next(n_stages);
          id = fetch(t + 1);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->piece_empty[n % kQueue]);
      }
      if (bars->abort_flag) {  // let every copy in flight land before shared memory goes away
        for (uint32_t s = 0; s < n_stages; ++s)
          if (issued & (1u << s)) drain_wait(&full[s], (last_ph >> s) & 1u, a.wait_limit_ns);
        for (int w = 0; w < 2; ++w)
          if (is_v && (q_used & (1u << w))) drain_wait(&bars->q_full[w], ((q_ph >> w) & 1u) ^ 1u, a.wait_limit_ns);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        const uint32_t q_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024));
        const uint32_t k_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024));
        const uint32_t v_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kVOff), C::kBlockBytes, 1024));
        const uint32_t lo_desc0 = ((smem_u32(smem + C::kLoOff) & 0x3FFFFu) >> 4) | ((BM * 16 >> 4) << 16);
        Ring kr, vr;
        uint32_t q_ph = 0, p_ph = 0, o_ph = 0, fix_ph = 0;  // parities, bits per worker (fix_ph: per V stage)
        // the K tile's byte offsets (>> 4) of the steps that Q's second part has
        uint32_t lo_off[LO ? C::kLoSteps : 1];
        if constexpr (LO) {
#pragma unroll
          for (int s = 0; s < C::kLoSteps; ++s) {
            const int kk = pl.lo_first + s;
            lo_off[s] = ((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4;
          }
        }
        // Q K^T: the steps of Q's first part, those of its second part
        auto qk_hi = [&](uint32_t w) {
          const uint32_t a0 = q_desc0 + ((w * C::kTileBytes) >> 4);
          const uint32_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < C::kSteps; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4;
            mma_ss_lo(tmem + w * 128u, a0 + off, b0 + off, C::kIdescQK, kk > 0 ? 1u : 0u);
          }
        };
        auto qk_lo = [&](uint32_t w) {
          const uint32_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int s = 0; s < C::kLoSteps; ++s)
            mma_lo(tmem + w * 128u, lo_desc0 + ((w * C::kLoBytes + s * (2 * BM * 16)) >> 4), b0 + lo_off[s], C::kIdescQK);
        };
        auto issue_qk = [&](uint32_t w) {
          qk_hi(w);
          qk_lo(w);
          mma_commit(&bars->s_full[w]);
        };
        // P V: P in columns 8 kk of the worker's S, its second part in columns 64 on
        auto issue_pv = [&](uint32_t w, bool first) {
          const uint32_t b0 = v_desc0 + ((vr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts_lo(tmem + C::kOCol + w * D, tmem + w * 128u + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescPV,
                      (!first || kk > 0) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < C::kPLoSteps; ++kk)
            mma_ts_lo(tmem + C::kOCol + w * D, tmem + w * 128u + 64 + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescPV, 1u);
        };
        auto wait_p = [&](uint32_t w) -> bool {
          const bool there = lane_wait(&bars->p_full[w], (p_ph >> w) & 1u, wc);
          p_ph ^= 1u << w;
          return there;
        };
        auto wait_o = [&](uint32_t w) -> bool {  // O has been read
          const bool there = lane_wait(&bars->o_empty[w], ((o_ph >> w) & 1u) ^ 1u, wc);
          o_ph ^= 1u << w;
          return there;
        };
        auto wait_q = [&](uint32_t w) -> bool {
          const bool there = lane_wait(LO ? &bars->q_ready[w] : &bars->q_full[w], (q_ph >> w) & 1u, wc);
          q_ph ^= 1u << w;
          return there;
        };
        auto wait_k = [&]() -> bool { return lane_wait(&bars->k_full[kr.st], kr.ph, wc); };
        auto wait_v = [&](bool care) -> bool {  // care: treated by warp 3
          if (!care) return lane_wait(&bars->v_full[vr.st], vr.ph, wc);
          const bool there = lane_wait(&bars->v_fixed[vr.st], (fix_ph >> vr.st) & 1u, wc);
          fix_ph ^= 1u << vr.st;
          return there;
        };
        auto k_done = [&]() {
          mma_commit(&bars->k_empty[kr.st]);
          kr.next(C::kKStages);
        };
        auto v_done = [&]() {
          mma_commit(&bars->v_empty[vr.st]);
          vr.next(C::kVStages);
        };
        for (uint32_t n = 0;; ++n) {
          if (!lane_wait(&bars->piece_full[n % kQueue], (n / kQueue) & 1u, wc)) break;
          const Piece* const pc = &bars->piece[n % kQueue];
          const int kind = pc->kind, nv = pc->t_end - pc->t, care = pc->care_t - pc->t;
          const int n0 = Share(*pc, 0).n;
          if (kind == kNone) break;
          mbar_arrive(&bars->piece_empty[n % kQueue]);
          bool ok = true;
          if (kind == kPair) {
            if (!wait_k()) break;
            if (n0 > 0) {
              if (!wait_q(0)) break;
              tc_fence_after();
              issue_qk(0);
              if (n0 == 1) mma_commit(&bars->q_empty[0]);
            }
            if (!wait_q(1)) break;
            tc_fence_after();
            issue_qk(1);
            if (nv == 1) mma_commit(&bars->q_empty[1]);
            k_done();
            const int ve = min(n0 - 2, care);
            for (int v = 0; v < nv; ++v) {
              if (v > 0 && v < ve) {
                // Both workers take this tile and two more, and no care is needed: a loop without decisions, in which
                // the waits for the next turn's tiles stand before this turn's last MMAs, so that the tensor pipe
                // does not run dry.
                if (!(ok = wait_v(false) && wait_k())) break;
                for (; v < ve; ++v) {
                  if (!(ok = wait_p(0))) break;
                  tc_fence_after();
                  issue_pv(0, false);
                  issue_qk(0);
                  if (!(ok = wait_p(1))) break;
                  tc_fence_after();
                  issue_pv(1, false);
                  v_done();
                  qk_hi(1);
                  Ring kn = kr;
                  kn.next(C::kKStages);
                  if (v + 1 < ve && !(ok = wait_v(false) && lane_wait(&bars->k_full[kn.st], kn.ph, wc))) break;
                  qk_lo(1);
                  mma_commit(&bars->s_full[1]);
                  mma_commit(&bars->k_empty[kr.st]);
                  kr = kn;
                }
                if (!ok) break;
              }
              const bool next = v + 1 < nv;
              if (!(ok = wait_v(v >= care))) break;
              bool have_k = false;
              if (v < n0) {
                if (!(ok = wait_p(0) && (v > 0 || wait_o(0)))) break;
                tc_fence_after();
                issue_pv(0, v == 0);
                if (v == n0 - 1) {
                  mma_commit(&bars->o_done[0]);
                } else {
                  if (!(ok = wait_k())) break;
                  have_k = true;
                  issue_qk(0);
                  if (v + 2 == n0) mma_commit(&bars->q_empty[0]);
                }
              }
              if (!(ok = wait_p(1) && (v > 0 || wait_o(1)))) break;
              tc_fence_after();
              issue_pv(1, v == 0);
              v_done();
              if (!next) {
                mma_commit(&bars->o_done[1]);
              } else {
                if (!have_k && !(ok = wait_k())) break;
                issue_qk(1);
                if (v + 2 == nv) mma_commit(&bars->q_empty[1]);
                k_done();
              }
            }
          } else {
            for (int v = 0; v < 2 && v < nv; ++v) {
              if (!(ok = wait_k() && wait_q(v))) break;
              tc_fence_after();
              issue_qk(v);
              k_done();
              if (v + 2 >= nv) mma_commit(&bars->q_empty[v]);
            }
            for (int v = 0; ok && v < nv; ++v) {
              const uint32_t w = v & 1;
              if (!(ok = wait_v(v >= care) && wait_p(w) && (v >= 2 || wait_o(w)))) break;
              tc_fence_after();
              issue_pv(w, v < 2);
              v_done();
              if (v + 2 >= nv) {
                mma_commit(&bars->o_done[w]);
              } else {
                if (!(ok = wait_k())) break;
                issue_qk(w);
                k_done();
                if (v + 4 >= nv) mma_commit(&bars->q_empty[w]);
              }
            }
          }
          if (!ok) break;
        }
        // every MMA issued so far completes before TMEM is released
        mma_commit(&bars->fin);
        drain_wait(&bars->fin, 0, a.wait_limit_ns);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ the walk, and care tiles
      Walk walk{0, 0, 0, 0, part_hi - part_lo, bars->start_b >= 0};
      if (walk.live) {
        const Seg s(a, pl, bars->start_b);
        const long long own = s.own();
        long long off = bars->start_off;
        walk.b = bars->start_b;
        walk.g = static_cast<int>(off / own);
        off -= walk.g * own;
        int lo = 0, hi = s.np;  // the last segment that starts at or before off
        if (s.rem == 0) --hi;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s.before(mid) <= off) lo = mid;
          else hi = mid - 1;
        }
        off -= s.before(lo);
        walk.p = lo;
        walk.end += off;
        walk.t = tile_at(off, s.lead(lo), s.weight(lo), tiles_of(s.seen(lo, min(2 * s.tt, s.r.rows - lo * 2 * s.tt))));
      }
      Record* const rec = reinterpret_cast<Record*>(static_cast<float*>(a.workspace) + pl.rec) + 2 * blockIdx.x;
      uint32_t recs = 0;  // bits: slots with a record
      uint32_t n_pub = 0;
      bool last = false;  // the end has been handed out
      Ring r;
      for (uint32_t n = 0;; ++n) {
        bool ok = true;
        for (; !last && n_pub < n + kAhead; ++n_pub) {
          const uint32_t e = n_pub % kQueue;
          if (n_pub >= kQueue && !(ok = warp_wait(&bars->piece_empty[e], (n_pub / kQueue - 1) & 1u, wc))) break;
          if (lane == 0) {
            Piece* const u = &bars->piece[e];
            next_piece(a, pl, walk, u);
            if (u->kind != kNone && u->slot >= 0) {
              rec[u->slot] = Record{u->kind, u->g, u->row0, u->ntok, u->t, u->t_end, u->kt, 0};
              recs |= 1u << u->slot;
            }
            last = u->kind == kNone;
            mbar_arrive(&bars->piece_full[e]);
          }
          last = __shfl_sync(0xffffffffu, last ? 1 : 0, 0) != 0;
        }
        if (!ok) break;
        __syncwarp();
        Piece* const u = &bars->piece[n % kQueue];
        if (u->kind == kNone) break;
        const int care = u->care_t, klim = u->klim;
        uint32_t any = 0;
        for (int t = u->t; t < u->t_end; ++t) {
          if (!(ok = warp_wait(&bars->v_full[r.st], r.ph, wc))) break;
          if (t >= care) {
            uint8_t* const v = smem + C::kVOff + r.st * C::kTileBytes;
#pragma unroll 1
            for (int q = 0; q < BN / 32; ++q) {
              // lane l: row 32 q + l, whose 16-byte pieces it takes from another one on than its neighbours
              const int row = 32 * q + lane;
              uint8_t* const p = v + row * 128;
              bool bad = false;
              if (t * BN + row >= klim) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                  *reinterpret_cast<uint4*>(p + (i >> 3) * C::kBlockBytes + (((i + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
              } else {
                uint32_t ones = 0;  // bits 15 and 31: an exponent of all ones
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                  const uint4 x = *reinterpret_cast<const uint4*>(p + (i >> 3) * C::kBlockBytes + (((i + lane) & 7) << 4));
                  ones |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                          ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                }
                bad = (ones & 0x80008000u) != 0;
                if (bad) {
#pragma unroll 1
                  for (int i = 0; i < D / 2; ++i) {
                    uint32_t* const y = reinterpret_cast<uint32_t*>(p + (i >> 5) * C::kBlockBytes + (i & 31) * 4);
                    uint32_t x = *y;
                    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                    *y = x;
                  }
                }
              }
              const uint32_t bits = __ballot_sync(0xffffffffu, bad);
              if (lane == 0 && t - care < kCare) u->bad[t - care][q] = bits;
              any |= bits;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->v_fixed[r.st]);
          }
          if (lane == 0) mbar_arrive(&bars->v_empty[r.st]);
          r.next(C::kVStages);
        }
        if (!ok) break;
        if (lane == 0) {
          u->bad_any = any;
          mbar_arrive(&bars->care_done[n % kQueue]);
        }
        __syncwarp();
      }
      if (lane < 2 && !((__shfl_sync(0x3u, recs, 0) >> lane) & 1u)) rec[lane] = Record{0, 0, 0, 0, 0, 0, 0, 0};
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax warpgroups (workers)
    const int w = (warp - 4) >> 2;
    const int quad = warp & 3;       // TMEM lane quadrant
    const int r = quad * 32 + lane;  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + (w ? 128u : 0u);
    const uint32_t o_addr = tmem + lane_off + C::kOCol + (w ? D : 0);
    const int my_tok = r / G;  // token of this row in its tile
    uint32_t s_ph = 0, q_ph = 0, o_ph = 0, x_ph = 0;
    bool ok = true;
    const float2* const angles = reinterpret_cast<const float2*>(static_cast<const float*>(a.workspace) + pl.angles);
    // Query tile of piece e of the queue, if this worker has one: rotate this thread's row and hand it over.
    auto prepare = [&](const Piece* u) -> bool {
      if constexpr (LO) {
        if (u->kind == kNone || Share(*u, w).n == 0) return true;
        if (!row_wait(&bars->q_full[w], q_ph, wc)) return false;
        q_ph ^= 1u;
        const int tok = (u->kind == kPair && w ? pl.tile_toks : 0) + my_tok;
        if (my_tok < pl.tile_toks && tok < u->ntok) {
          rotate_row<2 * C::kLoSteps>(smem + C::kQOff + w * C::kTileBytes, smem + C::kLoOff + w * C::kLoBytes, r,
                                      angles + static_cast<long long>(u->row0 + tok) * pl.n_pairs, a.rope_offset, pl.n_pairs,
                                      pl.half != 0, 2 * pl.lo_first);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->q_ready[w]);
      }
      return true;
    };
    if constexpr (LO) asm volatile("griddepcontrol.wait;" ::: "memory");  // the angles are there
    ok = row_wait(&bars->piece_full[0], 0, wc) && prepare(&bars->piece[0]);
    for (uint32_t n = 0; ok; ++n) {
      const Piece* const u = &bars->piece[n % kQueue];
      const int kind = u->kind;
      if (kind == kNone) break;
      const Share sh(*u, w);
      const int tok = (kind == kPair && w ? pl.tile_toks : 0) + my_tok;
      const bool real = my_tok < pl.tile_toks && tok < u->ntok;  // this row is a query
      const int place = u->place0 + tok;
      bool dead = !real || place < 0;
      uint32_t bits[4] = {0u, 0u, 0u, 0u};
      if (real) {
        const long long row = u->row0 + tok;
        if (a.positions != nullptr && a.positions[row] < 0) dead = true;
        if (a.visible != nullptr) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < a.words) bits[i] = static_cast<uint32_t>(a.visible[row * a.words + i]);
        }
      }
      const int lim = dead ? 0 : place + 1;
      float m_run = -INFINITY, l_run = 0.f;
      {
        const int care = u->care_t, base = u->base, klim = u->klim;
        int t = sh.first;
        for (int i = 0; i < sh.n; ++i, t += sh.step) {
          if (!row_wait(&bars->s_full[w], s_ph, wc)) { ok = false; break; }
          s_ph ^= 1u;
          tc_fence_after();
          uint32_t mask[4];
          const bool masked = t >= care;
          if (masked) {
            if (a.visible != nullptr) seen_tree(bits, base, klim, t * BN, mask);
            else seen_below(lim, t * BN, mask);
          }
          softmax_row<D, 16 * C::kPLoSteps>(s_addr, o_addr, masked, mask, i > 0, a.scale_log2, m_run, l_run);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[w]);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      if (!row_wait(&bars->piece_full[(n + 1) % kQueue], ((n + 1) / kQueue) & 1u, wc)) break;
      if (!prepare(&bars->piece[(n + 1) % kQueue])) break;

      // epilogue: the rows of the output, or the piece's normalised partial and its log-sum-exp
      if (sh.n > 0) {
        if (!row_wait(&bars->o_done[w], o_ph, wc)) break;
        o_ph ^= 1u;
      }
      // a single piece of more than one tile has a part of each row in both workers: worker 0 joins them
      const bool both = kind == kSingle && Share(*u, 1).n > 0;
      float2* const ml = reinterpret_cast<float2*>(smem + C::kMlOff) + r;
      float f0 = l_run > 0.f ? 1.f / l_run : l_run, f1 = 0.f;  // factors of O of this worker, and of worker 1
      if (both) {
        if (w == 1) {
          if (!row_wait(&bars->x_done, x_ph ^ 1u, wc)) break;
          *ml = make_float2(m_run, l_run);
          tc_fence_before();
          mbar_arrive(&bars->x_full);
        } else {
          if (!row_wait(&bars->x_full, x_ph, wc)) break;
          const float2 o = *ml;
          mbar_arrive(&bars->x_done);
          const float m = fmaxf(m_run, o.x), m_ref = m == -INFINITY ? 0.f : m;
          f0 = fast_exp2(m_run - m_ref);
          f1 = fast_exp2(o.x - m_ref);
          l_run = l_run * f0 + o.y * f1;
          m_run = m;
          const float inv = l_run > 0.f ? 1.f / l_run : l_run;
          f0 *= inv;
          f1 *= inv;
        }
        x_ph ^= 1u;
      }
      if (kind == kPair || w == 0) {
        if (!row_wait(&bars->care_done[n % kQueue], (n / kQueue) & 1u, wc)) break;
        const bool whole = u->slot < 0;
        const bool none = dead || l_run == 0.f;  // no key with a weight; NaN is one
        const bool bad = u->bad_any != 0;
        const int lj = lane & 3, r4 = r - lj;  // rows r4 .. r4 + 3 are stored by four lanes together, 64 bytes of each
        float* const ws = static_cast<float*>(a.workspace);
        const long long slot_row = (2 * static_cast<long long>(blockIdx.x) + (whole ? 0 : u->slot)) * pl.slot_rows + w * BM;
        int at[4];  // their rows of the output, -1: not a query
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tk = (r4 + k) / G, i = (r4 + k) - tk * G, tok_k = (kind == kPair && w ? pl.tile_toks : 0) + tk;
          at[k] = tk < pl.tile_toks && tok_k < u->ntok ? (u->row0 + tok_k) * a.n_h + u->g * G + i : -1;
        }
        const float lse2 = none ? -INFINITY : m_run + log2f(l_run);
        if (real) {
          if (!whole) ws[pl.l + slot_row + r] = lse2;
          else if (a.lse != nullptr)
            a.lse[static_cast<long long>(u->row0 + tok) * a.n_h + u->g * G + (r - my_tok * G)] = lse2 * 0.69314718055994530942f;
        }
        if (sh.n > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            {
              uint32_t x[32];
              tmem_ld32(o_addr + c, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(x[e]) * f0;
              if (both) {
                tmem_ld32(o_addr + D + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(x[e]), f1, o[e]);
              }
            }
            if (bad && real) {
              float y[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = o[e];
              add_bad(a, *u, lim, bits, c, y);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = y[e];
            }
            if (none) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
            uint4 pc[4];
            if (whole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) pc[e] = f32_to_bf16x8(o + 8 * e);
              transpose_pieces(pc, lj);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (at[k] >= 0)
                  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<long long>(at[k]) * D + c + lj * 8) = pc[k];
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  pc[e] = make_uint4(__float_as_uint(o[16 * h + 4 * e]), __float_as_uint(o[16 * h + 4 * e + 1]),
                                     __float_as_uint(o[16 * h + 4 * e + 2]), __float_as_uint(o[16 * h + 4 * e + 3]));
                transpose_pieces(pc, lj);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (at[k] >= 0)
                    *reinterpret_cast<uint4*>(ws + (slot_row + r4 + k) * D + c + 16 * h + lj * 4) = pc[k];
              }
            }
          }
          tc_fence_before();
          mbar_arrive(&bars->o_empty[w]);
          if (both) mbar_arrive(&bars->o_empty[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->piece_empty[n % kQueue]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Blocks (CTA c of the kernel before, rows): if c's last piece is the head of a segment that goes on in the next
// CTAs' first pieces, its rows are joined, a warp per row: the weights of the pieces by lanes, then D dims.
constexpr int kJoinWarps = 8, kJoinRows = 16;
constexpr int kMaxCtas = 160;  // the workspace is sized for this many (a GB300 has 152 SMs)

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    packed_tc_join_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ PackedTcPlan pl) {
  constexpr int kPer = D / 32;  // dims per lane
  __shared__ int slots[kMaxCtas];
  __shared__ float weights[kJoinWarps][kMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* const ws = static_cast<const float*>(a.workspace);
  const Record* const rec = reinterpret_cast<const Record*>(ws + pl.rec);
  const int parts = (pl.slot_rows + kJoinRows - 1) / kJoinRows;
  const int c = blockIdx.x / parts, part = blockIdx.x - c * parts;
  const Record head = rec[2 * c + 1];
  const int G = a.n_h / a.n_kv;
  if (head.kt == 0 || part * kJoinRows >= (head.kind == kPair ? 2 * BM : min(BM, head.ntok * G))) return;
  // the pieces: this one, then first pieces up to the one that ends the segment (a CTA may hold none)
  if (threadIdx.x == 0) slots[0] = 2 * c + 1;
  int n = 1;
  for (int c0 = c + 1; c0 < pl.ctas; c0 += 32) {
    const int cc = c0 + lane;
    const int kt = cc < pl.ctas ? rec[2 * cc].kt : 0, t_end = kt ? rec[2 * cc].t_end : 0;
    const uint32_t end = __ballot_sync(0xffffffffu, kt > 0 && t_end == kt);
    const uint32_t upto = end ? (end & (0u - end)) * 2u - 1u : 0xffffffffu;  // lanes up to the first that ends it
    const uint32_t some = __ballot_sync(0xffffffffu, kt > 0) & upto;
    if (warp == 0 && ((some >> lane) & 1u)) slots[n + __popc(some & ((1u << lane) - 1u))] = 2 * cc;
    n += __popc(some);
    if (end) break;
  }
  __syncthreads();
  float* const wt = weights[warp];
  for (int k = warp; k < kJoinRows; k += kJoinWarps) {
    const int rr = part * kJoinRows + k, r = rr & (BM - 1), w = rr / BM;
    const int tk = r / G, tok = (w ? pl.tile_toks : 0) + tk;
    if (tk >= pl.tile_toks || tok >= head.ntok || (w && head.kind != kPair)) continue;
    float m = -INFINITY;
    for (int j = lane; j < n; j += 32) {
      const float x = ws[pl.l + static_cast<long long>(slots[j]) * pl.slot_rows + rr];
      wt[j] = x;
      m = fmaxf(m, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float m_ref = m == -INFINITY ? 0.f : m;
    float den = 0.f;
    for (int j = lane; j < n; j += 32) {
      const float x = exp2f(wt[j] - m_ref);
      wt[j] = wt[j] == -INFINITY ? -1.f : x;  // nothing there
      den += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    __syncwarp();
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float x = wt[j];
      if (x == -1.f) continue;
      const float* const p = ws + (static_cast<long long>(slots[j]) * pl.slot_rows + rr) * D + lane * kPer;
      float v[kPer];
      if constexpr (kPer == 4) {
        const float4 y = *reinterpret_cast<const float4*>(p);
        v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(p);
        v[0] = y.x; v[1] = y.y;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(x, v[e], acc[e]);
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const long long at = (static_cast<long long>(head.row0) + tok) * a.n_h + head.g * G + (r - tk * G);
    uint32_t* const out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at * D + lane * kPer);
    out[0] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if constexpr (kPer == 4) out[1] = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[at] = den == 0.f ? -INFINITY : (m + log2f(den)) * 0.69314718055994530942f;
    __syncwarp();
  }
}

PackedTcPlan make_plan(const PackedArgs& a, int ctas, int max_ctas, int n_pairs, int half) {
  PackedTcPlan p{};
  const int G = a.n_h / a.n_kv;
  p.ctas = ctas;
  p.tile_toks = BM / G;
  p.slot_rows = a.T <= p.tile_toks ? a.T * G : 2 * BM;
  const int steps = a.D_qk / 16, rest = steps - a.D_qk / 32;
  p.lo_first = n_pairs ? (a.rope_offset / 16 < rest ? a.rope_offset / 16 : rest) : 0;
  p.n_pairs = n_pairs;
  p.half = half;
  p.l = 2LL * max_ctas * p.slot_rows * a.D_v;
  p.rec = (p.l + 2LL * max_ctas * p.slot_rows + 3) & ~3LL;
  p.angles = p.rec + 2LL * max_ctas * static_cast<long long>(sizeof(Record) / 4);
  p.end = p.angles + 2LL * a.T * n_pairs;
  return p;
}

// Opt in to the kernel's shared memory and check that the compiled kernel holds enough
// registers per thread for its register split (setmaxnreg.inc would wait forever otherwise).
template <int D, bool LO>
cudaError_t prepare() {
  static std::atomic<unsigned long long> ready{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, packed_tc_kernel<D, LO>)) != cudaSuccess) return e;
  if (static_cast<long long>(fa.numRegs) * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(packed_tc_kernel<D, LO>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<Cfg<D, LO>>());
  if (e != cudaSuccess) return e;
  ready.fetch_or(bit, std::memory_order_acq_rel);
  return cudaSuccess;
}

template <int D, bool LO>
cudaError_t launch(const PackedArgs& a, const RopeFreq& rope, const CUtensorMap* maps, const PackedTcPlan& pl,
                   cudaStream_t st, int* launches) {
  cudaError_t e = prepare<D, LO>();
  if (e != cudaSuccess) return e;
  if (LO) {
    const long long items = static_cast<long long>(a.T) * rope.n_pairs;
    packed_angles_kernel<<<static_cast<unsigned>((items + 255) / 256), 256, 0, st>>>(
        a, rope, reinterpret_cast<float2*>(static_cast<float*>(a.workspace) + pl.angles));
    *launches += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_early(packed_tc_kernel<D, LO>, pl.ctas, kThreads, smem_bytes<Cfg<D, LO>>(), st, LO, a, pl, maps[0], maps[1],
                   maps[2]);
  *launches += 1;
  if (e != cudaSuccess) return e;
  const unsigned parts = (pl.slot_rows + kJoinRows - 1) / kJoinRows;
  e = launch_early(packed_tc_join_kernel<D>, pl.ctas * parts, kJoinWarps * 32, 0, st, true, a, pl);
  *launches += 1;
  return e;
}

}  // namespace

bool packed_tc_supported(const PackedArgs& a, bool bf16, int rope_offset, int rope_dims, bool rope, bool half) {
  return bf16 && a.D_qk == a.D_v && (a.D_qk == 64 || a.D_qk == 128) && a.n_h / a.n_kv <= BM &&
         (!rope || (rope_offset % 8 == 0 && rope_dims % (half ? 16 : 8) == 0));
}

size_t packed_tc_workspace(const PackedArgs& a) {
  return static_cast<size_t>(make_plan(a, kMaxCtas, kMaxCtas, a.D_qk / 2, 0).end) * sizeof(float);
}

cudaError_t launch_packed_tc(const PackedArgs& a, const RopeFreq& rope, int num_sms, cudaStream_t st, int* launches) {
  const bool rotate = rope.n_pairs > 0;
  int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  // no more CTAs than the call can have tiles
  const long long segments = static_cast<long long>(a.T) * (a.n_h / a.n_kv) / (2 * BM - 2 * (a.n_h / a.n_kv) + 2) + a.B;
  const long long most = segments * a.n_kv * (((static_cast<long long>(a.max_blocks) << a.page_shift) + BN - 1) / BN);
  if (most < ctas) ctas = most > 0 ? static_cast<int>(most) : 1;
  const PackedTcPlan pl = make_plan(a, ctas, kMaxCtas, rope.n_pairs, rope.half);
  // query rows by (dim, head of the group, KV head, row), a row tile per box; K and V by (dim, KV head, row in
  // page, page), a page or a part of it per box
  const unsigned long long hs = static_cast<unsigned long long>(a.D_qk) * 2, page = 1ull << a.page_shift;
  const unsigned long long ks = hs * a.n_kv, vs = static_cast<unsigned long long>(a.v_token_stride) * 2;
  const int G = a.n_h / a.n_kv, rows = static_cast<int>(page);
  CUtensorMap maps[3];
  const bool wide = a.D_qk == 128;
  if (!make_map_box(&maps[0], a.q, a.D_qk, G, a.n_kv, a.T, hs, hs * G, hs * a.n_h, G, 1, pl.tile_toks, wide) ||
      !make_map_box(&maps[1], a.k_pages, a.D_qk, a.n_kv, rows, a.n_pages, hs, ks, ks * page, 1, rows < 128 ? rows : 128, 1, wide) ||
      !make_map_box(&maps[2], a.v_pages, a.D_v, a.n_kv, rows, a.n_pages, hs, vs, vs * page, 1, rows < 128 ? rows : 128, 1, wide))
    return cudaErrorInvalidValue;
  if (a.D_qk == 64)
    return rotate ? launch<64, true>(a, rope, maps, pl, st, launches) : launch<64, false>(a, rope, maps, pl, st, launches);
  return rotate ? launch<128, true>(a, rope, maps, pl, st, launches) : launch<128, false>(a, rope, maps, pl, st, launches);
}

}  // namespace attn
