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
// Rounding.  Sums and softmax statistics are fp32.  With RoPE a query is rotated by a kernel before and kept as the sum of
// two bf16 values, the second for 64 dims (from the start of the rotated span on), and with D = 128 the weights of
// each tile's last 64 keys are such sums too; the other weights are rounded to bf16 once.  One bf16 for both made the output's
// error against 64 bits 1.7 times that of its own rounding behind 30000 keys (normally distributed inputs); so it is
// 1.41 to 1.44 times, as without RoPE, where queries are exact and weights are rounded once.  The second parts are half as
// much work again for the tensor pipe, with D = 128 (24 MMAs of 128 columns for 16 per row tile and 128 keys) and with D = 64 (4
// of 128 columns beside 4 of 128 and 8 of 64), on the K and V tiles that are there anyway: 4 x 8192 tokens, 32 heads
// over 8, 2.0 to 2.1 ms, without RoPE 1.4 to 1.5; with 64 dims 1.23 and 1.12.
//
// What a row does not see.  Scores are masked by index.  A value whose weight is 0 still meets the MMA, so in
// the tiles that some row sees in part ("care" tiles: the last ones of a segment) warp 3 clears value rows
// behind the last key and replaces infinities and NaN by 0, noting their keys; the epilogue adds such
// values, times their weights, to the rows that do see them.  The rest of the tiles is seen whole by every row.
//
// A CTA (384 threads): warp 0 loads K tiles by TMA, warp 2 query rows and V tiles, a lane per box (two stages of
// each fill what shared memory both parts of two query tiles leave); warp 1 issues the MMAs; warp 3
// walks the line, hands the pieces out through a queue in shared memory and treats care tiles; warps
// 4-7 and 8-11 are the softmax of row tiles 0 and 1 (or of alternate key tiles), a row per thread.
// TMEM: S/P of the two in columns [0, 128) and [128, 256), O behind them.
//
// Bounds.  Long prompts: the tensor pipe (1 x 8192 tokens, 32 heads over 8, D = 128, RoPE: its counter is active 82% of
// the time; a turn of a pair piece - two row tiles, 128 keys - is 48 MMAs of 64 cycles and takes 3500 to 3600).  4 x 8192:
// 2.0 to 2.1 ms, 1.05 to 1.1 PFLOP/s as the formula counts and 1.6 as issued.  Drafts behind long caches: HBM (59 requests of 32
// drafts behind 4096 to 8192 tokens: 1.53 GB read in 243 us, 6.3 TB/s).  Few short requests: the chain launch, walk, TMA,
// MMA, softmax, MMA, store, and a join (one prompt of 77 tokens 14 us).  Heads of 64 dims: neither the tensor pipe (59% of
// the time, 1 x 8192 tokens) nor the exponentials (39% of their pipe).  Short prompts, where a start and end of a piece costs
// some 11000 to 14000 cycles beside its turns (16 prompts): per instruction issued, warps wait 3.5 cycles on long scoreboards
// (memory, TMEM and the like) and 0.77 for an instruction; in one long prompt 3.8 and 0.25, with 0.16 requests per cycle to
// a group of SMs' instruction cache instead of 0.43.  Five programs run side by side on an SM, so loops stay rolled and rare
// code is out of line.
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
  unsigned long long nth;  // 2^64 / ctas
  // float offsets into the workspace: partials [2 * ctas, slot_rows, D], their log-sum-exps, records, the rotated
  // queries (bf16 [T, n_h, D]) and what that rounding left (bf16 [T, n_h, 64])
  long long l, rec, q, lo, end;
};

namespace {

constexpr int BM = 128;  // rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kLoDims = 64;  // dims with a second part of Q: a column block
constexpr int kCare = 3;   // care tiles of a piece, at most: 256 tokens of a pair, or 128 drafts
constexpr int kQueue = 6;  // pieces in the queue; kAhead are handed out before warp 3 treats the first of them
constexpr int kAhead = 3;

// Points on the line: 2^shift per key of a segment, and a lead in front of its first tile, three tiles of a pair: of the 11000
// to 14000 cycles that starting and ending a piece takes, a single one saves little.  (With 2048 and 1024, 64 prompts of up to
// 500 tokens, 32 heads over 8, took 240 us instead of 214, 30 trees of up to 64 drafts, 16 heads, 52 instead of 43, 128 single
// tokens behind up to 3000 166 instead of 150; 4096 for either was no better.)
constexpr int kPairShift = 3, kSingleShift = 2;
constexpr int kPairLead = 3 * BN << kPairShift, kSingleLead = kPairLead;

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
  [[maybe_unused]] static constexpr int kLoSteps = LO ? kLoDims / 16 : 0;       // MMA steps with a second part of Q
  static constexpr int kLoBytes = LO ? kBlockBytes : 0;        // of a row tile
  static constexpr int kPLoSteps = LO && D == 128 ? 4 : 0;    // steps of 16 keys with a second part of P
  static constexpr int kKStages = 2;
  static constexpr int kVStages = 2;
  static_assert(kKStages == 2 && kVStages == 2, "the MMA issuer's turns are written for two stages");
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kLoOff = kVOff + kVStages * kTileBytes;
  static constexpr int kMlOff = kLoOff + 2 * kLoBytes;         // worker 1's maximum and sum of each row
  static constexpr int kMaxOff = kMlOff + BM * 8;              // the maximum of both workers
  static constexpr int kBarOff = kMaxOff + BM * 4;
  static constexpr uint32_t kOCol = 256;                       // O of worker w at kOCol + w D
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, true);
};

template <typename C>
struct Bars {
  uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  uint64_t v_full[C::kVStages], v_empty[C::kVStages], v_fixed[C::kVStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t x_full, x_back, x_done;  // single pieces: worker 1's sums are there, the rows' factors, worker 1 has read O
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
  __device__ __forceinline__ int shift(int p) const { return is_pair(p) ? kPairShift : kSingleShift; }
  __device__ __forceinline__ int lead(int p) const { return is_pair(p) ? kPairLead : kSingleLead; }
  __device__ __forceinline__ int count() const { return np + (rem > 0); }
  __device__ __forceinline__ long long keys_of(int p) const {  // for the length
    return tree ? keys : static_cast<long long>(keys) + min((p + 1) * 2 * tt, r.rows);
  }
  __device__ __forceinline__ long long length(int p) const { return lead(p) + (keys_of(p) << shift(p)); }
  // points in front of pair p <= np
  __device__ __forceinline__ long long before(int p) const {
    const long long q = p;
    return q * kPairLead + ((q * keys + (tree ? 0 : tt * q * (q + 1))) << kPairShift);
  }
  __device__ __forceinline__ long long own() const { return before(np) + (rem > 0 ? length(np) : 0); }
  // real keys of the segment's first n tokens, at least 1
  __device__ __forceinline__ int seen(int p, int n) const {
    return tree ? keys : max(min(r.len, r.base + p * 2 * tt + n), 1);
  }
};
__device__ __forceinline__ int tiles_of(int keys) { return static_cast<int>((static_cast<unsigned>(keys) + BN - 1) / BN); }
// The first tile that starts at or behind point x of a segment of kt tiles.
__device__ __forceinline__ int tile_at(long long x, int lead, int shift, int kt) {
  const long long d = x - lead;
  if (d <= 0) return 0;
  const long long t = (d + (BN << shift) - 1) >> (shift + 7);
  return t < kt ? static_cast<int>(t) : kt;
}
static_assert(BN == 1 << 7, "tile_at");

// A walk along one CTA's part: the segment (b, g, p), its next tile, and the part's end from its first point.
struct Walk {
  int b, g, p, t;
  long long end;
  bool live;
};

// To the next request that has rows, 32 at a time: the warp's lanes all walk alike.
__device__ __forceinline__ void next_request(const PackedArgs& a, Walk& w, int lane) {
  w.g = w.p = w.t = 0;
  for (int b = w.b + 1; b < a.B; b += 32) {
    const uint32_t some = __ballot_sync(0xffffffffu, b + lane < a.B && packed_request(a, b + lane).rows > 0);
    if (some) {
      w.b = b + __ffs(some) - 1;
      return;
    }
  }
  w.live = false;
}

// The next piece of a walk (kind kNone at its end).
// All lanes have its kind, slot and place in the line; lane 0 writes it.
__device__ __forceinline__ int next_piece(const PackedArgs& a, const PackedTcPlan& pl, Walk& w, Piece* out, int lane) {
  while (w.live && w.end > 0) {
    const Seg s(a, pl, w.b);
    const int p = w.p;
    const bool pair = s.is_pair(p);
    const int tok0 = p * 2 * s.tt, ntok = min(2 * s.tt, s.r.rows - tok0);
    const int klim = s.seen(p, ntok), kt = tiles_of(klim);
    const int t = w.t, t_end = tile_at(w.end, s.lead(p), s.shift(p), kt);
    if (t < t_end && lane == 0) {
      Piece u;
      u.kind = pair ? kPair : kSingle;
      u.g = w.g;
      u.b = w.b;
      u.row0 = s.r.first + tok0;
      u.ntok = ntok;
      u.t = t;
      u.t_end = t_end;
      u.kt = kt;
      u.kt0 = pair ? tiles_of(s.seen(p, s.tt)) : kt;
      u.place0 = s.r.base + tok0;
      u.base = s.r.base;
      u.klim = klim;
      u.care_t = max(s.tree ? s.r.base : s.r.base + tok0 + 1, 0) / BN;
      u.slot = t > 0 ? 0 : t_end < kt ? 1 : -1;
      u.bad_any = 0;
      *out = u;
    }
    w.t = t_end;
    if (t_end < kt) {  // the part ends here
      w.live = false;
    } else {
      w.t = 0;
      w.end -= s.length(p);
      if (++w.p == s.count()) {
        w.p = 0;
        if (++w.g == a.n_kv) next_request(a, w, lane);
      }
    }
    if (t < t_end) return pair ? kPair : kSingle;
  }
  w.live = false;
  if (lane == 0) out->kind = kNone;
  return kNone;
}

// One lane of a converged warp, which the compiler knows to be one: the MMA issuer's descriptors then stay in uniform
// registers (behind a test of the lane's number, each MMA took the issuer 70 to 90 cycles, more than the tensor pipe's 64,
// and a turn inside a pair piece 4680 cycles; 4 prompts of 8192 tokens 2388 -> 2017 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

// ------------------------------------------------------------------------------------- rows
// The new tokens' queries rotated at their positions, bf16 [T, n_h, D], and what that rounding left of dims
// [lo_dim, lo_dim + 64), bf16 [T, n_h, 64].  A thread owns 8 dims (and with split halves their partners) of a token for
// heads_per heads, so that an angle is computed once for all of them; bound by HBM (32768 tokens of 32 heads of 128 dims
// 104 us, 6.4 TB/s; 16384 of split halves 59).  (Rotated by the softmax warps
// of the attention kernel, where a query tile arrives with nothing to hide behind, it took 4 to 7 us per piece.)
template <int D>
__host__ __device__ __forceinline__ int rotate_owners(const RopeFreq& f) {  // threads for a token's dims
  return D / 8 - (f.half ? f.n_pairs / 8 : 0);
}
template <int D>
__global__ void __launch_bounds__(256, 4) packed_rotate_kernel(const __grid_constant__ PackedArgs a,
                                                            const __grid_constant__ RopeFreq f, __nv_bfloat16* hi,
                                                            __nv_bfloat16* lo, int lo_dim, int heads_per) {
  asm volatile("griddepcontrol.launch_dependents;");  // the attention kernel starts, and waits where it reads these
  constexpr int kChunks = D / 8;
  const int groups = a.n_h / heads_per, owners = rotate_owners<D>(f);
  const long long i = blockIdx.x * 256LL + threadIdx.x, tg = i / owners;
  const int t = static_cast<int>(tg / groups), h0 = static_cast<int>(tg - static_cast<long long>(t) * groups) * heads_per;
  if (t >= a.T) return;
  int c = static_cast<int>(i - tg * owners);
  if (f.half && c * 8 >= a.rope_offset + f.n_pairs) c += f.n_pairs / 8;  // chunks with a partner before them are its thread's
  const int rel = c * 8 - a.rope_offset;
  const bool in = rel >= 0 && rel < 2 * f.n_pairs;
  float sn[8], cs[8];
  if (in) {
    int pos;
    if (a.positions != nullptr) {
      pos = a.positions[t];
    } else {
      int b = 0, e = a.B - 1;  // the last request that starts at or before the row
      while (b < e) {
        const int mid = (b + e + 1) >> 1;
        if (packed_first(a, mid) <= t) b = mid;
        else e = mid - 1;
      }
      const PackedRequest r = packed_request(a, b);
      pos = r.base + t - r.first;
    }
    const int p0 = f.half ? rel : rel / 2, n = f.half ? 8 : 4;
    // (the hardware sines are off by 2^-21: less than the second part's own rounding)
    with_angles<true, true>(max(pos, 0), [&](auto angle) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) angle(f.hi[p0 + e], f.lo[p0 + e], &sn[e], &cs[e]);
    });
  }
  const long long row = static_cast<long long>(t) * a.n_h + h0;
  const uint4* const q = static_cast<const uint4*>(a.q) + row * kChunks + c;
  uint4* const o = reinterpret_cast<uint4*>(hi) + row * kChunks + c;
  uint4* const s = reinterpret_cast<uint4*>(lo) + row * (kLoDims / 8);
  const int lc = c - lo_dim / 8, partner = f.n_pairs / 8;
  const auto put = [&](int h, int at, const float* x) {  // chunk c + at
    const bool two = static_cast<unsigned>(lc + at) < static_cast<unsigned>(kLoDims / 8);
    // With a second part the first is what bf16 cuts off the next number nearer to 0, so that what is left is never 0 and of
    // the query's sign: an infinite key gives both products the same infinity.  (A value that bf16 holds exactly is a step
    // of bf16 less and that step.)  0 is 0 twice, and no finite key adds anything to it.  Infinities come as the largest
    // finite value and an infinity, NaN as NaN.
    const uint4 y = f32_to_bf16x8(x);
    uint32_t v[8], cut[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(x[e]) - (x[e] != 0.f ? 1u : 0u);
#pragma unroll
    for (int e = 0; e < 4; ++e) cut[e] = __byte_perm(v[2 * e], v[2 * e + 1], 0x7632);
    o[h * kChunks + at] = two ? make_uint4(cut[0], cut[1], cut[2], cut[3]) : y;
    if (two) {
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = x[e] - __uint_as_float(v[e] & 0xffff0000u);
      s[h * (kLoDims / 8) + lc + at] = f32_to_bf16x8(z);
    }
  };
  constexpr int kFlight = 4;  // heads whose loads are in flight together
  if (in && f.half) {
#pragma unroll 1
    for (int h = 0; h < heads_per; ++h) {  // (two at a time: the registers spill)
      float x[8], y[8];
      bf16x8_to_f32(__ldg(q + h * kChunks), x);
      bf16x8_to_f32(__ldg(q + h * kChunks + partner), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) rotate_pair(x[e], y[e], sn[e], cs[e]);
      put(h, 0, x);
      put(h, partner, y);
    }
  } else {
    for (int h0 = 0; h0 < heads_per; h0 += kFlight) {
      uint4 a0[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (h0 + k < heads_per) a0[k] = __ldg(q + (h0 + k) * kChunks);
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (h0 + k < heads_per) {
          float x[8];
          bf16x8_to_f32(a0[k], x);
          if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e) rotate_pair(x[2 * e], x[2 * e + 1], sn[e], cs[e]);
          }
          put(h0 + k, 0, x);
        }
    }
  }
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

// This thread's row of a tile's scores become its weights P (see prefill_tc.cu): p = 2^(s * scale*log2e - m), and m
// moves only when the row maximum grew by more than the threshold.  So a tile is taken with the m that is there, in one
// pass that finds the maximum beside the weights; P is stored behind the pass, where no row asks for another m, else
// (false) nothing is: prepare_row then moves m, and the tile is taken again (a copy of the code out of line: it is rare).
// Masked tiles go through prepare_row before.
// LO: the weights of the last 64 keys come as the sum of two bf16 values, the second ones in columns 64 on.
// (Short as it can be: all code that runs side by side in an SM has to fit its instruction cache, see the MMA issuer;
// and no more registers than there are: spilled ones are more than the L1 beside 226 KB of shared memory holds.)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16x2_down(float lo, float hi) {  // toward 0
  uint32_t d;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool LO>
__device__ __forceinline__ bool softmax_row(uint32_t s_addr, float scale_log2, float m_run, float& l_run) {
  uint32_t sr[2][16], pr[64], rest[LO ? 32 : 1];
  tmem_ld16(s_addr, sr[0]);
  const float m_ref = m_run == -INFINITY ? 0.f : m_run;  // every score so far is -inf: weights 0
  const float2 sl2 = make_float2(scale_log2, scale_log2), nm2 = make_float2(-m_ref, -m_ref);
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int q = 0; q < BN / 16; ++q) {
    tmem_wait_ld();
    if (q + 1 < BN / 16) tmem_ld16(s_addr + 16 * (q + 1), sr[(q + 1) & 1]);
    const uint32_t* const s = sr[q & 1];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 y = make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
      mx[c & 1] = fmax3(mx[c & 1], y.x, y.y);
      const float2 x = __ffma2_rn(y, sl2, nm2);
      const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      acc[c & 1] = __fadd2_rn(acc[c & 1], pp);
      if (LO && q >= 4) {
        // the first part cut off, and the second 2^-20 of the weight too large, never 0 or of the other sign: an infinite
        // value then gives both products the same infinity
        pr[8 * q + c] = pack_bf16x2_down(pp.x, pp.y);
        const float2 z = __ffma2_rn(pp, make_float2(1.f + 0x1p-20f, 1.f + 0x1p-20f),
                                    make_float2(__uint_as_float((pr[8 * q + c] << 16) | 0x80000000u),
                                                __uint_as_float((pr[8 * q + c] & 0xffff0000u) | 0x80000000u)));
        rest[8 * (q - 4) + c] = pack_bf16x2(z.x, z.y);
      } else {
        pr[8 * q + c] = pack_bf16x2(pp.x, pp.y);
      }
    }
  }
  const float top = fmaxf(mx[0], mx[1]) * scale_log2;
  if (__any_sync(0xffffffffu, top > m_run + kRescaleThreshold)) return false;
#pragma unroll
  for (int c = 0; c < 64; c += 16) tmem_st16(s_addr + c, pr + c);
  if constexpr (LO) {
    tmem_st16(s_addr + 64, rest);
    tmem_st16(s_addr + 80, rest + 16);
  }
  acc[0] = __fadd2_rn(acc[0], acc[1]);
  l_run += acc[0].x + acc[0].y;
  return true;
}

// The maximum of a row's first 32 scores: a piece's first m, mostly within the threshold of the whole tile's maximum.
__device__ __noinline__ float max_of_some(uint32_t s_addr) {
  uint32_t x[32];
  tmem_ld32(s_addr, x);
  tmem_wait_ld();
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 32; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// Scores that the row does not see become -inf where they are, and m moves to the tile's maximum if that is higher by more
// than the threshold, with l and O.
template <int D>
__device__ __noinline__ float2 prepare_row(uint32_t s_addr, uint32_t o_addr, bool masked, uint4 mask, bool rescale,
                                         float scale_log2, float m_run, float l_run) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    uint32_t x[32];
    tmem_ld32(s_addr + 32 * h, x);
    tmem_wait_ld();
    if (masked) {
      const uint32_t m = mask.x;
      mask = make_uint4(mask.y, mask.z, mask.w, 0u);
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!((m >> c) & 1u)) x[c] = 0xff800000u;
      tmem_st32(s_addr + 32 * h, x);
    }
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 32; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
    mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
  }
  mx *= scale_log2;
  const bool need = mx > m_run + kRescaleThreshold;
  float alpha = 1.f;
  if (need) {
    if (m_run != -INFINITY) alpha = fast_exp2(m_run - mx);
    l_run *= alpha;
    m_run = mx;
  }
  if (__any_sync(0xffffffffu, need && rescale)) rescale_o<D>(o_addr, alpha);
  tmem_wait_st();
  return make_float2(m_run, l_run);
}

template <bool LO>
__device__ __noinline__ float softmax_row_again(uint32_t s_addr, float scale_log2, float m_run, float l_run) {
  softmax_row<LO>(s_addr, scale_log2, m_run, l_run);
  return l_run;
}

// The bits of what a row of worker w sees in the tile from key0 on; a row that is no query sees nothing.  (Out of line, and
// so with the kernel's arguments by value: through a reference they are read like global memory.)
__device__ __noinline__ uint4 row_mask(const int* visible, int words, int tile_toks, const Piece* u, int w, int my_tok, int key0) {
  uint32_t m[4];
  const int tok = (u->kind == kPair && w ? tile_toks : 0) + my_tok;
  const bool real = my_tok < tile_toks && tok < u->ntok && u->place0 + tok >= 0;
  if (visible == nullptr || !real) {
    seen_below(real ? u->place0 + tok + 1 : 0, key0, m);
  } else {
    uint32_t bits[4];
    const int* const row = visible + static_cast<long long>(u->row0 + tok) * words;
#pragma unroll
    for (int i = 0; i < 4; ++i) bits[i] = i < words ? static_cast<uint32_t>(row[i]) : 0u;
    seen_tree(bits, u->base, u->klim, key0, m);
  }
  return make_uint4(m[0], m[1], m[2], m[3]);
}

// The values that are not finite in care tiles, of dims [c0, c1), added to what has been stored of a row that sees them, times
// their weights: the infinity, or NaN where the key has no weight, as the MMA gives in the other tiles.  The weights are
// gone by then: the score is summed once more from the query that the MMA had (row q_row of it), and m is the row's
// maximum.
template <int D, bool LO>
__device__ __noinline__ void add_bad(const PackedArgs& a, const PackedTcPlan& pl, const Piece& u, int w, int my_tok, long long q_row,
                                   float m_run, int c0, int c1, __nv_bfloat16* out, float* partial) {
  if (LO) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rotated queries are there (long since)
  const float* const ws = static_cast<const float*>(a.workspace);
  const __nv_bfloat16* const q = (LO ? reinterpret_cast<const __nv_bfloat16*>(ws + pl.q) : static_cast<const __nv_bfloat16*>(a.q)) + q_row * D;
  const __nv_bfloat16* const rest = reinterpret_cast<const __nv_bfloat16*>(ws + pl.lo) + q_row * kLoDims;
  const float m_ref = m_run == -INFINITY ? 0.f : m_run;
  for (int i = 0; i < kCare; ++i) {
    const int key0 = (u.care_t + i) * BN;
    if (u.care_t + i >= u.t_end) break;
    if (u.care_t + i < u.t) continue;
    const uint4 seen = row_mask(a.visible, a.words, pl.tile_toks, &u, w, my_tok, key0);
    const uint32_t m[4] = {seen.x, seen.y, seen.z, seen.w};
    for (int j = 0; j < 4; ++j) {
      for (uint32_t left = u.bad[i][j] & m[j]; left; left &= left - 1) {
        const int key = key0 + 32 * j + __ffs(left) - 1;
        const int page = a.block_table[static_cast<long long>(u.b) * a.max_blocks + (key >> a.page_shift)];
        const long long slot = (static_cast<long long>(page) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        const __nv_bfloat16* const v = static_cast<const __nv_bfloat16*>(a.v_pages) + slot * a.v_token_stride + u.g * a.D_v;
        const __nv_bfloat16* const k = static_cast<const __nv_bfloat16*>(a.k_pages) + (slot * a.n_kv + u.g) * D;
        float score = 0.f;
#pragma unroll 1
        for (int d = 0; d < D; ++d) score = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), score);
#pragma unroll 1
        for (int d = 0; LO && d < kLoDims; ++d)
          score = fmaf(__bfloat162float(rest[d]), __bfloat162float(k[pl.lo_first * 16 + d]), score);
        const float weight = __bfloat162float(__float2bfloat16_rn(fast_exp2(fmaf(score, a.scale_log2, -m_ref))));
        for (int d = c0; d < c1; ++d) {
          float x = __bfloat162float(v[d]);
          if (fabsf(x) < INFINITY) continue;
          x *= weight;
          if (partial != nullptr) partial[d] += x;
          else out[d] = __float2bfloat16_rn(__bfloat162float(out[d]) + x);
        }
      }
    }
  }
}

// Columns [c0, c1) of the rows' O times f0 (both: and the one D columns on times f1), as bf16 to the output (whole) or as
// fp32 to a partial; `to`: where this lane's row begins, `row` its number there (-1: not a query), step bytes per row.
// zero: zeros.  Four lanes exchange 16-byte pieces of their rows, so that a store instruction writes 64 bytes of each of
// eight rows: with a row per lane it made 32 lines, and the load/store unit took 550 cycles for 16 columns.  Out of line:
// beside the softmax it had registers of that spilled.
template <int D>
__device__ __noinline__ void store_rows(uint32_t o_col, int c0, int c1, bool both, bool whole, bool zero, float f0, float f1, char* to,
                                      int row, int step) {
  const int lane = threadIdx.x & 31, lj = lane & 3;
  to += lj * 16;
  const auto put = [&](uint4* pc, int offset) {
    transpose_pieces(pc, lj);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int other = __shfl_sync(0xffffffffu, row, (lane & 28) + k);
      if (other >= 0) *reinterpret_cast<uint4*>(to + static_cast<long long>(other - (row >= 0 ? row : 0)) * step + offset) = pc[k];
    }
  };
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    float o[32];
    {
      uint32_t x[32];
      tmem_ld32(o_col + c, x);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(x[e]) * f0;
      if (both) {
        tmem_ld32(o_col + D + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(x[e]), f1, o[e]);
      }
    }
    if (zero) {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0.f;
    }
    uint4 pc[4];
    if (whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e) pc[e] = f32_to_bf16x8(o + 8 * e);
      put(pc, 0);
      to += 64;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* const v = o + 16 * h + 4 * e;
          pc[e] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        }
        put(pc, 64 * h);
      }
      to += 128;
    }
  }
}

template <int D, bool LO>
__global__ void __launch_bounds__(kThreads, 1)
    packed_tc_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ PackedTcPlan pl,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_lo,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, LO>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // no room is left for aligning it here
    if (threadIdx.x == 0) atomicOr(a.status, STATUS_LAYOUT);
    if (threadIdx.x < 2)  // nothing to join
      (reinterpret_cast<Record*>(static_cast<float*>(a.workspace) + pl.rec) + 2 * blockIdx.x)[threadIdx.x] = Record{0, 0, 0, 0, 0, 0, 0, 0};
    return;
  }
  Bars<C>* bars = reinterpret_cast<Bars<C>*>(smem + C::kBarOff);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
      mbar_init(&bars->q_empty[w], 1);
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->p_full[w], 128);
      mbar_init(&bars->o_done[w], 1);
      mbar_init(&bars->o_empty[w], 128);
    }
    mbar_init(&bars->x_full, 128);
    mbar_init(&bars->x_back, 128);
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
  // part k of n starts at the k / n-th of the line (n parts of equal length up to rounding; no divisions here)
  const auto cut = [&](uint32_t k) {
    return k == gridDim.x ? total : static_cast<long long>(__umul64hi(static_cast<unsigned long long>(total), k * pl.nth));
  };
  const long long part_lo = cut(blockIdx.x), part_hi = cut(blockIdx.x + 1);
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
      if (LO && is_v) {  // the rotated queries come from the kernel before
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("fence.proxy.async.global;" ::: "memory");
      }
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
              mbar_arrive_expect_tx(&bars->q_full[w], static_cast<uint32_t>(pl.tile_toks * G) * 128u * (C::kBlocks + LO));
              for (int d = 0; d < C::kBlocks; ++d)
                tma_load_4d(smem + C::kQOff + w * C::kTileBytes + d * C::kBlockBytes, &tm_q, &bars->q_full[w], d * 64, 0, g, row);
              if (LO) tma_load_4d(smem + C::kLoOff + w * C::kLoBytes, &tm_lo, &bars->q_full[w], 0, 0, g, row);
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
      if (elect_one()) {
        const uint32_t q_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024));
        const uint32_t k_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024));
        const uint32_t v_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kVOff), C::kBlockBytes, 1024));
        const uint32_t lo_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kLoOff), 16, 1024));
        Ring kr, vr;
        uint32_t q_ph = 0, p_ph = 0, o_ph = 0, fix_ph = 0;  // parities, bits per worker (fix_ph: per V stage)
        // Q K^T: the steps of Q's first part, those of its second part.  Loops, a few at a time: all code that runs side by
        // side in an SM has to fit its instruction cache (with 96 MMAs written out, a tile's softmax took 2350 cycles in
        // the mean and 1600 at best).
        auto qk_hi = [&](uint32_t w) {
          uint32_t a0 = q_desc0 + ((w * C::kTileBytes) >> 4), b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll 1
          for (int blk = 0; blk < C::kBlocks; ++blk) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_lo(tmem + w * 128u, a0 + kk * 2, b0 + kk * 2, C::kIdescQK, kk > 0 || blk > 0 ? 1u : 0u);
            a0 += C::kBlockBytes >> 4;
            b0 += C::kBlockBytes >> 4;
          }
        };
        auto qk_lo = [&](uint32_t w) {
          if constexpr (LO) {
            const uint32_t a0 = lo_desc0 + ((w * C::kLoBytes) >> 4);
            uint32_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll 1
            for (int s = 0; s < C::kLoSteps; ++s) {
              const int kk = pl.lo_first + s;
              mma_ss_lo(tmem + w * 128u, a0 + s * 2, b0 + (((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4), C::kIdescQK, 1u);
            }
          }
        };
        auto issue_qk = [&](uint32_t w) {
          qk_hi(w);
          qk_lo(w);
          mma_commit(&bars->s_full[w]);
        };
        // P V: P in columns 8 kk of the worker's S, its second part in columns 64 on
        auto issue_pv = [&](uint32_t w, bool first) {
          const uint32_t b0 = v_desc0 + ((vr.st * C::kTileBytes) >> 4), p0 = tmem + w * 128u, o0 = tmem + C::kOCol + w * D;
#pragma unroll 1
          for (int i = 0; i < BN / 16 + C::kPLoSteps; i += 4) {
            const uint32_t a0 = p0 + i * 8, v0 = b0 + ((i < BN / 16 ? i : i - 4) * 128);  // steps of 16 keys x 128 bytes
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_lo(o0, a0 + kk * 8, v0 + kk * 128, C::kIdescPV, (!first || i > 0 || kk > 0) ? 1u : 0u);
          }
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
          const bool there = lane_wait(&bars->q_full[w], (q_ph >> w) & 1u, wc);
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
        // A turn inside a pair piece (see below); more: another one follows.
        auto turn = [&](bool more) -> bool {
          if (!wait_p(0)) return false;
          tc_fence_after();
          issue_pv(0, false);
          issue_qk(0);
          if (!wait_p(1)) return false;
          tc_fence_after();
          issue_pv(1, false);
          v_done();
          qk_hi(1);
          Ring kn = kr;
          kn.next(C::kKStages);
          if (more && !(wait_v(false) && lane_wait(&bars->k_full[kn.st], kn.ph, wc))) return false;
          qk_lo(1);
          mma_commit(&bars->s_full[1]);
          mma_commit(&bars->k_empty[kr.st]);
          kr = kn;
          return true;
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
                for (; ok && v < ve; ++v) ok = turn(v + 1 < ve);
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
        // KV head off / own: the quotient of floats is off by one at most
        int g = min(static_cast<int>(static_cast<float>(off) / static_cast<float>(own)), a.n_kv - 1);
        while (g > 0 && g * own > off) --g;
        while (g + 1 < a.n_kv && (g + 1) * own <= off) ++g;
        walk.g = g;
        off -= g * own;
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
        walk.t = tile_at(off, s.lead(lo), s.shift(lo), tiles_of(s.seen(lo, min(2 * s.tt, s.r.rows - lo * 2 * s.tt))));
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
          Piece* const u = &bars->piece[e];
          const int kind = next_piece(a, pl, walk, u, lane);
          last = kind == kNone;
          if (lane == 0) {
            if (!last && u->slot >= 0) {
              rec[u->slot] = Record{u->kind, u->g, u->row0, u->ntok, u->t, u->t_end, u->kt, 0};
              recs |= 1u << u->slot;
            }
            mbar_arrive(&bars->piece_full[e]);
          }
          __syncwarp();
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
    uint32_t s_ph = 0, o_ph = 0, x_ph = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!row_wait(&bars->piece_full[n % kQueue], (n / kQueue) & 1u, wc)) break;
      const Piece* const u = &bars->piece[n % kQueue];
      const int kind = u->kind;
      if (kind == kNone) break;
      const Share sh(*u, w);
      // (what a row sees is looked up again for each care tile, and a row's place in the output for the epilogue: kept in
      // registers beside the scores, it is spilled)
      float m_run = -INFINITY, l_run = 0.f;
      {
        // beside the scores and second parts there are no registers for these: they are read again where they are needed
        constexpr bool kReload = C::kPLoSteps > 0;
        const int care_t = u->care_t, first_t = sh.first;
        const auto care = [&] { return kReload ? u->care_t : care_t; };
        const auto first = [&] { return kReload ? Share(*u, w).first : first_t; };
        int left = sh.n;
        for (int t = sh.first; left > 0; --left, t += kReload ? (kind == kPair ? 1 : 2) : sh.step) {
          if (!row_wait(&bars->s_full[w], s_ph, wc)) { ok = false; break; }
          s_ph ^= 1u;
          tc_fence_after();
          if (t >= care()) {
            const uint4 mask = row_mask(a.visible, a.words, pl.tile_toks, u, w, my_tok, t * BN);
            const float2 ml = prepare_row<D>(s_addr, o_addr, true, mask, t != first(), a.scale_log2, m_run, l_run);
            m_run = ml.x;
            l_run = ml.y;
          } else if (t == first()) {
            m_run = max_of_some(s_addr) * a.scale_log2;
          }
          if (!softmax_row<C::kPLoSteps != 0>(s_addr, a.scale_log2, m_run, l_run)) {
            const float2 ml = prepare_row<D>(s_addr, o_addr, false, make_uint4(0u, 0u, 0u, 0u), t != first(),
                                             a.scale_log2, m_run, l_run);
            m_run = ml.x;
            l_run = softmax_row_again<C::kPLoSteps != 0>(s_addr, a.scale_log2, ml.x, ml.y);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[w]);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      // epilogue: the rows of the output, or the piece's normalised partial and its log-sum-exp
      const int tok = (kind == kPair && w ? pl.tile_toks : 0) + my_tok;
      const bool real = my_tok < pl.tile_toks && tok < u->ntok;  // this row is a query
      const int position = real && a.positions != nullptr ? a.positions[u->row0 + tok] : 0;  // there by the time O is
      if (sh.n > 0) {
        if (!row_wait(&bars->o_done[w], o_ph, wc)) break;
        o_ph ^= 1u;
      }
      // A single piece of more than one tile has a part of each row in both workers: worker 0 joins the sums, and each
      // worker writes half of the dims.
      const bool both = kind == kSingle && Share(*u, 1).n > 0;
      float2* const ml = reinterpret_cast<float2*>(smem + C::kMlOff) + r;
      float f0 = l_run > 0.f ? 1.f / l_run : l_run, f1 = 0.f;  // factors of O of this worker (both: of worker 0), and of worker 1
      if (both) {
        if (w == 1) {
          *ml = make_float2(m_run, l_run);
          tc_fence_before();
          mbar_arrive(&bars->x_full);
          if (!row_wait(&bars->x_back, x_ph, wc)) break;
          f0 = ml->x;
          f1 = ml->y;
        } else {
          if (!row_wait(&bars->x_full, x_ph, wc)) break;
          const float2 o = *ml;
          const float m = fmaxf(m_run, o.x), m_ref = m == -INFINITY ? 0.f : m;
          f0 = fast_exp2(m_run - m_ref);
          f1 = fast_exp2(o.x - m_ref);
          l_run = l_run * f0 + o.y * f1;
          m_run = m;
          const float inv = l_run > 0.f ? 1.f / l_run : l_run;
          f0 *= inv;
          f1 *= inv;
          *ml = make_float2(f0, f1);
          reinterpret_cast<float*>(smem + C::kMaxOff)[r] = m;
          tc_fence_before();
          mbar_arrive(&bars->x_back);
        }
      }
      if (kind == kPair || w == 0 || both) {
        if (!row_wait(&bars->care_done[n % kQueue], (n / kQueue) & 1u, wc)) break;
        const bool whole = u->slot < 0;
        const bool lead = !both || w == 0;  // writes the log-sum-exp
        const bool dead = !real || u->place0 + tok < 0 || position < 0;
        const bool none = dead || (f0 == 0.f && f1 == 0.f && l_run == 0.f);  // no key with a weight; NaN is one
        float* const ws = static_cast<float*>(a.workspace);
        const long long slot_row = (2 * static_cast<long long>(blockIdx.x) + (whole ? 0 : u->slot)) * pl.slot_rows + (kind == kPair ? w * BM : 0) + r;
        const long long out_row = static_cast<long long>(u->row0 + tok) * a.n_h + u->g * G + (r - my_tok * G);
        const float lse2 = none ? -INFINITY : m_run + log2f(l_run);
        if (real && lead) {
          if (!whole) ws[pl.l + slot_row] = lse2;
          else if (a.lse != nullptr) a.lse[out_row] = lse2 * 0.69314718055994530942f;
        }
        if (sh.n > 0) {
          tc_fence_after();
          const int c0 = both && w == 1 ? D / 2 : 0, c1 = both && w == 0 ? D / 2 : D;
          // A row without any weight is 0; a piece of it is 0 or, beside values that are not finite, NaN.
          const bool zero = whole ? none : dead;
          // rows that are no queries take the place of row 0 (they store nothing of their own)
          const long long at = whole ? (real ? out_row : 0) : slot_row;
          char* const to = whole ? static_cast<char*>(a.out) + at * (D * 2) : reinterpret_cast<char*>(ws + (real ? at : at - r) * D);
          store_rows<D>(tmem + lane_off + C::kOCol + (both || w == 0 ? 0 : D), c0, c1, both, whole, zero, f0, f1,
                        to + c0 * (whole ? 2 : 4), real ? (whole ? static_cast<int>(at) : r) : -1, whole ? D * 2 : D * 4);
          if (u->bad_any) {
            __syncwarp();  // the row has been stored by four lanes
            if (!zero)
              add_bad<D, LO>(a, pl, *u, w, my_tok, out_row, both && w == 1 ? reinterpret_cast<float*>(smem + C::kMaxOff)[r] : m_run,
                             c0, c1, whole ? static_cast<__nv_bfloat16*>(a.out) + at * D : nullptr,
                             whole ? nullptr : ws + slot_row * D);
          }
          tc_fence_before();
          if (!both) {
            mbar_arrive(&bars->o_empty[w]);
          } else if (w == 1) {
            mbar_arrive(&bars->x_done);
          } else {
            if (!row_wait(&bars->x_done, x_ph, wc)) break;
            mbar_arrive(&bars->o_empty[0]);
            mbar_arrive(&bars->o_empty[1]);
          }
        } else if (real) {  // a pair's first row tile behind its last key: a part that holds nothing
#pragma unroll 1
          for (int c = 0; c < D; c += 4) *reinterpret_cast<float4*>(ws + slot_row * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (both) x_ph ^= 1u;
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
constexpr int kJoinWarps = 8, kJoinPer = 1, kJoinFlight = 4, kJoinRows = 2 * kJoinWarps * kJoinPer;
constexpr int kMaxCtas = 160;  // the workspace is sized for this many (a GB300 has 152 SMs)

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 6)
    packed_tc_join_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ PackedTcPlan pl) {
  constexpr int kPer = D / 32;  // dims per lane
  __shared__ int slots[kMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* const ws = static_cast<const float*>(a.workspace);
  const Record* const rec = reinterpret_cast<const Record*>(ws + pl.rec);
  const int parts = (pl.slot_rows + kJoinRows - 1) / kJoinRows;
  const int c = blockIdx.x / parts, part = blockIdx.x - c * parts;
  const Record head = rec[2 * c + 1];
  // the pieces: this one, then first pieces up to the one that ends the segment (a CTA may hold none)
  int kt = 0, t_end = 0;
  if (c + 1 + lane < pl.ctas) {
    kt = rec[2 * (c + 1 + lane)].kt;
    t_end = rec[2 * (c + 1 + lane)].t_end;
  }
  const int G = a.n_h / a.n_kv;
  if (head.kt == 0 || part * kJoinRows >= (head.kind == kPair ? 2 * BM : min(BM, head.ntok * G))) return;
  if (threadIdx.x == 0) slots[0] = 2 * c + 1;
  int n = 1;
  for (int c0 = c + 1; c0 < pl.ctas; c0 += 32) {
    const int cc = c0 + lane;
    if (c0 > c + 1) {
      kt = cc < pl.ctas ? rec[2 * cc].kt : 0;
      t_end = cc < pl.ctas ? rec[2 * cc].t_end : 0;
    }
    const uint32_t end = __ballot_sync(0xffffffffu, kt > 0 && t_end == kt);
    const uint32_t upto = end ? (end & (0u - end)) * 2u - 1u : 0xffffffffu;  // lanes up to the first that ends it
    const uint32_t some = __ballot_sync(0xffffffffu, kt > 0) & upto;
    if (warp == 0 && ((some >> lane) & 1u)) slots[n + __popc(some & ((1u << lane) - 1u))] = 2 * cc;
    n += __popc(some);
    if (end) break;
  }
  __syncthreads();
  // kJoinPer rows per warp, all loads of kJoinFlight pieces in flight, with a running maximum of their log-sum-exps
#pragma unroll 1
  for (int pass = 0; pass < kJoinRows; pass += kJoinWarps * kJoinPer) {
    int rr[kJoinPer], at[kJoinPer];
    float M[kJoinPer], den[kJoinPer], acc[kJoinPer][kPer];
#pragma unroll
    for (int k = 0; k < kJoinPer; ++k) {
      rr[k] = part * kJoinRows + pass + warp * kJoinPer + k;
      const int r = rr[k] & (BM - 1), w = rr[k] / BM, tk = r / G, tok = (w ? pl.tile_toks : 0) + tk;
      at[k] = tk < pl.tile_toks && tok < head.ntok && (!w || head.kind == kPair)
                  ? (head.row0 + tok) * a.n_h + head.g * G + (r - tk * G) : -1;
      M[k] = -INFINITY;
      den[k] = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[k][e] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < n; j += kJoinFlight) {
      float l[kJoinFlight][kJoinPer], v[kJoinFlight][kJoinPer][kPer];
#pragma unroll
      for (int q = 0; q < kJoinFlight; ++q)
#pragma unroll
        for (int k = 0; k < kJoinPer; ++k) {
          l[q][k] = -INFINITY;
#pragma unroll
          for (int e = 0; e < kPer; ++e) v[q][k][e] = 0.f;
          if (j + q < n && at[k] >= 0) {
            const long long row = static_cast<long long>(slots[j + q]) * pl.slot_rows + rr[k];
            l[q][k] = ws[pl.l + row];
            const float* const p = ws + row * D + lane * kPer;
            if constexpr (kPer == 4) {
              const float4 y = *reinterpret_cast<const float4*>(p);
              v[q][k][0] = y.x; v[q][k][1] = y.y; v[q][k][2] = y.z; v[q][k][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(p);
              v[q][k][0] = y.x; v[q][k][1] = y.y;
            }
          }
        }
#pragma unroll
      for (int k = 0; k < kJoinPer; ++k) {
        float m = M[k];
#pragma unroll
        for (int q = 0; q < kJoinFlight; ++q) m = fmaxf(m, l[q][k]);
        const float m_ref = m == -INFINITY ? 0.f : m;
        const float x = exp2f(M[k] - m_ref);
        M[k] = m;
        den[k] *= x;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[k][e] *= x;
#pragma unroll
        for (int q = 0; q < kJoinFlight; ++q) {
          const float y = exp2f(l[q][k] - m_ref);  // a part without a weight holds 0, or NaN
          den[k] += y;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[k][e] = fmaf(y, v[q][k][e], acc[k][e]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kJoinPer; ++k) {
      if (at[k] < 0) continue;
      const float inv = 1.f / den[k];
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[k][e] = den[k] == 0.f ? 0.f : acc[k][e] * inv;
      uint32_t* const out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<long long>(at[k]) * D + lane * kPer);
      if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(acc[k][0], acc[k][1]), pack_bf16x2(acc[k][2], acc[k][3]));
      else
        out[0] = pack_bf16x2(acc[k][0], acc[k][1]);
      if (lane == 0 && a.lse != nullptr)
        a.lse[at[k]] = den[k] == 0.f ? -INFINITY : (M[k] + log2f(den[k])) * 0.69314718055994530942f;
    }
  }
}

PackedTcPlan make_plan(const PackedArgs& a, int ctas, int max_ctas, bool rotate) {
  PackedTcPlan p{};
  const int G = a.n_h / a.n_kv;
  p.ctas = ctas;
  p.nth = ctas > 1 ? ~0ull / ctas : 0;
  p.tile_toks = BM / G;
  p.slot_rows = a.T <= p.tile_toks ? a.T * G : 2 * BM;
  const int rest = (a.D_qk - kLoDims) / 16;
  p.lo_first = a.rope_offset / 16 < rest ? a.rope_offset / 16 : rest;
  p.l = 2LL * max_ctas * p.slot_rows * a.D_v;
  p.rec = (p.l + 2LL * max_ctas * p.slot_rows + 3) & ~3LL;
  p.q = (p.rec + 2LL * max_ctas * static_cast<long long>(sizeof(Record) / 4) + 31) & ~31LL;
  const long long rows = rotate ? static_cast<long long>(a.T) * a.n_h : 0;
  p.lo = p.q + rows * a.D_qk / 2;
  p.end = p.lo + rows * kLoDims / 2;
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
    // few tokens: fewer heads per thread, but for four or more the angles are worth sharing (one head each: 36 us for
    // 1888 tokens of 32, instead of 12)
    int heads = a.n_h;
    const int owners = rotate_owners<D>(rope);
    while (heads % 2 == 0 && heads > 4 && static_cast<long long>(a.T) * (a.n_h / heads) * owners < 152LL * 1024) heads /= 2;
    const long long items = static_cast<long long>(a.T) * (a.n_h / heads) * owners;
    float* const ws = static_cast<float*>(a.workspace);
    packed_rotate_kernel<D><<<static_cast<unsigned>((items + 255) / 256), 256, 0, st>>>(
        a, rope, reinterpret_cast<__nv_bfloat16*>(ws + pl.q), reinterpret_cast<__nv_bfloat16*>(ws + pl.lo),
        pl.lo_first * 16, heads);
    *launches += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_early(packed_tc_kernel<D, LO>, pl.ctas, kThreads, smem_bytes<Cfg<D, LO>>(), st, LO, a, pl, maps[0], maps[1],
                   maps[2], maps[3]);
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
  return static_cast<size_t>(make_plan(a, kMaxCtas, kMaxCtas, true).end) * sizeof(float);
}

cudaError_t launch_packed_tc(const PackedArgs& a, const RopeFreq& rope, int num_sms, cudaStream_t st, int* launches) {
  const bool rotate = rope.n_pairs > 0;
  int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  // no more CTAs than twice the tiles that the call can have (fewer would have to share)
  const long long segments = static_cast<long long>(a.T) * (a.n_h / a.n_kv) / (2 * BM - 2 * (a.n_h / a.n_kv) + 2) + a.B;
  const long long most = 2 * segments * a.n_kv * (((static_cast<long long>(a.max_blocks) << a.page_shift) + BN - 1) / BN);
  if (most < ctas) ctas = static_cast<int>(most);
  const PackedTcPlan pl = make_plan(a, ctas, kMaxCtas, rotate);
  // query rows by (dim, head of the group, KV head, row), a row tile per box; K and V by (dim, KV head, row in
  // page, page), a page or a part of it per box
  const unsigned long long hs = static_cast<unsigned long long>(a.D_qk) * 2, page = 1ull << a.page_shift;
  const unsigned long long ks = hs * a.n_kv, vs = static_cast<unsigned long long>(a.v_token_stride) * 2;
  const int G = a.n_h / a.n_kv, rows = static_cast<int>(page);
  CUtensorMap maps[4];
  float* const ws = static_cast<float*>(a.workspace);
  const void* q = rotate ? ws + pl.q : a.q;
  const bool wide = a.D_qk == 128;
  if (!make_map_box(&maps[0], q, a.D_qk, G, a.n_kv, a.T, hs, hs * G, hs * a.n_h, G, 1, pl.tile_toks, wide) ||
      !make_map_box(&maps[2], a.k_pages, a.D_qk, a.n_kv, rows, a.n_pages, hs, ks, ks * page, 1, rows < 128 ? rows : 128, 1, wide) ||
      !make_map_box(&maps[3], a.v_pages, a.D_v, a.n_kv, rows, a.n_pages, hs, vs, vs * page, 1, rows < 128 ? rows : 128, 1, wide))
    return cudaErrorInvalidValue;
  maps[1] = maps[0];
  const unsigned long long ls = kLoDims * 2;
  if (rotate && !make_map_box(&maps[1], ws + pl.lo, kLoDims, G, a.n_kv, a.T, ls, ls * G, ls * a.n_h, G, 1, pl.tile_toks, false))
    return cudaErrorInvalidValue;
  if (a.D_qk == 64)
    return rotate ? launch<64, true>(a, rope, maps, pl, st, launches) : launch<64, false>(a, rope, maps, pl, st, launches);
  return rotate ? launch<128, true>(a, rope, maps, pl, st, launches) : launch<128, false>(a, rope, maps, pl, st, launches);
}

}  // namespace attn
