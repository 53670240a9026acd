// decode_paged_tc.cu - single-token decode over a paged KV cache on the tensor cores
// (bf16, D_qk = D_v = 64 or 128), alone or behind a prefix that the batch shares.
//
// Every piece of the work is one product of up to 128 query rows with the keys of
// one KV head in tiles of 128: S = Q K^T, an online softmax over the rows, O += P V
// ("Transformer架构完全深度解析" §13).  The same code serves
//   own     the G = n_h / n_kv rows of one request against its own keys
//           [P, L) (P = prefix_len, 0 without a prefix), and
//   prefix  up to 128 of the B * G rows of a KV head against the P shared keys,
//           read once for all of them; with more than 128 rows two row tiles
//           share each K/V tile (a pair).
// A request reads 4 D bytes per key and KV head and does 4 D G flop: HBM-bound.
// The prefix does B G flop per byte: HBM-bound up to ~290 rows, then bound by the
// tensor pipe.  An MMA of 128 rows costs the same however few of them are real, and
// with 1024 pipe cycles per 64 KB tile (D = 128) against ~2800 cycles for which an SM
// waits for those bytes at HBM speed, padding a request's rows to 128 costs nothing.
// Pieces of at most 64 rows use the padding: each row comes with a second one, for what
// rounding to bf16 left of its rotated query and then of its weights, so that only the
// result is rounded (in 64 bits: error 0.0017 of the largest output, 0.0029 with both
// rounded; at 59 requests of 4096 to 16384 keys the same time).  Rows of larger pieces are
// a TMEM lane each, and rounded.
//
// Work split.  The pair tiles lie on one line, KV head by KV head, and the single ones on
// another: prefix tiles of an odd last row tile, then request after request, KV head
// fastest.  A tile is a few points long and each segment is led by kPieceCost points for
// what starting it costs; the first line is cut into equal parts, one per CTA (one
// persistent CTA per SM), the second into twice as many, one per worker (a CTA has two).
// A CTA does its pair tiles, then its workers their single ones.  (Cut as one line, so
// that some CTAs got pairs and others single tiles, the shares hung on how well the costs
// of the two were guessed: of 256 requests behind 16384 shared tokens the first CTA ended
// after 80 us and the last after 137.)  Cuts fall anywhere, also inside a request: each
// (worker, segment) piece writes one normalised partial and its log-sum-exp, and the
// combine kernel merges the pieces of a row.  So the SMs finish together whatever the
// lengths are, without a counter in memory, and partials are few.
// Where a piece's partial goes needs no table either: walking the line, each step to
// the next piece raises the worker's index or the segment's, so their sum numbers the
// pieces.
//
// A CTA (384 threads): warp 3 walks the CTA's part of the line (it sums the requests'
// points at its start; CTA 0's leaves the sums for the combine kernel) and hands the
// pieces to the other roles through two small queues in shared memory, a few pieces
// ahead; it also clears value rows behind a segment's last key, which may hold anything.
// Warps 0 and 2 load the query rows, K and V tiles by TMA - K and V one box per page and
// 64 dims (a page is part of a tile, the tile, or twice the tile), the lanes of the warp
// issuing one box each; warp 1 issues the MMAs; warps 4-7 and 8-11 are the two workers'
// softmax.  The workers run separate pieces (their tiles alternate in the K and V rings),
// so that one's MMAs and loads fill the other's softmax and piece ends; on pair tiles
// they hold the two row tiles and share each K/V tile.
// A role's code is one small loop, the same for pair and single tiles: with the walk, the
// query rotation and the two cases written out in each role (120 KB of instructions) a
// one-tile piece took 10 us, the instruction fetches of the SMs saturating their shared
// caches.  For the same reason the queries are rotated before, by a kernel of their own
// that this one overlaps with its start (programmatic launch).
// Measured (32 query heads over 8 KV heads, D = 128): 59 requests of 4096 to 8192 keys, 1.49 GB in 224 to 232 us
// (0.95 to 0.99 of the card's copy rate), whether pages hold 16 tokens or 128, with 64-dim heads 137 us (0.81);
// 64 requests behind 32768 shared tokens 56.5 us (0.54 of the copy rate), 256 behind 16384 100 us (690 TFLOP/s).
// TMEM: S/P of the workers in columns [0, 128) and [128, 256), O behind them.
#include <float.h>
#include <math.h>

#include <atomic>

#include "api.h"

namespace attn {

// The cut of a call that does not depend on the lengths, and the layout of its workspace.
struct PagedTcPlan {
  int ctas;
  int row_reqs;      // requests per row tile: 128 / G
  int rows;          // rows per row tile: row_reqs * G
  int n_pairs;       // pairs of row tiles of a KV head's prefix rows
  int odd;           // 1: one more row tile
  int prefix_tiles;  // key tiles of the prefix
  // pieces of few rows have them in groups of up to 8 (kGroups):
  int own_groups;     // groups of an own piece, 0: its rows lie one after the other
  int prefix_groups;  // of a prefix piece
  int own_group, prefix_group;  // rows per group
  int group_reqs;     // requests per group of prefix rows: 8 / G, at least 1
  int req_groups;     // groups per request: G / 8 rounded up
  int lo_reqs;        // B with RoPE: the rest of request b's rotated queries is request b + B of the maps; 0 without
  // float offsets into the workspace: partial outputs and log-sum-exps of pair pieces [2 * rows],
  // single prefix pieces [rows] and own pieces [G]; then (int) B + 1 sums of points and the rotated
  // queries (bf16 [2, B, n_h, D]: the rounded values and what the rounding left)
  long long o2, o1, o0, l2, l1, l0, sums, q, end;
};

namespace {

constexpr int BM = 128;  // rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Points on the lines: a tile, the start of a segment.
constexpr int kTileCost = 8, kPieceCost = 8;

// Register split as in prefill_tc.cu: a softmax thread holds a row of 128 scores.
constexpr int kLaunchRegs = 168;
constexpr int kRegsCtl = 152, kRegsSoftmax = 176;
constexpr int kRegsNeeded = 4 * 32 * kRegsCtl + 8 * 32 * kRegsSoftmax;
static_assert(kRegsNeeded <= kThreads * kLaunchRegs, "register split exceeds the launch's pool");

// A piece: tiles [t, t_end) of one segment for one worker (or, on pair tiles, both).
enum : int { kNone = -1, kPair = 0, kPrefix = 1, kOwn = 2 };
struct Piece {
  int kind, g;
  int b;         // own: the request; pair: the pair of row tiles
  int t, t_end;
  int keys;      // keys of the whole segment: tile t holds min(128, keys - 128 t) of them
  int q_alt;     // 1: the query rows lie kAltRows further on
  int q_back;    // they may be loaded when the Q K of this many pieces before are done
};

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kBlocks = D / 64;             // 64-dim column blocks of a tile
  static constexpr int kBlockBytes = BM * 128;       // one column block (128 rows x 128 bytes, swizzled)
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kKStages = D == 128 ? 2 : 5;
  static constexpr int kVStages = D == 128 ? 3 : 6;
  // Pieces that warp 3 has handed out and not passed itself, and the queues' length.  An entry is
  // written again kQueue - kAhead pieces after warp 3 saw its piece's last V tile, and then at most
  // kVStages + 1 of a worker's pieces are unfinished (a V stage is reloaded only after its P V, a
  // piece's P only written after the epilogue of the piece before).
  static constexpr int kAhead = 4;
  static constexpr int kQueue = D == 128 ? 8 : 16;
  static_assert(kQueue - kAhead >= kVStages + 1, "queue entries in use");
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kVStages * kTileBytes;
  static constexpr int kBarBytes = D == 128 ? 1024 : 2048;
  static constexpr int kSmemBytes = kBarOff + kBarBytes + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kOCol = 256;             // O of worker w at kOCol + w D
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, true);
};

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  uint64_t v_full[C::kVStages], v_empty[C::kVStages], v_fixed[C::kVStages];
  uint64_t q_full[2][2], q_free[2][2];  // per worker, alternating between its pieces
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t piece_full[2][C::kQueue];
  uint64_t fin;
  Piece piece[2][C::kQueue];
  WaitCtl wc;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars<64>) <= Cfg<64>::kBarBytes && sizeof(Bars<128>) <= Cfg<128>::kBarBytes, "barrier block");

// ------------------------------------------------------------------------------------- the line
// Points are 32-bit: decode_paged_tc_supported bounds the line.
// The first tile of a segment (n tiles, the first one at point p0) that starts at or behind point x.
__device__ __forceinline__ int tile_at(int x, int p0, int n) {
  const int d = x - p0;
  return d <= 0 ? 0 : min(n, static_cast<int>((static_cast<unsigned>(d) + kTileCost - 1) / kTileCost));
}
__device__ __forceinline__ int seg_points(int tiles) { return tiles > 0 ? tiles * kTileCost + kPieceCost : 0; }
__device__ __forceinline__ int own_tiles(const PagedDecodeArgs& a, int b) {
  const int L = paged_len(a, b);
  return L > a.prefix_len ? static_cast<int>((static_cast<unsigned>(L - a.prefix_len) + BN - 1) / BN) : 0;
}

// [0, total) cut into n equal parts, the first `extra` of them one point longer.
struct Cut {
  int part, extra;
  __device__ __forceinline__ Cut(int total, int n) {
    part = static_cast<int>(static_cast<unsigned>(total) / static_cast<unsigned>(n));
    extra = total - part * n;
  }
  __device__ __forceinline__ int at(int k) const { return part * k + min(k, extra); }
  __device__ __forceinline__ int holder(int x) const {  // the part that holds point x
    const int wide = extra * (part + 1);                // the end of the longer parts
    const bool in_wide = x < wide;
    const unsigned len = in_wide ? part + 1 : part;     // part > 0 behind `wide`
    return (in_wide ? 0 : extra) + static_cast<int>(static_cast<unsigned>(in_wide ? x : x - wide) / len);
  }
};

// The two lines, once the sum of the requests' own points (of one KV head) is known: pair tiles on
// [0, pair_end); single prefix tiles on [0, prefix_end), then own tiles.
struct Lines {
  int pair_end, prefix_end;
  Cut pairs, singles;
  __device__ __forceinline__ Lines(const PagedTcPlan& p, int n_kv, int own)
      : pair_end(p.n_pairs * n_kv * seg_points(p.prefix_tiles)),
        prefix_end(p.odd * n_kv * seg_points(p.prefix_tiles)),
        pairs(pair_end, p.ctas),
        singles(prefix_end + own * n_kv, 2 * p.ctas) {}
};

// Where a piece's query rows lie in its worker's Q tile.  Up to kGroups groups of eight rows (an own piece's,
// or the prefix's for a small batch): group j in rows 32 (j mod 4) + 16 (j / 4), so that a softmax warp has
// one before any has two, followed by the rests of the same rows.  More rows than that: one after the other.
// Own pieces of at most 4 groups alternate between the tile and the tile 16 rows on, so that the next piece's
// rows load while this one's are read (an MMA reads 128 rows from either; what lies between a piece's rows
// reaches only lanes that nobody reads).  A piece whose rows alternate waits for the Q K of the piece two
// before it, any other for those of the piece before.
constexpr int kGroups = 8;
__host__ __device__ __forceinline__ int group_row(int j) { return 32 * (j & 3) + 16 * (j >> 2); }
constexpr int kAltRows = 16;

// A walk along one worker's parts of the lines: the next segment, its first point, its next tile, and
// where the part ends.  Pair pieces come first (in both workers' walks), then single prefix pieces,
// then own ones.
struct Walk {
  int kind, g, b, t, s0, end;                                   // of the pairs, then of the rest
  int rest_kind, rest_g, rest_b, rest_t, rest_s0, rest_end;  // where the single tiles begin
  int q_alt;  // Piece::q_alt of the last piece; -1: that piece's rows do not alternate
  int keys, nt;  // own keys and tiles of request b, once the walk is there
};

// To the first request from w.b on that has keys of its own.
__device__ __forceinline__ void seek_request(const PagedDecodeArgs& a, Walk& w) {
  for (; w.b < a.B; ++w.b) {
    w.keys = paged_len(a, w.b) - a.prefix_len;
    if (w.keys > 0) break;
  }
  w.nt = static_cast<int>((static_cast<unsigned>(w.keys) + BN - 1) / BN);
}

// The next piece of a walk; kind kNone at its end.  Own pieces, of which there may be thousands, take few
// instructions: one warp hands out all pieces of a CTA, and its code is fetched again for each.
__device__ __forceinline__ Piece next_piece(const PagedDecodeArgs& a, const PagedTcPlan& pl, Walk& w) {
  Piece u;
  u.kind = kNone;
  if (w.kind != kOwn) {
    if (w.kind == kPair) {
      const int t_end = tile_at(w.end, w.s0 + kPieceCost, pl.prefix_tiles);
      if (w.g < a.n_kv && w.t < t_end) {
        u = Piece{kPair, w.g, w.b, w.t, t_end, a.prefix_len, 0, 1};
        w.t = t_end;
        if (t_end == pl.prefix_tiles) {
          w.t = 0;
          w.s0 += seg_points(pl.prefix_tiles);
          if (++w.b == pl.n_pairs) {
            w.b = 0;
            ++w.g;
          }
        }
        return u;
      }
      w.kind = w.rest_kind;
      w.g = w.rest_g;
      w.b = w.rest_b;
      w.t = w.rest_t;
      w.s0 = w.rest_s0;
      w.end = w.rest_end;
    }
    for (; w.kind == kPrefix && w.g < a.n_kv; ++w.g) {
      const int t_end = tile_at(w.end, w.s0 + kPieceCost, pl.prefix_tiles), t = w.t;
      if (t >= t_end && t < pl.prefix_tiles) return u;  // the part ends here
      if (t < t_end) u = Piece{kPrefix, w.g, 0, t, t_end, a.prefix_len, 0, 1};
      w.t = t_end;
      if (t_end < pl.prefix_tiles) return u;
      w.t = 0;
      w.s0 += seg_points(pl.prefix_tiles);
      if (t < t_end) {
        ++w.g;
        return u;
      }
    }
    if (w.kind == kPrefix) w.g = 0;
    w.kind = kOwn;
    seek_request(a, w);
  }
  while (w.b < a.B) {
    const int t_end = tile_at(w.end, w.s0 + kPieceCost, w.nt), t = w.t;
    if (t >= t_end && t < w.nt) break;  // the part ends here
    if (t < t_end) {
      const bool turn = w.q_alt >= 0;
      const int alt = turn ? w.q_alt ^ 1 : 0;
      if (pl.own_groups > 0 && pl.own_groups <= 4) w.q_alt = alt;
      u = Piece{kOwn, w.g, w.b, t, t_end, w.keys, alt, turn ? 2 : 1};
    }
    w.t = t_end;
    if (t_end == w.nt) {
      w.t = 0;
      w.s0 += seg_points(w.nt);
      if (++w.g == a.n_kv) {
        w.g = 0;
        ++w.b;
        seek_request(a, w);
      }
    }
    if (t < t_end) break;
  }
  return u;
}

// Keys of tile t.
__device__ __forceinline__ int tile_keys(const Piece& u, int t) { return min(BN, u.keys - t * BN); }

// ------------------------------------------------------------------------------------- waits
// A wait whose slow part is out of line: two dozen inlined copies of it were a quarter of the code.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  return mbar_wait(bar, parity, *w);
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, w);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  const bool ok = lane_wait(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
}
// In line, for the softmax warps (beside their tile loops the compiler finds no registers for a call),
// and short: what they wait for comes from the other roles, whose waits keep the time and raise the
// abort flag; the count only bounds the loop should none of them be left.
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 26) && !(ok = mbar_try_wait(bar, parity)) && !*w->abort_flag; ++it) {
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __noinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

// The MMAs with shared-memory descriptors by their low words (address and leading offset): the high words of all
// tiles here are the same, and a burst's descriptors differ by constants that never carry.  Half the instructions
// per MMA of 64-bit descriptors.
constexpr uint32_t kDescHigh = static_cast<uint32_t>(sdesc_sw128(0, 16, 1024) >> 32);
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}

struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// A role's place in one worker's queue: the piece it is in and its tile there.
template <int D>
struct Cursor {
  Piece u;
  int t, w;
  uint32_t n;  // pieces taken
  enum { kLane, kWarp, kRow };  // who waits: one lane, a warp, a softmax warp
  template <int WHO>
  __device__ __forceinline__ bool take(Bars<D>* bars, const WaitCtl* wc) {
    constexpr uint32_t kQueue = Cfg<D>::kQueue;
    uint64_t* bar = &bars->piece_full[w][n % kQueue];
    const uint32_t par = (n / kQueue) & 1u;
    const bool ok = WHO == kWarp ? warp_wait(bar, par, wc) : WHO == kRow ? row_wait(bar, par, wc) : lane_wait(bar, par, wc);
    if (ok) u = bars->piece[w][n % kQueue];
    else u.kind = kNone;
    t = u.t;
    ++n;
    return ok;
  }
  __device__ __forceinline__ bool live() const { return u.kind != kNone; }
};

// What the MMA issuer keeps of a piece: its tiles left (0: no piece), whether none has its P V yet, whether its last
// tile is not whole.  (With whole pieces kept, a visit took long enough to bound short pieces and 64-dim heads.)
struct Slim {
  int left;
  uint32_t n, w;  // pieces taken, the worker
  bool first, part, alt, pair;
  __device__ __forceinline__ Slim(const Piece& u, uint32_t taken, uint32_t worker)
      : left(u.kind == kNone ? 0 : u.t_end - u.t),
        n(taken),
        w(worker),
        first(true),
        part(u.keys < u.t_end * BN),
        alt(u.q_alt != 0),
        pair(u.kind == kPair) {}
};

// ------------------------------------------------------------------------------------- softmax of a tile
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 TMEM lanes as MMA fragments, 32 columns of 32 bits: thread t has, for j = 0 .. 3, columns
// 8 j + 2 (t & 3) + {0, 1} of lane t / 4 in r[4 j], r[4 j + 1] and of lane t / 4 + 8 in r[4 j + 2], r[4 j + 3].
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 columns of bf16 in 16 of 32 bits: the pair 8 j + 2 (t & 3) + {0, 1} of lane t / 4 in r[2 j], of lane t / 4 + 8
// in r[2 j + 1].
__device__ __forceinline__ void tmem_st_frag_bf16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// This thread's row of O times alpha, before the tile's P V; the P V before has completed (the
// tile's scores were committed after it).
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t o_addr, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t orow[32];
    tmem_ld32(o_addr + c * 32, orow);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) orow[e] = __float_as_uint(__uint_as_float(orow[e]) * alpha);
    tmem_st32(o_addr + c * 32, orow);
  }
}

__device__ __forceinline__ void swap(float& x, float& y) {
  const float z = x;
  x = y;
  y = z;
}

// Among four lanes (lj = lane & 3): piece e of lane k becomes piece k of lane e.
__device__ __forceinline__ void transpose_pieces(uint4* pc, int lj) {
  const bool b1 = (lj & 2) != 0, b0 = (lj & 1) != 0;
  const uint4 r0 = shfl_xor_u4(b1 ? pc[0] : pc[2], 2), r1 = shfl_xor_u4(b1 ? pc[1] : pc[3], 2);
  pc[0] = b1 ? r0 : pc[0];
  pc[1] = b1 ? r1 : pc[1];
  pc[2] = b1 ? pc[2] : r0;
  pc[3] = b1 ? pc[3] : r1;
  const uint4 q0 = shfl_xor_u4(b0 ? pc[0] : pc[1], 1), q1 = shfl_xor_u4(b0 ? pc[2] : pc[3], 1);
  pc[0] = b0 ? q0 : pc[0];
  pc[1] = b0 ? pc[1] : q0;
  pc[2] = b0 ? q1 : pc[2];
  pc[3] = b0 ? pc[3] : q1;
}

// A sum and the rest that belongs to it.  A sum that an infinity has made infinite is the result: the rests of the
// factors it met may be 0 or of the other sign, and make NaN of it.
__device__ __forceinline__ float with_rest(uint32_t sum, uint32_t rest) {
  const float x = __uint_as_float(sum);
  return fabsf(x) < INFINITY ? x + __uint_as_float(rest) : x;
}

// A tile's scores (n real keys) of one group of eight rows become its weights P: p = 2^(s * scale*log2e - m).
// m moves only when the row maximum grew by more than the threshold; O and l are then scaled by
// 2^(m_old - m_new), exactly (l and O share their reference).
// TMEM lane i of the group's 16 holds row i's product with the rounded queries, lane i + 8 (with RoPE) the one
// with what that rounding left; their sum is the score.  The weights go back in the same way: lane i their
// value as bf16, lane i + 8 what is left, so that O's two lanes add up to P V with P to 17 bits.  The MMA's
// 128 rows cost the same, filled or not, so neither costs tensor time.  Four threads hold a row, both lanes of
// a key in the same thread; l_run is this thread's keys' share.
// An infinite key's score is the rounded queries' alone: a rest of 0 or of the other sign would make NaN of a score of
// -inf.  The maximum passes NaN over, so only the weights ask, one min per score (asking both times whether the score
// is finite made 64-dim heads 15% slower).
// 32 keys at a time and every score read twice, for the sake of a short loop: many pieces are a tile or two,
// and the roles' code is fetched again for each (1024 requests of 100 keys: 117 us; 64 keys at a time 126,
// all 128 at once 136).
template <int D>
__device__ __forceinline__ void softmax_group(uint32_t s_addr, uint32_t o_addr, int n, bool rescale, bool lo, int col,
                                              float scale_log2, float& m_run, float& l_run) {
  const auto scores = [&](float* s, int c, bool weigh) {
    uint32_t v[16];
    tmem_ld_frag(s_addr + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = __uint_as_float(v[4 * (e >> 1) + (e & 1)]);
    if (lo) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 rest = make_float2(__uint_as_float(v[2 * e + 2]), __uint_as_float(v[2 * e + 3]));
        if (weigh) rest = make_float2(fminf(rest.x, FLT_MAX), fminf(rest.y, FLT_MAX));
        const float2 x = __fadd2_rn(make_float2(s[e], s[e + 1]), rest);
        s[e] = x.x;
        s[e + 1] = x.y;
      }
    }
    if (n < c + 32) {  // keys behind the segment's end
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * (e >> 1) + (e & 1) >= n - col - c) s[e] = -INFINITY;
    }
  };
  float mx = -INFINITY, m2 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < BN; c += 32) {
    float s[8];
    scores(s, c, false);
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      mx = fmax3(mx, s[e], s[e + 1]);
      m2 = fmax3(m2, s[e + 2], s[e + 3]);
    }
  }
  mx = fmaxf(mx, m2);
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * scale_log2;
  const bool need = mx > m_run + kRescaleThreshold;
  float alpha = 1.f;
  if (need) {
    if (m_run != -INFINITY) alpha = fast_exp2(m_run - mx);
    l_run *= alpha;
    m_run = mx;
  }
  if (__any_sync(0xffffffffu, need && rescale)) {  // the P V before has completed
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[16];
      tmem_ld_frag(o_addr + c, o);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
      tmem_st_frag(o_addr + c, o);
    }
  }
  const float2 sl2 = make_float2(scale_log2, scale_log2);
  const float m_ref = (m_run == -INFINITY) ? 0.f : m_run;  // every score so far is -inf: weights 0
  const float2 nm2 = make_float2(-m_ref, -m_ref);
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < BN; c += 32) {
    float s[8];
    scores(s, c, true);
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8 / 2; ++j) {
      const float2 x = __ffma2_rn(make_float2(s[2 * j], s[2 * j + 1]), sl2, nm2);
      const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      acc[j & 1] = __fadd2_rn(acc[j & 1], pp);
      p[2 * j] = pack_bf16x2(pp.x, pp.y);
      p[2 * j + 1] = pack_bf16x2(pp.x - __uint_as_float(p[2 * j] << 16), pp.y - __uint_as_float(p[2 * j] & 0xffff0000u));
    }
    tmem_st_frag_bf16(s_addr + c / 2, p);  // over scores already taken
  }
  acc[0] = __fadd2_rn(acc[0], acc[1]);
  l_run += acc[0].x + acc[0].y;
}

// The same for a row per thread (TMEM lane), with Q and P rounded to bf16: each of the two moves an output by
// about as much as its own rounding to bf16 does (0.0029 of the largest output against 64 bits, instead of
// 0.0017).  The rows fill the MMA here, and the products for what the roundings leave would be more MMAs: for P's,
// 256 requests behind 16384 tokens took 138 us, without 92; for Q's there is no shared memory.
// The whole row is in registers, each score read once and the chains independent: on pair tiles the tensor pipe
// waits for the softmax (0.6 us of a worker's 1.6 us per tile; handing P over in two halves, for the first half's
// P V to run beside the second's exponentials, made it 1.7).
template <int D>
__device__ __forceinline__ void softmax_row(uint32_t s_addr, uint32_t o_addr, int n, bool rescale,
                                                  float scale_log2, float& m_run, float& l_run) {
  uint32_t sr[BN];
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_addr + c * 32, sr + c * 32);
  tmem_wait_ld();
  float s[BN];
#pragma unroll
  for (int c = 0; c < BN; ++c) s[c] = __uint_as_float(sr[c]);
  if (n < BN) {
#pragma unroll
    for (int c = 0; c < BN; ++c)
      if (c >= n) s[c] = -INFINITY;
  }
  // row maximum: 8 independent chains of three-input max, then a tree
  float m8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) m8[e] = s[e];
#pragma unroll
  for (int c = 8; c + 16 <= BN; c += 16)
#pragma unroll
    for (int e = 0; e < 8; ++e) m8[e] = fmax3(m8[e], s[c + e], s[c + 8 + e]);
#pragma unroll
  for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], s[BN - 8 + e]);
  const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7])) *
                   scale_log2;
  // the reference maximum moves only when the row's grew by more than the threshold
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
#pragma unroll
  for (int c = 0; c < BN / 4; ++c) {
    const float2 x = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sl2, nm2);
    const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    acc[c & 3] = __fadd2_rn(acc[c & 3], pp);
    pr[c] = pack_bf16x2(pp.x, pp.y);
  }
  tmem_st32(s_addr, pr);
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

// What the rounding of x to bf16 left, as bf16; 0 behind an infinity.
__device__ __forceinline__ uint4 bf16_rest(const float* x, uint4 rounded) {
  float y[8];
  bf16x8_to_f32(rounded, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fabsf(y[e]) < INFINITY ? x[e] - y[e] : 0.f;
  return f32_to_bf16x8(y);
}

// The new tokens' queries rotated at their positions, bf16 [2, B, n_h, D] (the values and the rests): one
// thread per (row, chunks of 8 dims c and c + D / 16).  The decode kernel may start as soon as this one has.
// ANY: for tables of more than 2^24 tokens, at any position.
template <int D, bool ANY>
__global__ void __launch_bounds__(256) paged_rope_q_kernel(const __grid_constant__ PagedDecodeArgs a,
                                                           const __grid_constant__ RopeFreq f, __nv_bfloat16* out) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kCP = D / 16;
  __shared__ float f_hi[D / 2], f_lo[D / 2];
  for (int i = threadIdx.x; i < f.n_pairs; i += 256) {
    f_hi[i] = f.hi[i];
    f_lo[i] = f.lo[i];
  }
  __syncthreads();
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = idx / kCP;
  if (row >= static_cast<long long>(a.B) * a.n_h) return;
  const int c = static_cast<int>(idx % kCP);
  const int pos = max(paged_len(a, static_cast<int>(row / a.n_h)), 1) - 1;
  const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row * D) + c;
  uint4* const o = reinterpret_cast<uint4*>(out + row * D) + c;
  float x0[8], x1[8];
  bf16x8_to_f32(q[0], x0);
  bf16x8_to_f32(q[kCP], x1);
  with_angles<ANY, true>(pos, [&](auto angle) {
    if (f.half) {  // pair 8 c + e is (x0[e], x1[e])
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float sn, cs;
        angle(f_hi[c * 8 + e], f_lo[c * 8 + e], &sn, &cs);
        rotate_pair(x0[e], x1[e], sn, cs);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sn, cs;
        angle(f_hi[c * 4 + e], f_lo[c * 4 + e], &sn, &cs);
        rotate_pair(x0[2 * e], x0[2 * e + 1], sn, cs);
        angle(f_hi[D / 4 + c * 4 + e], f_lo[D / 4 + c * 4 + e], &sn, &cs);
        rotate_pair(x1[2 * e], x1[2 * e + 1], sn, cs);
      }
    }
  });
  o[0] = f32_to_bf16x8(x0);
  o[kCP] = f32_to_bf16x8(x1);
  uint4* const rest = o + static_cast<long long>(a.B) * a.n_h * (D / 8);
  rest[0] = bf16_rest(x0, o[0]);
  rest[kCP] = bf16_rest(x1, o[kCP]);
}

// tm_q: boxes of the query rows of one request and KV head (own pieces: all G of them, or a group's); tm_qn: of
// the requests of a prefix piece (a row tile's, or a group's).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ PagedTcPlan pl,
                    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qn,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars<D>* bars = reinterpret_cast<Bars<D>*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");  // the combine kernel may start to wait
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 2);  // the MMA issuer and the clearing warp, which passes every tile
      mbar_init(&bars->v_fixed[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars->q_full[w][i], 1);
        mbar_init(&bars->q_free[w][i], 1);
      }
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->p_full[w], 128);
      mbar_init(&bars->o_done[w], 1);
      mbar_init(&bars->o_empty[w], 128);
      for (int i = 0; i < C::kQueue; ++i) mbar_init(&bars->piece_full[w][i], 1);
    }
    mbar_init(&bars->fin, 1);
    bars->abort_flag = 0;
    bars->wc.abort_flag = &bars->abort_flag;
    bars->wc.status = a.status;
    bars->wc.limit_ns = a.wait_limit_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl* const wc = &bars->wc;

  if (warp < 4) {
    setmaxnreg_dec<kRegsCtl>();
    // Every role visits the two workers' tiles in turns, worker 0 first, one worker alone when the
    // other is done.  A pair tile is in both workers' queues: its K and V belong to worker 0's visit.
    Cursor<D> cur, oth;  // the worker whose turn it is, and the other one
    cur.w = 0;
    oth.w = 1;
    cur.n = oth.n = 0;
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ TMA producers
      const bool is_v = warp == 2;
      const uint32_t n_stages = is_v ? C::kVStages : C::kKStages;
      uint8_t* const ring = smem + (is_v ? C::kVOff : C::kKOff);
      uint64_t* const full = is_v ? bars->v_full : bars->k_full;
      uint64_t* const empty = is_v ? bars->v_empty : bars->k_empty;
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      if (lane == 0) tma_prefetch_desc(map);
      const int box_shift = min(a.page_shift, 7);  // rows per box: a page, or half of a 256-token page
      const int boxes = BN >> box_shift;            // per column block of a tile
      const int box = lane & (boxes - 1), blk = lane / boxes;  // lane l loads block l / boxes of page l mod boxes
      // query rows, a lane per box: 64 dims of group q_j's rows, or (q_lo) of what their rounding left
      const int q_lo = (lane / C::kBlocks) & 1, q_j = lane / (2 * C::kBlocks), q_dim = (lane & (C::kBlocks - 1)) * 64;
      const int q_dst = (group_row(q_j) + q_lo * 8) * 128 + q_dim / 64 * C::kBlockBytes;
      const int q_head = 8 * q_j, q_rest = q_lo * pl.lo_reqs;  // of an own piece
      const bool q_box = pl.own_groups > 0 ? q_j < pl.own_groups && (!q_lo || pl.lo_reqs > 0) : q_j == 0 && !q_lo;
      const int q_bytes = (pl.own_groups > 0 ? pl.own_groups * pl.own_group * (pl.lo_reqs > 0 ? 2 : 1) : a.n_h / a.n_kv) *
                          128 * C::kBlocks;
      Ring r;
      uint32_t issued = 0, last_ph = 0;
      int id_cur = -1, id_oth = -1;  // the lane's page of each worker's next tile
      auto fetch = [&](const Cursor<D>& s) -> int {
        const int* tbl = s.u.kind == kOwn ? a.block_table + static_cast<long long>(s.u.b) * a.max_blocks +
                                                (a.prefix_len >> a.page_shift)
                                          : a.prefix_pages;
        const int key = s.t * BN + (box << box_shift);
        return s.live() && blk < C::kBlocks && key < s.u.keys ? tbl[key >> a.page_shift] : -1;
      };
      bool ok = cur.template take<Cursor<D>::kWarp>(bars, wc) && oth.template take<Cursor<D>::kWarp>(bars, wc);
      id_cur = fetch(cur);
      id_oth = fetch(oth);
      if (!is_v) {  // the rotated queries come from the kernel before
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("fence.proxy.async.global;" ::: "memory");
      }
      while (ok && (cur.live() || oth.live())) {
        if (cur.live()) {
          if (!is_v && cur.t == cur.u.t) {
            // the piece's query rows
            const uint32_t n = cur.n - 1;
            const bool own = cur.u.kind == kOwn;
            const uint32_t back = cur.u.q_back;
            if (n >= back) {
              const uint32_t m = n - back;
              if (!warp_wait(&bars->q_free[cur.w][m & 1u], (m >> 1) & 1u, wc)) break;
            }
            uint64_t* const bar = &bars->q_full[cur.w][n & 1u];
            uint8_t* const dst = smem + C::kQOff + cur.w * C::kTileBytes + q_dst + cur.u.q_alt * (kAltRows * 128);
            if (own) {
              if (lane == 0) mbar_arrive_expect_tx(bar, q_bytes);
              __syncwarp();
              if (q_box) tma_load_4d(dst, &tm_q, bar, q_dim, q_head, cur.u.g, cur.u.b + q_rest);
            } else {
              const int groups = pl.prefix_groups;
              if (lane == 0)
                mbar_arrive_expect_tx(bar, (groups > 0 ? groups * pl.prefix_group * (pl.lo_reqs > 0 ? 2 : 1) : pl.rows) *
                                               128 * C::kBlocks);
              __syncwarp();
              if (groups > 0 ? q_j < groups && (!q_lo || pl.lo_reqs > 0) : q_j == 0 && !q_lo) {
                const int before = q_j / pl.req_groups;  // requests (groups of G <= 8 rows) before the group's
                const int tile = cur.u.kind == kPair ? 2 * cur.u.b + cur.w : 2 * pl.n_pairs;  // row tile of the prefix
                tma_load_4d(dst, &tm_qn, bar, q_dim, 8 * (q_j - before * pl.req_groups), cur.u.g,
                            (groups > 0 ? before * pl.group_reqs : tile * pl.row_reqs) + q_rest);
              }
            }
            __syncwarp();
          }
          if (cur.u.kind != kPair || cur.w == 0) {
            if (!warp_wait(&empty[r.st], r.ph ^ 1, wc)) break;
            const int n_boxes = (tile_keys(cur.u, cur.t) + (1 << box_shift) - 1) >> box_shift;  // others hold no key
            if (lane == 0)
              mbar_arrive_expect_tx(&full[r.st], static_cast<uint32_t>(n_boxes * C::kBlocks) << (box_shift + 7));
            __syncwarp();
            if (blk < C::kBlocks && box < n_boxes)
              tma_load_4d(ring + r.st * C::kTileBytes + blk * C::kBlockBytes + (box << (box_shift + 7)), map,
                          &full[r.st], blk * 64, cur.u.g, (cur.t * BN) & ((1 << a.page_shift) - 1), id_cur);
            issued |= 1u << r.st;
            last_ph = (last_ph & ~(1u << r.st)) | (r.ph << r.st);
            r.next(n_stages);
          }
          if (++cur.t == cur.u.t_end) ok = cur.template take<Cursor<D>::kWarp>(bars, wc);
          id_cur = fetch(cur);
        }
        if (oth.live()) {
          const Cursor<D> x = cur;
          cur = oth;
          oth = x;
          const int y = id_cur;
          id_cur = id_oth;
          id_oth = y;
        }
      }
      if (bars->abort_flag) {  // let every copy in flight land before shared memory goes away
        for (uint32_t s = 0; s < n_stages; ++s)
          if (issued & (1u << s)) drain_wait(&full[s], (last_ph >> s) & 1, a.wait_limit_ns);
        if (!is_v)  // query rows of the piece a worker is in, or before it
          for (int i = 0; i < 4; ++i) {
            const uint32_t n = ((i & 1) ? oth.n : cur.n) - 1 - (i >> 1);
            const int w = (i & 1) ? oth.w : cur.w;
            if (static_cast<int>(n) >= 0) drain_wait(&bars->q_full[w][n & 1u], (n >> 1) & 1u, 1000000ull);
          }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        const uint32_t q_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024));
        const uint32_t k_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024));
        const uint32_t v_desc0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kVOff), C::kBlockBytes, 1024));
        Ring kr, vr;
        uint32_t pph = 0, oph = 0, fix_ph = 0;  // parities, one bit per worker (fix_ph: per stage)
        uint32_t pending = 0;                   // bit w: worker w's Q K is out, its P V not yet
        bool ok = cur.template take<Cursor<D>::kLane>(bars, wc) && oth.template take<Cursor<D>::kLane>(bars, wc);
        auto issue_qk = [&](uint32_t w, uint32_t alt, int from, int to) {
          const uint32_t a0 = q_desc0 + ((w * C::kTileBytes + alt * (kAltRows * 128)) >> 4);
          const uint32_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = from; kk < to; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4;
            mma_ss_lo(tmem + w * 128u, a0 + off, b0 + off, C::kIdescQK, kk > 0 ? 1u : 0u);
          }
        };
        auto issue_pv = [&](uint32_t w, bool first) {
          const uint32_t b0 = v_desc0 + ((vr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts_lo(tmem + C::kOCol + w * D, tmem + w * 128u + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescPV,
                   (!first || kk > 0) ? 1u : 0u);
        };
        Slim me(cur.u, cur.n, 0), you(oth.u, oth.n, 1);
        // one visit: P V of the worker's tile, then Q K of its next one
        while (ok && (me.left || you.left)) {
          if (me.pair && me.w == 0 && pending == 3u && !me.first && me.left > 2) {
            // inside a pair piece, both workers at the same tile: no piece begins or ends before its last two, and the
            // tiles are whole (only a segment's last one may not be).  What the next turn needs is waited for in front
            // of this turn's last MMAs, so that the tensor pipe does not run dry.
            if (!(ok = lane_wait(&bars->v_full[vr.st], vr.ph, wc) && lane_wait(&bars->k_full[kr.st], kr.ph, wc))) break;
            for (; me.left > 2; --me.left) {
              if (!(ok = lane_wait(&bars->p_full[0], pph & 1u, wc))) break;
              pph ^= 1u;
              tc_fence_after();
              issue_pv(0, false);
              issue_qk(0, 0, 0, D / 16);
              mma_commit(&bars->s_full[0]);
              if (!(ok = lane_wait(&bars->p_full[1], (pph >> 1) & 1u, wc))) break;
              pph ^= 2u;
              tc_fence_after();
              issue_pv(1, false);
              mma_commit(&bars->v_empty[vr.st]);
              vr.next(C::kVStages);
              issue_qk(1, 0, 0, D / 32);
              Ring kn = kr;
              kn.next(C::kKStages);
              if (!(ok = lane_wait(&bars->v_full[vr.st], vr.ph, wc) && lane_wait(&bars->k_full[kn.st], kn.ph, wc))) break;
              tc_fence_after();
              issue_qk(1, 0, D / 32, D / 16);
              mma_commit(&bars->s_full[1]);
              mma_commit(&bars->k_empty[kr.st]);
              kr = kn;
            }
            you.left = me.left;
            if (!ok) break;
          }
          if constexpr (D == 64) {
            // likewise inside two single pieces: a tile of 64-dim heads comes every 0.75 us from HBM, less than a
            // visit with all its questions takes
            int turns = min(me.left, you.left) - 2;
            if (turns > 0 && !me.pair && !you.pair && pending == 3u && !me.first && !you.first) {
              me.left -= turns;
              you.left -= turns;
              uint32_t w = me.w;
              for (turns *= 2; turns > 0; --turns) {
                if (!(ok = lane_wait(&bars->v_full[vr.st], vr.ph, wc) && lane_wait(&bars->p_full[w], (pph >> w) & 1u, wc) &&
                           lane_wait(&bars->k_full[kr.st], kr.ph, wc)))
                  break;
                tc_fence_after();
                issue_pv(w, false);
                mma_commit(&bars->v_empty[vr.st]);
                issue_qk(w, me.w == w ? me.alt : you.alt, 0, D / 16);
                mma_commit(&bars->s_full[w]);
                mma_commit(&bars->k_empty[kr.st]);
                vr.next(C::kVStages);
                kr.next(C::kKStages);
                pph ^= 1u << w;
                w ^= 1u;
              }
              if (!ok) break;
            }
          }
          if (me.left) {
            const uint32_t w = me.w, bit = 1u << w;
            if (pending & bit) {
              if (!me.pair || w == 0) {
                if (!(ok = lane_wait(&bars->v_full[vr.st], vr.ph, wc))) break;
                if (me.left == 1 && me.part) {  // the rows behind the last key are cleared first
                  if (!(ok = lane_wait(&bars->v_fixed[vr.st], (fix_ph >> vr.st) & 1u, wc))) break;
                  fix_ph ^= 1u << vr.st;
                }
              }
              if (!(ok = lane_wait(&bars->p_full[w], (pph >> w) & 1u, wc))) break;
              pph ^= bit;
              if (me.first) {  // O has been read
                if (!(ok = lane_wait(&bars->o_empty[w], ((oph >> w) & 1u) ^ 1u, wc))) break;
                oph ^= bit;
              }
              tc_fence_after();
              issue_pv(w, me.first);
              if (!me.pair || w == 1) {
                mma_commit(&bars->v_empty[vr.st]);
                vr.next(C::kVStages);
              }
              me.first = false;
              pending &= ~bit;
              if (--me.left == 0) {
                mma_commit(&bars->o_done[w]);
                if (!(ok = lane_wait(&bars->piece_full[w][me.n % C::kQueue], (me.n / C::kQueue) & 1u, wc))) break;
                me = Slim(bars->piece[w][me.n % C::kQueue], me.n + 1, w);
              }
            }
            if (me.left) {
              if (!me.pair || w == 0) {
                if (!(ok = lane_wait(&bars->k_full[kr.st], kr.ph, wc))) break;
              }
              const uint32_t n = me.n - 1;
              if (me.first && !(ok = lane_wait(&bars->q_full[w][n & 1u], (n >> 1) & 1u, wc))) break;
              tc_fence_after();
              issue_qk(w, me.alt, 0, D / 16);
              mma_commit(&bars->s_full[w]);
              if (!me.pair || w == 1) {
                mma_commit(&bars->k_empty[kr.st]);
                kr.next(C::kKStages);
              }
              if (me.left == 1) mma_commit(&bars->q_free[w][n & 1u]);
              pending |= bit;
            }
          }
          if (you.left) {
            const Slim x = me;
            me = you;
            you = x;
          }
        }
        // every MMA issued so far completes before TMEM is released
        mma_commit(&bars->fin);
        drain_wait(&bars->fin, 0, a.wait_limit_ns);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ the walk, and value rows behind a segment's end
      // lanes 0-15 walk for worker 0, lanes 16-31 for worker 1, each half all alike
      const int me = lane >> 4;
      Walk walk;
      int own_sum, before_sum;
      {
        // lane i sums the points of requests [i s, (i + 1) s)
        const int strip = (a.B + 31) / 32;
        const int b_lo = min(a.B, lane * strip), b_hi = min(a.B, b_lo + strip);
        int mine = 0;
#pragma unroll 8
        for (int b = b_lo; b < b_hi; ++b) mine += seg_points(own_tiles(a, b));
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        const int own = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
        const Lines lines(pl, a.n_kv, own);
        const int cta = blockIdx.x;
        const int lo = lines.singles.at(2 * cta + me), hi = lines.singles.at(2 * cta + me + 1);
        // where the single tiles begin
        walk.rest_end = lo < hi ? hi : 0;  // an empty part: no tile starts before point 0
        walk.rest_kind = kOwn;
        walk.rest_g = walk.rest_b = walk.rest_t = 0;
        walk.rest_s0 = lines.prefix_end;
        if (lo < lines.prefix_end) {
          const int len = seg_points(pl.prefix_tiles);
          walk.rest_kind = kPrefix;
          walk.rest_g = lo / len;
          walk.rest_s0 = walk.rest_g * len;
          walk.rest_t = tile_at(lo, walk.rest_s0 + kPieceCost, pl.prefix_tiles);
        }
        // own tiles: the lane whose requests hold the part's first point finds the tile there (for each worker)
        const bool own_start = lo < hi && lo >= lines.prefix_end;
        const int first = own_start ? lo - lines.prefix_end : -1;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const int x = __shfl_sync(0xffffffffu, first, 16 * w);
          int fb = 0, fat = 0;
          const bool here = x >= before * a.n_kv && x < (before + mine) * a.n_kv;
          if (here) {
            int b = b_lo, at = before, len = seg_points(own_tiles(a, b));
            while (x >= (at + len) * a.n_kv) {
              at += len;
              len = seg_points(own_tiles(a, ++b));
            }
            fb = b;
            fat = at;
          }
          const int src = max(__ffs(__ballot_sync(0xffffffffu, here)) - 1, 0);
          fb = __shfl_sync(0xffffffffu, fb, src);
          fat = __shfl_sync(0xffffffffu, fat, src);
          if (own_start && me == w) {
            const int nt = own_tiles(a, fb), len = seg_points(nt);
            walk.rest_b = fb;
            walk.rest_g = (x - fat * a.n_kv) / len;
            walk.rest_s0 = lines.prefix_end + fat * a.n_kv + walk.rest_g * len;
            walk.rest_t = tile_at(lo, walk.rest_s0 + kPieceCost, nt);
          }
          __syncwarp();
        }
        // and the pairs before them
        const int x0 = lines.pairs.at(cta);
        walk.kind = kPair;
        walk.g = walk.b = walk.t = 0;
        walk.s0 = 0;
        walk.end = 0;
        walk.q_alt = -1;
        if (x0 < lines.pair_end) {
          const int len = seg_points(pl.prefix_tiles);
          const int seg = x0 / len;
          walk.end = lines.pairs.at(cta + 1);
          walk.s0 = seg * len;
          walk.t = tile_at(x0, walk.s0 + kPieceCost, pl.prefix_tiles);
          walk.g = seg / pl.n_pairs;
          walk.b = seg - walk.g * pl.n_pairs;
          if (walk.t == pl.prefix_tiles) {  // behind the segment's last tile
            walk.t = 0;
            walk.s0 += len;
            if (++walk.b == pl.n_pairs) {
              walk.b = 0;
              ++walk.g;
            }
          }
        }
        own_sum = own;
        before_sum = before;
      }
      uint32_t n_pub = 0, n_end = C::kAhead;  // pieces handed out by this half; and to be, so far
      Ring r;
      bool ok = true, take_cur = true, take_oth = true, first_round = true;
      for (;;) {
        // hand out pieces, kAhead in front of the ones this warp is in
        while (__any_sync(0xffffffffu, n_pub < n_end)) {
          if (n_pub < n_end) {
            const Piece u = next_piece(a, pl, walk);
            if ((lane & 15) == 0) {
              bars->piece[me][n_pub % C::kQueue] = u;
              mbar_arrive(&bars->piece_full[me][n_pub % C::kQueue]);
            }
            ++n_pub;
            if (u.kind == kNone) n_end = 0;  // the last one
          }
        }
        if (first_round) {  // CTA 0 leaves the sums of points for the combine kernel
          first_round = false;
          if (blockIdx.x == 0) {
            int* const sums = static_cast<int*>(a.workspace) + pl.sums;
            const int strip = (a.B + 31) / 32;
            for (int b = min(a.B, lane * strip), e = min(a.B, b + strip); b < e; ++b) {
              sums[b] = before_sum;
              before_sum += seg_points(own_tiles(a, b));
            }
            if (lane == 0) sums[a.B] = own_sum;
          }
        }
        if (take_cur) ok = cur.template take<Cursor<D>::kWarp>(bars, wc);
        if (take_oth) ok = ok && oth.template take<Cursor<D>::kWarp>(bars, wc);
        take_cur = take_oth = false;
        if (!ok || !(cur.live() || oth.live())) break;
        if (cur.live()) {
          if (cur.u.kind != kPair || cur.w == 0) {
            if (!warp_wait(&bars->v_full[r.st], r.ph, wc)) break;
            const int n = tile_keys(cur.u, cur.t);
            if (n < BN) {
              // rows n.. were not loaded or hold no token: their weights are 0, and 0 times anything must be 0
              uint8_t* const v = smem + C::kVOff + r.st * C::kTileBytes + n * 128;
#pragma unroll 1
              for (int i = lane; i < (BN - n) * 8; i += 32) {
#pragma unroll
                for (int blk = 0; blk < C::kBlocks; ++blk)
                  *reinterpret_cast<uint4*>(v + blk * C::kBlockBytes + i * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->v_fixed[r.st]);
            }
            if (lane == 0) mbar_arrive(&bars->v_empty[r.st]);
            r.next(C::kVStages);
          }
          if (++cur.t == cur.u.t_end) {
            take_cur = true;
            if (me == cur.w && n_end) ++n_end;
          }
        }
        // the finished piece's successor is taken before its worker's next turn
        if (oth.live()) {
          const Cursor<D> x = cur;
          cur = oth;
          oth = x;
          take_oth = take_cur;
          take_cur = false;
        }
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax warpgroups (workers)
    Cursor<D> cur;
    cur.w = (warp - 4) >> 2;
    cur.n = 0;
    const int w = cur.w;
    const int quad = warp & 3;       // TMEM lane quadrant
    const int r = quad * 32 + lane;  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + (w ? 128u : 0u);
    const uint32_t o_addr = tmem + lane_off + C::kOCol + (w ? D : 0);
    constexpr uint32_t kSecond = 16u << 16;  // to a warp's second group
    const int G = a.n_h / a.n_kv;
    uint32_t sph = 0, n_done = 0;
    bool ok = true;
    while (ok && cur.template take<Cursor<D>::kRow>(bars, wc) && cur.live()) {
      const Piece& u = cur.u;
      const int tile = u.kind == kPair ? 2 * u.b + w : 2 * pl.n_pairs;  // row tile of the prefix
      const int n_rows = u.kind == kOwn ? G : min(pl.row_reqs, a.B - tile * pl.row_reqs) * G;
      const int groups = u.kind == kOwn ? pl.own_groups : pl.prefix_groups;
      const bool active = groups > 0 ? quad < groups : quad * 32 < n_rows;  // this warp holds rows of the piece
      const int per_group = u.kind == kOwn ? pl.own_group : pl.prefix_group;
      const bool two = quad + 4 < groups;                                  // and two groups of them
      float m_run = -INFINITY, l_run = 0.f, m_2nd = -INFINITY, l_2nd = 0.f;
      if (groups == 0 && active) {  // a loop of its own (both kinds in one: 256 requests behind 16384 tokens 98 us, so 95)
        for (int t = u.t; t < u.t_end; ++t) {
          if (!row_wait(&bars->s_full[w], sph, wc)) { ok = false; break; }
          sph ^= 1;
          tc_fence_after();
          softmax_row<D>(s_addr, o_addr, tile_keys(u, t), t > u.t, a.scale_log2, m_run, l_run);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[w]);
        }
      } else {
        for (int t = u.t; t < u.t_end; ++t) {
          if (!row_wait(&bars->s_full[w], sph, wc)) { ok = false; break; }
          sph ^= 1;
          if (!active) {  // padding rows: whatever their P is, it reaches only their own O
            mbar_arrive(&bars->p_full[w]);
            continue;
          }
          tc_fence_after();
#pragma unroll 1
          for (uint32_t k = 0;; k = kSecond) {
            softmax_group<D>(s_addr + k, o_addr + k, tile_keys(u, t), t > u.t, pl.lo_reqs > 0, 2 * (lane & 3),
                             a.scale_log2, m_run, l_run);
            if (!two) break;
            swap(m_run, m_2nd);
            swap(l_run, l_2nd);
            if (k) break;
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[w]);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      // epilogue: the piece's normalised partial and its log-sum-exp
      if (!row_wait(&bars->o_done[w], n_done & 1, wc)) break;
      ++n_done;
      if (active) {
        tc_fence_after();
        float* const ws = static_cast<float*>(a.workspace);
        const long long worker = 2 * static_cast<long long>(blockIdx.x) + w;
        long long row = worker, o_at = pl.o0, l_at = pl.l0;
        if (u.kind == kOwn) {
          row = (row + static_cast<long long>(u.b) * a.n_kv + u.g) * G;
        } else if (u.kind == kPrefix) {
          row = (row + u.g) * pl.rows;
          o_at = pl.o1;
          l_at = pl.l1;
        } else {
          row = ((blockIdx.x + static_cast<long long>(u.g) * pl.n_pairs + u.b) * 2 + w) * pl.rows;
          o_at = pl.o2;
          l_at = pl.l2;
        }
        if (groups > 0) {
#pragma unroll 1
          for (int k = 0; k < (two ? 2 : 1); ++k) {
            const int i = lane >> 2;                  // this thread's row of the group
            int rr = (quad + 4 * k) * per_group + i;  // and of the piece
            bool real = i < per_group && rr < n_rows;
            if (u.kind == kPrefix && G > 8) {  // a request's last group may be a part of one
              const int req = (quad + 4 * k) / pl.req_groups, head = rr - 8 * req * pl.req_groups;
              rr = req * G + head;
              real = head < G && rr < n_rows;
            }
            float l = l_run + __shfl_xor_sync(0xffffffffu, l_run, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const float inv_l = l > 0.f ? 1.f / l : l;  // 0: every score is -inf; NaN stays
            float* const po = ws + o_at + (row + rr) * D + 2 * (lane & 3);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_ld_frag(o_addr + k * kSecond + c * 32, o);
              tmem_wait_ld();
              if (real) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  *reinterpret_cast<float2*>(po + c * 32 + e * 8) =
                      make_float2(with_rest(o[4 * e], o[4 * e + 2]) * inv_l, with_rest(o[4 * e + 1], o[4 * e + 3]) * inv_l);
              }
            }
            if (real && (lane & 3) == 0) ws[l_at + row + rr] = m_run + log2f(l);
            m_run = m_2nd;
            l_run = l_2nd;
          }
        } else {
          row += r;
          const float inv_l = l_run > 0.f ? 1.f / l_run : l_run;
          // four lanes exchange their rows' 16-byte pieces, so that a store writes 64 contiguous bytes of each
          // of eight rows
          const int lj = lane & 3;
          float* const pg = ws + o_at + (row - lj) * D + lj * 4;  // the four lanes' first row, this lane's piece
          const int left = n_rows - (r - lj);                     // rows of the four that exist
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t orow[16];
            tmem_ld16(o_addr + c * 16, orow);
            tmem_wait_ld();
            uint4 pc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t* o4 = orow + 4 * e;
              pc[e] = make_uint4(__float_as_uint(__uint_as_float(o4[0]) * inv_l),
                                 __float_as_uint(__uint_as_float(o4[1]) * inv_l),
                                 __float_as_uint(__uint_as_float(o4[2]) * inv_l),
                                 __float_as_uint(__uint_as_float(o4[3]) * inv_l));
            }
            transpose_pieces(pc, lj);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < left) *reinterpret_cast<uint4*>(pg + k * D + c * 16) = pc[k];
          }
          if (r < n_rows) ws[l_at + row] = m_run + log2f(l_run);
        }
        tc_fence_before();
      }
      mbar_arrive(&bars->o_empty[w]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The rows of one (request b, KV head g): their pieces are those of the CTAs (pair tiles) or workers
// (single tiles) between the one that holds the segment's first tile and the one that holds its last;
// a CTA or worker between them in whose part no tile starts wrote none.  A warp lists 32 candidates at
// a time, one per lane, then takes the pieces two by two: each lane four dims of up to four rows
// (kItems), all loads of the two pieces in flight, with a running maximum of their log-sum-exps.
// SPLIT: the warps of a block share the candidates of one (b, g) and merge in shared memory, for rows in
// many pieces; otherwise each warp has its own (b, g).
constexpr int kItems = 4;

template <int D, int WARPS, bool SPLIT>
__global__ void __launch_bounds__(WARPS * 32)
    paged_tc_combine_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ PagedTcPlan pl) {
  constexpr int kChunk = 32 * kItems;  // items (row, four dims) per pass
  __shared__ float4 red_acc[SPLIT ? WARPS * kChunk : 1];
  __shared__ float2 red_ml[SPLIT ? WARPS * kChunk : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned bg = SPLIT ? blockIdx.x : blockIdx.x * WARPS + warp;
  const int b = static_cast<int>(bg / static_cast<unsigned>(a.n_kv)), g = static_cast<int>(bg) - b * a.n_kv;
  if (b >= a.B) return;  // whole warps only
  const int nt = own_tiles(a, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials of the kernel before
  const float* const ws = static_cast<const float*>(a.workspace);
  const int* const sums = reinterpret_cast<const int*>(ws + pl.sums);
  const int sum_b = sums[b], sum_all = sums[a.B];
  const int G = a.n_h / a.n_kv;
  const int items = G * (D / 4);
  const long long out_row = static_cast<long long>(b) * a.n_h + g * G;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + out_row * D;
  if (nt == 0) {  // an empty place of the batch
    const int first = SPLIT ? threadIdx.x : lane, step = SPLIT ? WARPS * 32 : 32;
    for (int it = first; it < items; it += step) *reinterpret_cast<uint2*>(out + 4 * it) = make_uint2(0, 0);
    if (a.lse != nullptr)
      for (int i = first; i < G; i += step) a.lse[out_row + i] = -INFINITY;
    return;
  }
  const Lines lines(pl, a.n_kv, sum_all);
  // the rows' two segments, each from its first tile's point: the prefix (pair or single) and their own keys;
  // lanes 0 to 3 find who holds the first and the last tile of each
  const int tile = b / pl.row_reqs;  // row tile of the prefix
  const bool pair = tile < 2 * pl.n_pairs;
  const int seg = pair ? g * pl.n_pairs + tile / 2 : g;
  const int pre_p0 = kPieceCost + seg * seg_points(pl.prefix_tiles);
  const int own_p0 = lines.prefix_end + sum_b * a.n_kv + g * seg_points(nt) + kPieceCost;
  int held;
  {
    const bool own = lane & 2;
    const int x = (own ? own_p0 : pre_p0) + ((lane & 1) ? ((own ? nt : pl.prefix_tiles) - 1) * kTileCost : 0);
    held = pl.prefix_tiles > 0 || own ? (pair && !own ? lines.pairs : lines.singles).holder(x) : 0;
  }
  const int c0 = __shfl_sync(0xffffffffu, held, 0), w0 = __shfl_sync(0xffffffffu, held, 2);
  const int c1 = __shfl_sync(0xffffffffu, held, 1), w1 = __shfl_sync(0xffffffffu, held, 3);
  const int n_pre = pl.prefix_tiles > 0 ? c1 - c0 + 1 : 0;
  const int n = n_pre + w1 - w0 + 1;
  const long long pre_o = pair ? pl.o2 : pl.o1, pre_l = pair ? pl.l2 : pl.l1;
  auto find = [&](int j) -> long long {  // the first row of candidate j's partials of this request, -1: none
    if (j >= n) return -1;
    const bool pre = j < n_pre;
    const int w = pre ? c0 + j : w0 + j - n_pre;
    const Cut& c = pair && pre ? lines.pairs : lines.singles;
    const int p0 = pre ? pre_p0 : own_p0, tiles = pre ? pl.prefix_tiles : nt;
    if (tile_at(c.at(w), p0, tiles) >= tile_at(c.at(w + 1), p0, tiles)) return -1;
    if (!pre) return (w + static_cast<long long>(b) * a.n_kv + g) * G;
    const long long slot = static_cast<long long>(w) + seg;
    return (pair ? slot * 2 + (tile & 1) : slot) * pl.rows + (b - tile * pl.row_reqs) * G;
  };
  constexpr int kStep = SPLIT ? WARPS : 1;  // this warp's candidates: every kStep-th
  for (int it0 = 0; it0 < items; it0 += kChunk) {
    float M[kItems], den[kItems];
    float4 acc[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      M[k] = -INFINITY;
      den[k] = 0.f;
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int j0 = SPLIT ? warp : 0; j0 < n; j0 += 32 * kStep) {
      const int j = j0 + kStep * lane;
      const long long mine = find(j);
      uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
      const uint32_t pre_mask = __ballot_sync(0xffffffffu, j < n_pre);
#pragma unroll 1
      while (left) {
        float l[2][kItems];
        float4 v[2][kItems];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const bool any = left != 0;
          const int from = any ? __ffs(left) - 1 : 0;
          left &= left - 1;
          const long long row = __shfl_sync(0xffffffffu, mine, from);
          const bool pre = (pre_mask >> from) & 1u;
          const float* const o = ws + (pre ? pre_o : pl.o0) + row * D + 4 * it0;
          const float* const ll = ws + (pre ? pre_l : pl.l0) + row;
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            const int it = it0 + 32 * k + lane;
            l[q][k] = -INFINITY;
            v[q][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (any && it < items) {
              l[q][k] = ll[it / (D / 4)];
              v[q][k] = *reinterpret_cast<const float4*>(o + 4 * (32 * k + lane));
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const float m = fmax3(M[k], l[0][k], l[1][k]);
          const float m_ref = m == -INFINITY ? 0.f : m;
          const float x = exp2f(M[k] - m_ref), y = exp2f(l[0][k] - m_ref), z = exp2f(l[1][k] - m_ref);
          M[k] = m;
          den[k] = fmaf(den[k], x, y + z);
          acc[k].x = fmaf(z, v[1][k].x, fmaf(y, v[0][k].x, acc[k].x * x));
          acc[k].y = fmaf(z, v[1][k].y, fmaf(y, v[0][k].y, acc[k].y * x));
          acc[k].z = fmaf(z, v[1][k].z, fmaf(y, v[0][k].z, acc[k].z * x));
          acc[k].w = fmaf(z, v[1][k].w, fmaf(y, v[0][k].w, acc[k].w * x));
        }
      }
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        red_acc[warp * kChunk + 32 * k + lane] = acc[k];
        red_ml[warp * kChunk + 32 * k + lane] = make_float2(M[k], den[k]);
      }
      __syncthreads();
      if (threadIdx.x < kChunk) {  // thread t merges item t
        M[0] = -INFINITY;
        den[0] = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < WARPS; ++q) M[0] = fmaxf(M[0], red_ml[q * kChunk + threadIdx.x].x);
        const float m_ref = M[0] == -INFINITY ? 0.f : M[0];
#pragma unroll
        for (int q = 0; q < WARPS; ++q) {
          const float2 ml = red_ml[q * kChunk + threadIdx.x];
          const float4 v = red_acc[q * kChunk + threadIdx.x];
          const float x = exp2f(ml.x - m_ref);
          den[0] = fmaf(ml.y, x, den[0]);
          acc[0] = make_float4(fmaf(v.x, x, acc[0].x), fmaf(v.y, x, acc[0].y), fmaf(v.z, x, acc[0].z),
                               fmaf(v.w, x, acc[0].w));
        }
      }
      if (it0 + kChunk < items) __syncthreads();  // the next pass writes there again
    }
#pragma unroll
    for (int k = 0; k < (SPLIT ? 1 : kItems); ++k) {
      const int it = it0 + (SPLIT ? static_cast<int>(threadIdx.x) : 32 * k + lane);
      if (it < items && (!SPLIT || threadIdx.x < kChunk)) {
        const float inv = 1.f / den[k];
        *reinterpret_cast<uint2*>(out + 4LL * it) =
            make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
        if (a.lse != nullptr && it % (D / 4) == 0)
          a.lse[out_row + it / (D / 4)] = (M[k] + log2f(den[k])) * 0.69314718055994530942f;
      }
    }
  }
}

// CTAs at most: the workspace is sized for this many (a GB300 has 152 SMs).
constexpr int kMaxCtas = 160;

PagedTcPlan make_plan(const PagedDecodeArgs& a, int ctas, bool rotate) {
  PagedTcPlan p{};
  const int G = a.n_h / a.n_kv;
  p.ctas = ctas;
  p.group_reqs = G <= 8 ? 8 / G : 1;
  p.req_groups = (G + 7) / 8;
  p.own_groups = p.req_groups <= kGroups ? p.req_groups : 0;
  const long long groups = G <= 8 ? (a.B + p.group_reqs - 1) / p.group_reqs : static_cast<long long>(a.B) * p.req_groups;
  p.prefix_groups = groups <= kGroups ? static_cast<int>(groups) : 0;
  p.own_group = G < 8 ? G : 8;
  p.prefix_group = G < 8 ? G * p.group_reqs : 8;
  p.row_reqs = p.prefix_groups ? a.B : BM / G;
  p.rows = p.row_reqs * G;
  p.lo_reqs = rotate ? a.B : 0;
  const int row_tiles = a.prefix_len > 0 ? (a.B + p.row_reqs - 1) / p.row_reqs : 0;
  p.n_pairs = row_tiles / 2;
  p.odd = row_tiles & 1;
  p.prefix_tiles = static_cast<int>((static_cast<long long>(a.prefix_len) + BN - 1) / BN);
  const long long pieces2 = p.n_pairs ? kMaxCtas + static_cast<long long>(p.n_pairs) * a.n_kv : 0;
  const long long pieces1 = p.odd ? 2 * kMaxCtas + static_cast<long long>(a.n_kv) : 0;
  const long long pieces0 = 2 * kMaxCtas + static_cast<long long>(a.B) * a.n_kv;
  p.o2 = 0;
  p.o1 = p.o2 + pieces2 * 2 * p.rows * a.D_v;
  p.o0 = p.o1 + pieces1 * p.rows * a.D_v;
  p.l2 = p.o0 + pieces0 * G * a.D_v;
  p.l1 = p.l2 + pieces2 * 2 * p.rows;
  p.l0 = p.l1 + pieces1 * p.rows;
  p.sums = p.l0 + pieces0 * G;
  p.q = (p.sums + a.B + 1 + 31) & ~31LL;  // 128-byte aligned
  p.end = p.q + static_cast<long long>(a.B) * a.n_h * a.D_qk;
  return p;
}

// Opt in to the kernel's shared memory and check that the compiled kernel holds enough
// registers per thread for its register split (setmaxnreg.inc would wait forever otherwise).
template <int D>
cudaError_t prepare() {
  static std::atomic<unsigned long long> ready{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, paged_tc_kernel<D>)) != cudaSuccess) return e;
  if (static_cast<long long>(fa.numRegs) * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  ready.fetch_or(bit, std::memory_order_acq_rel);
  return cudaSuccess;
}

// Launches a kernel that may start before the one in front of it has ended.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, bool early,
                         A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch(const PagedDecodeArgs& a, const RopeFreq& rope, const CUtensorMap* maps, const PagedTcPlan& pl,
                   cudaStream_t st, int* launches) {
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess) return e;
  const bool rotate = rope.n_pairs > 0;
  if (rotate) {
    const long long items = static_cast<long long>(a.B) * a.n_h * (D / 16);
    __nv_bfloat16* const q = reinterpret_cast<__nv_bfloat16*>(static_cast<float*>(a.workspace) + pl.q);
    const bool any = (a.max_blocks << a.page_shift) > 1 << 24;
    auto rope_q = any ? paged_rope_q_kernel<D, true> : paged_rope_q_kernel<D, false>;
    rope_q<<<static_cast<unsigned>((items + 255) / 256), 256, 0, st>>>(a, rope, q);
    *launches += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_early(paged_tc_kernel<D>, pl.ctas, kThreads, Cfg<D>::kSmemBytes, st, rotate, a, pl, maps[0], maps[1],
                   maps[2], maps[3]);
  if (e != cudaSuccess) return e;
  *launches += 1;
  const unsigned teams = static_cast<unsigned>(a.B) * a.n_kv;
  // A warp per (b, g) where its rows have one to three pieces (no prefix, and rows enough for the workers) or
  // there are more (b, g) than blocks that run at a time.  Behind a prefix they have dozens of pieces: eight
  // warps while two such blocks per SM hold all, else four (64 requests behind 32768 tokens, 512 (b, g):
  // 58.4 us with four, 60.3 with eight; 8 behind 4096, 64 (b, g): 17.9 and 16.4).
  const bool split = teams < (a.prefix_len > 0 ? 1216u : 152u);
  if (split && teams <= 304)
    e = launch_early(paged_tc_combine_kernel<D, 8, true>, teams, 8 * 32, 0, st, true, a, pl);
  else if (split)
    e = launch_early(paged_tc_combine_kernel<D, 4, true>, teams, 4 * 32, 0, st, true, a, pl);
  else
    e = launch_early(paged_tc_combine_kernel<D, 8, false>, (teams + 7) / 8, 8 * 32, 0, st, true, a, pl);
  *launches += 1;
  return e;
}

}  // namespace

bool decode_paged_tc_supported(const PagedDecodeArgs& a, bool bf16, int rope_offset, int rope_dims, bool rope) {
  const int G = a.n_h / a.n_kv;
  if (!(bf16 && a.D_qk == a.D_v && (a.D_qk == 64 || a.D_qk == 128) && G <= BM &&
        (!rope || (rope_offset == 0 && rope_dims == a.D_qk))))
    return false;
  // the line of tiles in 32-bit points: B * n_kv * keys up to some 3e10 (a table far wider than a cache's pages)
  const PagedTcPlan p = make_plan(a, 1, rope);
  const long long own = ((static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len + BN - 1) / BN;
  const double points = static_cast<double>(a.n_kv) *
                        ((static_cast<double>(p.n_pairs) + p.odd) * (static_cast<double>(p.prefix_tiles) * kTileCost + kPieceCost) +
                         static_cast<double>(a.B) * (static_cast<double>(own) * kTileCost + kPieceCost));
  return points < 2147483647.0;
}

size_t decode_paged_tc_workspace(const PagedDecodeArgs& a) {
  return static_cast<size_t>(make_plan(a, kMaxCtas, true).end) * sizeof(float);
}

cudaError_t launch_decode_paged_tc(const PagedDecodeArgs& a, const RopeFreq& rope, int num_sms, cudaStream_t st,
                                   int* launches) {
  // no more CTAs than the call can have tiles
  const long long own = ((static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len + BN - 1) / BN;
  const bool rotate = rope.n_pairs > 0;
  const PagedTcPlan p = make_plan(a, 1, rotate);
  const long long most = static_cast<long long>(a.n_kv) *
                         (static_cast<long long>(p.n_pairs + p.odd) * p.prefix_tiles + own * a.B);
  long long ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (most < ctas) ctas = most > 0 ? most : 1;
  const PagedTcPlan pl = make_plan(a, static_cast<int>(ctas), rotate);
  // query rows by (dim, head of the group, KV head, request); K and V by (dim, KV head, row in page, page),
  // a page per box (half of a 256-token page)
  const void* q = rotate ? static_cast<const float*>(a.workspace) + pl.q : a.q;
  const unsigned long long hs = static_cast<unsigned long long>(a.D_qk) * 2, page = 1ull << a.page_shift;
  const unsigned long long ks = hs * a.n_kv, vs = static_cast<unsigned long long>(a.v_token_stride) * 2;
  const int G = a.n_h / a.n_kv, box_rows = page < 128 ? static_cast<int>(page) : 128;
  const int g8 = G < 8 ? G : 8;  // heads per group of rows
  const int reqs = a.B + pl.lo_reqs;
  CUtensorMap maps[4];
  // (a head's row of 64 dims is 128 bytes: fetched with its neighbour's, half of the traffic would be wasted)
  const bool wide = a.D_qk == 128;
  const int rows = static_cast<int>(page);
  if (!make_map_box(&maps[0], q, a.D_qk, G, a.n_kv, reqs, hs, hs * G, hs * a.n_h, pl.own_groups ? g8 : G, 1, 1, wide) ||
      !make_map_box(&maps[1], q, a.D_qk, G, a.n_kv, reqs, hs, hs * G, hs * a.n_h, pl.prefix_groups ? g8 : G, 1,
                    pl.prefix_groups ? pl.group_reqs : pl.row_reqs, wide) ||
      !make_map_box(&maps[2], a.k_pages, a.D_qk, a.n_kv, rows, a.n_pages, hs, ks, ks * page, 1, box_rows, 1, wide) ||
      !make_map_box(&maps[3], a.v_pages, a.D_v, a.n_kv, rows, a.n_pages, hs, vs, vs * page, 1, box_rows, 1, wide))
    return cudaErrorInvalidValue;
  return a.D_qk == 64 ? launch<64>(a, rope, maps, pl, st, launches) : launch<128>(a, rope, maps, pl, st, launches);
}

}  // namespace attn
