// decode_paged_tc.cu - single-token decode over a paged KV cache on the tensor cores
// (bf16, D_qk = D_v = 64 or 128), alone or behind a prefix that the batch shares.
//
// Every piece of the work is one product of up to 128 query rows with the keys of
// one KV head in tiles of 128: S = Q K^T, an online softmax over the rows, O += P V
// ("Transformer架构完全深度解析" §13).  Rows are TMEM lanes (one thread per row, no
// exchange between threads), so the same code serves
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
//
// Work split.  All tiles of the call lie on one line - first the pair tiles, KV head by
// KV head, then the single ones (prefix tiles of an odd last row tile, then request
// after request, KV head fastest).  A tile is a few points long (kPairCost, kSingleCost)
// and each segment is led by kPieceCost points for what starting it costs; the line is
// cut into equal parts, one per CTA (one persistent CTA per SM), and the single tiles of
// a CTA's part once more, into halves for its two workers.  Cuts fall anywhere, also
// inside a request: each (worker, segment) piece writes one normalised partial and its
// log-sum-exp, and the combine kernel merges the pieces of a row.  So the SMs finish
// together whatever the lengths are, without a counter in memory, and partials are few.
// Where a piece's partial goes needs no table either: walking the line, each step to
// the next piece raises the worker's index or the segment's, so their sum numbers the
// pieces.
//
// A CTA (384 threads): warp 3 walks the CTA's part of the line (it sums the requests'
// points at its start; CTA 0's leaves the sums for the combine kernel) and hands the
// pieces to the other roles through two small queues in shared memory, a few pieces
// ahead; it also clears value rows behind a segment's last key, which may hold anything.
// Warps 0 and 2 load K and V tiles by TMA, one box per page and 64 dims (a page is part
// of a tile, the tile, or twice the tile), the lanes of the warp issuing one box each;
// warp 1 issues the MMAs; warps 4-7 and 8-11 are the two workers' softmax.  The workers
// run separate pieces (their tiles alternate in the K and V rings), so that one's MMAs
// and loads fill the other's softmax and piece ends; on pair tiles they hold the two
// row tiles.  Every role's code at a piece's boundary is kept small, one copy of each
// part: with the walk inlined into every role a one-tile piece took 7 us, most of it
// instruction fetches.
// TMEM: S/P of the workers in columns [0, 128) and [128, 256), O behind them.
#include <math.h>

#include <atomic>

#include "kernels.h"

namespace attn {

// The cut of a call that does not depend on the lengths, and the layout of its workspace.
struct PagedTcPlan {
  int ctas;
  int n_pairs;       // pairs of 128-row tiles of a KV head's prefix rows
  int odd;           // 1: one more row tile, of rows1 rows
  int rows1;
  int prefix_tiles;  // key tiles of the prefix
  // float offsets into the workspace: partial outputs and log-sum-exps of pair pieces [256 rows],
  // single prefix pieces [rows1] and own pieces [G]; then (int) B + 1 sums of points
  long long o2, o1, o0, l2, l1, l0, sums, end;
};

namespace {

constexpr int BM = 128;  // rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Points on the line: a pair tile, a single tile, the start of a segment.
constexpr int kPairCost = 14, kSingleCost = 8, kPieceCost = 8;

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
  static constexpr int kFreqOff = kBarOff + kBarBytes;  // RoPE frequencies, hi then lo words
  static constexpr int kSmemBytes = kFreqOff + D * 4 + 1024;  // + alignment slack
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
  uint64_t q_ready[2][2];  // per worker, alternating between its pieces: the next one's rows may be ready early
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t piece_full[2][C::kQueue];
  uint64_t fin;
  Piece piece[2][C::kQueue];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars<64>) <= Cfg<64>::kBarBytes && sizeof(Bars<128>) <= Cfg<128>::kBarBytes, "barrier block");

// ------------------------------------------------------------------------------------- the line
// Points are 32-bit: decode_paged_tc_supported bounds the line.
// The first tile of a segment (n tiles of `cost` points each, its first one at point p0) that starts
// at or behind point x.
__device__ __forceinline__ int tile_at(int x, int p0, int cost, int n) {
  const int d = x - p0;
  return d <= 0 ? 0 : min(n, static_cast<int>((static_cast<unsigned>(d) + cost - 1) / static_cast<unsigned>(cost)));
}
__device__ __forceinline__ int seg_points(int tiles, int cost) { return tiles > 0 ? tiles * cost + kPieceCost : 0; }
__device__ __forceinline__ int own_tiles(const PagedDecodeArgs& a, int b) {
  const int L = paged_len(a, b);
  return L > a.prefix_len ? static_cast<int>((static_cast<unsigned>(L - a.prefix_len) + BN - 1) / BN) : 0;
}

// The line and its cut, once the sum of the requests' own points (of one KV head) is known.
struct Line {
  int pair_end, prefix_end, total;  // [0, pair_end) pairs, [.., prefix_end) single prefix tiles, own tiles
  int part, extra, ctas;            // points per CTA, one more for the first `extra` CTAs
  __device__ __forceinline__ Line(const PagedTcPlan& p, int n_kv, int own) {
    pair_end = p.n_pairs * n_kv * seg_points(p.prefix_tiles, kPairCost);
    prefix_end = pair_end + p.odd * n_kv * seg_points(p.prefix_tiles, kSingleCost);
    total = prefix_end + own * n_kv;
    ctas = p.ctas;
    part = static_cast<int>(static_cast<unsigned>(total) / static_cast<unsigned>(ctas));
    extra = total - part * ctas;
  }
  __device__ __forceinline__ int cut(int c) const { return part * c + min(c, extra); }
  // The CTA whose part holds point x.
  __device__ __forceinline__ int cta_of(int x) const {
    const int wide = extra * (part + 1);  // the end of the parts that are one point longer
    const bool in_wide = x < wide;
    const unsigned len = in_wide ? part + 1 : part;  // part > 0 behind `wide`
    return (in_wide ? 0 : extra) + static_cast<int>(static_cast<unsigned>(in_wide ? x : x - wide) / len);
  }
  // Worker w of CTA c takes the single tiles that start in [lo, hi).
  __device__ __forceinline__ void single_part(int c, int w, int* lo, int* hi) const {
    const int a = max(cut(c), pair_end), b = max(cut(c + 1), pair_end);
    const int mid = a + (b - a + 1) / 2;
    *lo = w ? mid : a;
    *hi = w ? b : mid;
  }
  __device__ __forceinline__ int worker_of(int x) const {  // x >= pair_end
    const int c = cta_of(x);
    int lo, hi;
    single_part(c, 1, &lo, &hi);
    return 2 * c + (x >= lo ? 1 : 0);
  }
};

// A walk along one worker's part of the line: the next segment, its first point, its next tile, and
// where the part ends.  Pair pieces come first (in both workers' walks), then single prefix pieces,
// then own ones.
struct Walk {
  int kind, g, b, t, s0, end;                                   // of the pairs, then of the rest
  int rest_kind, rest_g, rest_b, rest_t, rest_s0, rest_end;  // where the single tiles begin
};

// The next piece of a walk; kind kNone at its end.
__device__ __forceinline__ Piece next_piece(const PagedDecodeArgs& a, const PagedTcPlan& pl, Walk& w) {
  Piece u;
  if (w.kind == kPair) {
    const int t_end = tile_at(w.end, w.s0 + kPieceCost, kPairCost, pl.prefix_tiles);
    if (w.g < a.n_kv && w.t < t_end) {
      u = Piece{kPair, w.g, w.b, w.t, t_end, a.prefix_len};
      w.t = t_end;
      if (t_end == pl.prefix_tiles) {
        w.t = 0;
        w.s0 += seg_points(pl.prefix_tiles, kPairCost);
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
  u.kind = kNone;
  for (;;) {
    if (w.kind == kPrefix && w.g == a.n_kv) {  // on to the requests
      w.kind = kOwn;
      w.g = 0;
    }
    if (w.kind == kOwn && w.b >= a.B) return u;
    const int keys = w.kind == kOwn ? paged_len(a, w.b) - a.prefix_len : a.prefix_len;
    if (keys <= 0) {  // an empty place of the batch
      ++w.b;
      continue;
    }
    const int nt = static_cast<int>((static_cast<unsigned>(keys) + BN - 1) / BN);
    const int t_end = tile_at(w.end, w.s0 + kPieceCost, kSingleCost, nt);
    if (w.t >= t_end) {
      if (w.t < nt) return u;  // the part ends here
    } else {
      u = Piece{w.kind, w.g, w.b, w.t, t_end, keys};
      w.t = t_end;
    }
    if (w.t == nt) {
      w.t = 0;
      w.s0 += seg_points(nt, kSingleCost);
      if (++w.g == a.n_kv && w.kind == kOwn) {
        w.g = 0;
        ++w.b;
      }
    }
    if (u.kind != kNone) return u;
  }
}

// Keys of tile t.
__device__ __forceinline__ int tile_keys(const Piece& u, int t) { return min(BN, u.keys - t * BN); }

// ------------------------------------------------------------------------------------- waits
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  const bool ok = mbar_wait(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
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
  __device__ __forceinline__ bool take(Bars<D>* bars, const WaitCtl& wc, bool whole_warp) {
    constexpr uint32_t kQueue = Cfg<D>::kQueue;
    uint64_t* bar = &bars->piece_full[w][n % kQueue];
    const uint32_t par = (n / kQueue) & 1u;
    const bool ok = whole_warp ? warp_wait(bar, par, wc) : mbar_wait(bar, par, wc);
    if (ok) u = bars->piece[w][n % kQueue];
    else u.kind = kNone;
    t = u.t;
    ++n;
    return ok;
  }
  __device__ __forceinline__ bool live() const { return u.kind != kNone; }
};

// ------------------------------------------------------------------------------------- query rows
// Byte offset of the 16-byte chunk c (dims 8 c ..) of row r of a K-major, 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Where a piece's query rows lie in its worker's Q tile: pieces of at most 64 rows alternate between
// the tile's halves, so that the next piece's rows are written while this one's are read (an MMA reads
// 128 rows from either; what lies behind a piece's rows reaches only lanes that nobody reads).
constexpr int kHalfRows = 64;
__device__ __forceinline__ uint32_t next_q_off(int prev_rows, uint32_t prev_off, int rows) {
  return prev_rows <= kHalfRows && rows <= kHalfRows ? prev_off ^ (kHalfRows * 128u) : 0u;
}
// Rows that a piece's Q tile is counted with there (a pair's tiles as full ones).
__device__ __forceinline__ int q_rows(const PagedDecodeArgs& a, const PagedTcPlan& pl, const Piece& u) {
  return u.kind == kPair ? BM : u.kind == kPrefix ? pl.rows1 : a.n_h / a.n_kv;
}

// Query rows row0 .. row0 + n_rows - 1 of KV head g (row r: head r mod G of request r / G) into the
// swizzled tile at dst, rotated at their requests' last positions.  Thread r of 128 copies and
// rotates the chunk pairs (c, c + D / 16) of row i with i D / 16 + c = r mod 128.  One copy of this
// code, out of line, with the frequencies in shared memory.
template <int D>
__device__ __noinline__ void load_q_rows(const PagedDecodeArgs* ap, uint8_t* dst, const float* f_hi, const float* f_lo,
                                         int n_pairs, int half, int g, int row0, int n_rows, int r) {
  constexpr int kCP = D / 16;
  const int G = ap->n_h / ap->n_kv, n_h = ap->n_h;
  const __nv_bfloat16* const q0 = static_cast<const __nv_bfloat16*>(ap->q) + static_cast<long long>(g) * G * D;
  const int n_items = n_rows * kCP;
#pragma unroll 4
  for (int idx = r; idx < n_items; idx += 128) {
    const int i = idx / kCP, c = idx % kCP;
    const int b = (row0 + i) / G, h = row0 + i - b * G;
    const uint4* q = reinterpret_cast<const uint4*>(q0 + (static_cast<long long>(b) * n_h + h) * D) + c;
    const uint4 lo = __ldg(q), hi = __ldg(q + kCP);
    *reinterpret_cast<uint4*>(dst + chunk_off(i, c)) = lo;
    *reinterpret_cast<uint4*>(dst + chunk_off(i, c + kCP)) = hi;
  }
  if (n_pairs) {
#pragma unroll 1
    for (int idx = r; idx < n_items; idx += 128) {
      const int i = idx / kCP, c = idx % kCP;
      const int pos = max(paged_len(*ap, (row0 + i) / G), 1) - 1;
      uint4* const p0 = reinterpret_cast<uint4*>(dst + chunk_off(i, c));
      uint4* const p1 = reinterpret_cast<uint4*>(dst + chunk_off(i, c + kCP));
      float x0[8], x1[8], sn[8], cs[8];
      bf16x8_to_f32(*p0, x0);
      bf16x8_to_f32(*p1, x1);
      // split halves: pair c 8 + e is (x0[e], x1[e]); adjacent: the chunks hold four whole pairs each
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = half ? c * 8 + e : (e < 4 ? c * 4 + e : D / 4 + c * 4 + e - 4);
        rope_sincos_fast(pos, f_hi[j], f_lo[j], &sn[e], &cs[e]);
      }
      if (half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate_pair(x0[e], x1[e], sn[e], cs[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rotate_pair(x0[2 * e], x0[2 * e + 1], sn[e], cs[e]);
          rotate_pair(x1[2 * e], x1[2 * e + 1], sn[4 + e], cs[4 + e]);
        }
      }
      *p0 = f32_to_bf16x8(x0);
      *p1 = f32_to_bf16x8(x1);
    }
  }
  fence_proxy_async_smem();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ RopeFreq f,
                    const __grid_constant__ PagedTcPlan pl, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars<D>* bars = reinterpret_cast<Bars<D>*>(smem + C::kBarOff);
  float* const f_hi = reinterpret_cast<float*>(smem + C::kFreqOff);
  float* const f_lo = f_hi + D / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < f.n_pairs; i += kThreads) {
    f_hi[i] = f.hi[i];
    f_lo[i] = f.lo[i];
  }
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
      mbar_init(&bars->q_ready[w][0], 128);
      mbar_init(&bars->q_ready[w][1], 128);
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->p_full[w], 128);
      mbar_init(&bars->o_done[w], 1);
      mbar_init(&bars->o_empty[w], 128);
      for (int i = 0; i < C::kQueue; ++i) mbar_init(&bars->piece_full[w][i], 1);
    }
    mbar_init(&bars->fin, 1);
    bars->abort_flag = 0;
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
  const WaitCtl wc{&bars->abort_flag, a.status, a.wait_limit_ns};

  if (warp < 4) {
    setmaxnreg_dec<kRegsCtl>();
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
      bool ok = cur.take(bars, wc, true) && oth.take(bars, wc, true);
      id_cur = fetch(cur);
      id_oth = fetch(oth);
      while (ok && (cur.live() || oth.live())) {
        if (cur.live()) {
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
          const bool pair = cur.u.kind == kPair;
          if (++cur.t == cur.u.t_end) {
            ok = cur.take(bars, wc, true);
            if (ok && pair) {  // a pair piece stands in both queues
              ok = oth.take(bars, wc, true);
              id_oth = fetch(oth);
            }
          }
          id_cur = fetch(cur);
          if (pair) continue;  // the first single tile is worker 0's
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
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        const uint64_t q_desc0 = sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024);
        const uint64_t k_desc0 = sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
        const uint64_t v_desc0 = sdesc_sw128(smem_u32(smem + C::kVOff), C::kBlockBytes, 1024);
        Ring kr, vr;
        uint32_t pph = 0, oph = 0, fix_ph = 0;  // parities, one bit per worker (fix_ph: per stage)
        uint32_t n_q0 = 0, n_q1 = 0;            // pieces begun by each worker
        // Q K of worker w's next tile; new_piece: its query rows have to be there first
        auto issue_qk = [&](int w, bool new_piece, uint32_t q_off) -> bool {
          if (new_piece) {
            const uint32_t n = w ? n_q1++ : n_q0++;
            if (!mbar_wait(&bars->q_ready[w][n & 1u], (n >> 1) & 1u, wc)) return false;
          }
          tc_fence_after();
          const uint64_t a0 = q_desc0 + ((w * C::kTileBytes + q_off) >> 4);
          const uint64_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4;
            mma_ss(tmem + w * 128u, a0 + off, b0 + off, C::kIdescQK, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full[w]);
          return true;
        };
        // P V of worker w's tile, once its P is there (and, for a piece's first tile, O is free)
        auto issue_pv = [&](int w, bool first, bool last) -> bool {
          if (!mbar_wait(&bars->p_full[w], (pph >> w) & 1u, wc)) return false;
          pph ^= 1u << w;
          if (first) {
            if (!mbar_wait(&bars->o_empty[w], ((oph >> w) & 1u) ^ 1u, wc)) return false;
            oph ^= 1u << w;
          }
          tc_fence_after();
          const uint64_t b0 = v_desc0 + ((vr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + C::kOCol + w * D, tmem + w * 128u + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescPV,
                   (!first || kk > 0) ? 1u : 0u);
          if (last) mma_commit(&bars->o_done[w]);
          return true;
        };
        auto wait_k = [&]() -> bool { return mbar_wait(&bars->k_full[kr.st], kr.ph, wc); };
        auto done_k = [&]() {
          mma_commit(&bars->k_empty[kr.st]);
          kr.next(C::kKStages);
        };
        auto wait_v = [&](int n) -> bool {  // n keys of the tile are real; fewer than 128: the rest is cleared first
          if (!mbar_wait(&bars->v_full[vr.st], vr.ph, wc)) return false;
          if (n == BN) return true;
          const bool ok = mbar_wait(&bars->v_fixed[vr.st], (fix_ph >> vr.st) & 1u, wc);
          fix_ph ^= 1u << vr.st;
          return ok;
        };
        auto done_v = [&]() {
          mma_commit(&bars->v_empty[vr.st]);
          vr.next(C::kVStages);
        };
        if (!cur.take(bars, wc, false) || !oth.take(bars, wc, false)) goto mma_done;
        if (cur.u.kind == kPair) {
          // pair tiles: both workers' rows on each K/V tile
          if (!wait_k()) goto mma_done;
          for (int w = 0; w < 2; ++w)
            if (!issue_qk(w, true, 0)) goto mma_done;
          done_k();
          bool first = true;  // the tile is its piece's first
          while (cur.u.kind == kPair) {
            const bool last = cur.t + 1 == cur.u.t_end;
            if (!wait_v(tile_keys(cur.u, cur.t))) goto mma_done;
            ++cur.t;
            if (last && (!cur.take(bars, wc, false) || !oth.take(bars, wc, false))) goto mma_done;
            const bool more = cur.u.kind == kPair;
            for (int w = 0; w < 2; ++w) {
              if (!issue_pv(w, first, last)) goto mma_done;
              if (w == 1) done_v();
              if (more) {
                if (w == 0 && !wait_k()) goto mma_done;
                if (!issue_qk(w, last, 0)) goto mma_done;
              }
            }
            if (more) done_k();
            first = last;
          }
        }
        {
          // single tiles: the workers take turns, each P V followed by its next Q K
          bool first_cur = true, first_oth = true;
          uint32_t off_cur = 0, off_oth = 0;  // Q rows of each worker's piece (next_q_off)
          for (int w = 0; w < 2; ++w)
            if ((w ? oth : cur).live()) {
              if (!wait_k() || !issue_qk(w, true, 0)) goto mma_done;
              done_k();
            }
          while (cur.live() || oth.live()) {
            if (cur.live()) {
              const bool last = cur.t + 1 == cur.u.t_end;
              if (!wait_v(tile_keys(cur.u, cur.t))) goto mma_done;
              if (!issue_pv(cur.w, first_cur, last)) goto mma_done;
              done_v();
              ++cur.t;
              if (last) {
                const int rows = q_rows(a, pl, cur.u);
                if (!cur.take(bars, wc, false)) goto mma_done;
                off_cur = next_q_off(rows, off_cur, q_rows(a, pl, cur.u));
              }
              first_cur = last;
              if (cur.live()) {
                if (!wait_k() || !issue_qk(cur.w, last, off_cur)) goto mma_done;
                done_k();
              }
            }
            if (oth.live()) {
              const Cursor<D> x = cur;
              cur = oth;
              oth = x;
              const bool y = first_cur;
              first_cur = first_oth;
              first_oth = y;
              const uint32_t z = off_cur;
              off_cur = off_oth;
              off_oth = z;
            }
          }
        }
      mma_done:
        // every MMA issued so far completes before TMEM is released
        mma_commit(&bars->fin);
        drain_wait(&bars->fin, 0, a.wait_limit_ns);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ the walk, and value rows behind a segment's end
      Walk walk[2];
      {
        // lane i sums the points of requests [i s, (i + 1) s)
        const int strip = (a.B + 31) / 32;
        const int b_lo = min(a.B, lane * strip), b_hi = min(a.B, b_lo + strip);
        int mine = 0;
#pragma unroll 4
        for (int b = b_lo; b < b_hi; ++b) mine += seg_points(own_tiles(a, b), kSingleCost);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        const int own = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
        const Line line(pl, a.n_kv, own);
        const int cta = blockIdx.x;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          Walk k;
          int lo, hi;
          line.single_part(cta, w, &lo, &hi);
          // where the single tiles begin
          k.rest_end = lo < hi ? hi : 0;  // an empty part: no tile starts before point 0
          k.rest_kind = kOwn;
          k.rest_g = k.rest_b = k.rest_t = 0;
          k.rest_s0 = line.prefix_end;
          if (lo < line.prefix_end) {
            const int len = seg_points(pl.prefix_tiles, kSingleCost);
            k.rest_kind = kPrefix;
            k.rest_g = (lo - line.pair_end) / len;
            k.rest_s0 = line.pair_end + k.rest_g * len;
            k.rest_t = tile_at(lo, k.rest_s0 + kPieceCost, kSingleCost, pl.prefix_tiles);
          } else if (lo < hi) {
            // the lane whose requests hold the part's first point finds the tile there
            const int x = lo - line.prefix_end;
            const bool here = x >= before * a.n_kv && x < (before + mine) * a.n_kv;
            if (here) {
              int at = before;
              int b = b_lo;
              int len = seg_points(own_tiles(a, b), kSingleCost);
              while (x >= (at + len) * a.n_kv) {
                at += len;
                len = seg_points(own_tiles(a, ++b), kSingleCost);
              }
              k.rest_b = b;
              k.rest_g = (x - at * a.n_kv) / len;
              k.rest_s0 = line.prefix_end + at * a.n_kv + k.rest_g * len;
              k.rest_t = tile_at(lo, k.rest_s0 + kPieceCost, kSingleCost, own_tiles(a, b));
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            k.rest_b = __shfl_sync(0xffffffffu, k.rest_b, src);
            k.rest_g = __shfl_sync(0xffffffffu, k.rest_g, src);
            k.rest_t = __shfl_sync(0xffffffffu, k.rest_t, src);
            k.rest_s0 = __shfl_sync(0xffffffffu, k.rest_s0, src);
          }
          // and the pairs before them
          const int x0 = line.cut(cta);
          k.kind = kPair;
          k.g = k.b = k.t = 0;
          k.s0 = 0;
          k.end = 0;
          if (x0 < line.pair_end) {
            const int len = seg_points(pl.prefix_tiles, kPairCost);
            const int seg = x0 / len;
            k.end = min(line.cut(cta + 1), line.pair_end);
            k.s0 = seg * len;
            k.t = tile_at(x0, k.s0 + kPieceCost, kPairCost, pl.prefix_tiles);
            k.g = seg / pl.n_pairs;
            k.b = seg - k.g * pl.n_pairs;
            if (k.t == pl.prefix_tiles) {  // behind the segment's last tile
              k.t = 0;
              k.s0 += len;
              if (++k.b == pl.n_pairs) {
                k.b = 0;
                ++k.g;
              }
            }
          }
          walk[w] = k;
        }
        if (cta == 0) {
          int* const sums = static_cast<int*>(a.workspace) + pl.sums;
          int at = before;
          for (int b = b_lo; b < b_hi; ++b) {
            sums[b] = at;
            at += seg_points(own_tiles(a, b), kSingleCost);
          }
          if (lane == 0) sums[a.B] = own;
        }
      }
      uint32_t n_pub[2] = {0, 0}, n_end[2] = {C::kAhead, C::kAhead};  // pieces handed out; and to be, so far
      Ring r;
      bool ok = true, take_cur = true, take_oth = true;
      for (;;) {
        // hand out pieces, kAhead in front of the one this warp is in
        for (;;) {
          const int w = n_pub[0] < n_end[0] ? 0 : 1;
          if (n_pub[w] >= n_end[w]) break;
          const Piece u = next_piece(a, pl, walk[w]);
          if (lane == 0) {
            bars->piece[w][n_pub[w] % C::kQueue] = u;
            mbar_arrive(&bars->piece_full[w][n_pub[w] % C::kQueue]);
          }
          ++n_pub[w];
          if (u.kind == kNone) n_end[w] = 0;  // the last one
        }
        if (take_cur) ok = cur.take(bars, wc, true);
        if (take_oth) ok = ok && oth.take(bars, wc, true);
        take_cur = take_oth = false;
        if (!ok || !(cur.live() || oth.live())) break;
        if (cur.live()) {
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
          const bool pair = cur.u.kind == kPair;
          if (++cur.t == cur.u.t_end) {
            take_cur = true;
            take_oth = pair;
            if (n_end[cur.w]) ++n_end[cur.w];
            if (pair && n_end[oth.w]) ++n_end[oth.w];
          }
          // on pair tiles worker 0 goes on until its first single tile; a finished piece is replaced first
          if (pair) continue;
        }
        if (take_cur ? true : oth.live()) {
          if (!oth.live()) continue;
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
    const int G = a.n_h / a.n_kv;
    uint32_t sph = 0, n_done = 0, n_q = 0, q_off = 0;

    // the first of a piece's rows among its KV head's prefix rows (row r: request r / G), and how many it has
    auto first_row = [&](const Piece& u) {
      return u.kind == kOwn ? u.b * G : (u.kind == kPair ? u.b * 2 * BM + w * BM : pl.n_pairs * 2 * BM);
    };
    auto rows_of = [&](const Piece& u) {
      return u.kind == kOwn ? G : u.kind == kPrefix ? pl.rows1 : min(BM, a.B * G - first_row(u));
    };
    // the query rows of the piece in cur; what the place held before has been read by its Q K
    auto prepare_q = [&]() {
      load_q_rows<D>(&a, smem + C::kQOff + w * C::kTileBytes + q_off, f_hi, f_lo, f.n_pairs, f.half, cur.u.g,
                     first_row(cur.u), rows_of(cur.u), r);
      mbar_arrive(&bars->q_ready[w][n_q & 1u]);
      ++n_q;
    };

    bool ok = cur.take(bars, wc, true);
    bool prepared = false;
    while (ok && cur.live()) {
      // the first piece's rows, or those that could not be written while the piece before ran
      if (!prepared) prepare_q();
      const Piece u = cur.u;
      const int n_rows = rows_of(u);
      const bool active = quad * 32 < n_rows;  // this warp holds rows of the piece
      // the next piece's rows go to the tile's other half while this piece runs, if both fit a half
      if (!cur.take(bars, wc, true)) break;
      prepared = false;
      if (cur.live()) {
        const int p = q_rows(a, pl, u), q = q_rows(a, pl, cur.u);
        q_off = next_q_off(p, q_off, q);
        prepared = p <= kHalfRows && q <= kHalfRows;
        if (prepared) prepare_q();
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int t = u.t; t < u.t_end; ++t) {
        if (!warp_wait(&bars->s_full[w], sph, wc)) { ok = false; break; }
        sph ^= 1;
        if (!active) {  // padding rows: whatever their P is, it reaches only their own O
          mbar_arrive(&bars->p_full[w]);
          continue;
        }
        tc_fence_after();
        uint32_t sr[BN];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_addr + c * 32, sr + c * 32);
        tmem_wait_ld();
        float s[BN];
#pragma unroll
        for (int c = 0; c < BN; ++c) s[c] = __uint_as_float(sr[c]);
        const int n = tile_keys(u, t);
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
                         a.scale_log2;
        // the reference maximum moves only when the row's grew by more than the threshold
        const bool need = mx > m_run + kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          if (m_run != -INFINITY) alpha = fast_exp2(m_run - mx);
          l_run *= alpha;
          m_run = mx;
        }
        uint32_t pr[BN / 2];
        const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
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
        // O rescale before this tile's P V; the P V before has completed (s_full of this tile was
        // committed after it)
        if (__any_sync(0xffffffffu, need && t > u.t)) {
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
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[w]);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      // rows of the next piece that take the whole tile: the Q K of this piece have completed
      if (cur.live() && !prepared) {
        prepare_q();
        prepared = true;
      }

      // epilogue: the piece's normalised partial and its log-sum-exp
      if (!warp_wait(&bars->o_done[w], n_done & 1, wc)) break;
      ++n_done;
      if (active) {
        tc_fence_after();
        float* const ws = static_cast<float*>(a.workspace);
        const long long worker = 2 * static_cast<long long>(blockIdx.x) + w;
        long long row, o_at, l_at;
        if (u.kind == kOwn) {
          row = (worker + static_cast<long long>(u.b) * a.n_kv + u.g) * G;
          o_at = pl.o0;
          l_at = pl.l0;
        } else if (u.kind == kPrefix) {
          row = (worker + u.g) * pl.rows1;
          o_at = pl.o1;
          l_at = pl.l1;
        } else {
          row = (blockIdx.x + static_cast<long long>(u.g) * pl.n_pairs + u.b) * (2 * BM) + w * BM;
          o_at = pl.o2;
          l_at = pl.l2;
        }
        row += r;
        float* const po = ws + o_at + row * D;
        const float inv_l = l_run > 0.f ? 1.f / l_run : l_run;  // 0: every score is -inf; NaN stays
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orow[32];
          tmem_ld32(o_addr + c * 32, orow);
          tmem_wait_ld();
          if (r < n_rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(po + c * 32 + e) =
                  make_float4(__uint_as_float(orow[e]) * inv_l, __uint_as_float(orow[e + 1]) * inv_l,
                              __uint_as_float(orow[e + 2]) * inv_l, __uint_as_float(orow[e + 3]) * inv_l);
          }
        }
        if (r < n_rows) ws[l_at + row] = m_run + log2f(l_run);
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

// One warp per (request b, head h): its row's pieces are those of the CTAs (pair tiles) or workers
// (single tiles) between the one that holds the segment's first tile and the one that holds its
// last; a CTA or worker between them in whose part no tile starts wrote none.
constexpr int kCombineWarps = 4;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    paged_tc_combine_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ PagedTcPlan pl) {
  const int lane = threadIdx.x & 31;
  const long long bh = static_cast<long long>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  if (bh >= static_cast<long long>(a.B) * a.n_h) return;  // whole warps only
  const int b = static_cast<int>(bh / a.n_h), h = static_cast<int>(bh % a.n_h);
  const int G = a.n_h / a.n_kv, g = h / G, i = h % G;
  const int L = paged_len(a, b);
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + bh * D;
  if (L <= a.prefix_len) {  // an empty place of the batch
    if (lane < D / 4) *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(0, 0);
    if (a.lse != nullptr && lane == 0) a.lse[bh] = -INFINITY;
    return;
  }
  const float* const ws = static_cast<const float*>(a.workspace);
  const int* const sums = reinterpret_cast<const int*>(ws + pl.sums);
  const int sum_b = sums[b];
  const Line line(pl, a.n_kv, sums[a.B]);
  // the row's two segments, each from its first tile's point p0: the prefix (pair or single) and its own keys
  const int row = b * G + i;  // among the KV head's prefix rows
  const bool pair = row < pl.n_pairs * 2 * BM;
  const int seg = pair ? g * pl.n_pairs + row / (2 * BM) : g;
  const int pre_cost = pair ? kPairCost : kSingleCost;
  const int pre_p0 = (pair ? 0 : line.pair_end) + kPieceCost + seg * seg_points(pl.prefix_tiles, pre_cost);
  int c0 = 0, n_pre = 0;  // first CTA (pair) or worker (single) of the prefix pieces, and how many to look at
  if (pl.prefix_tiles > 0) {
    const int last = pre_p0 + (pl.prefix_tiles - 1) * pre_cost;
    c0 = pair ? line.cta_of(pre_p0) : line.worker_of(pre_p0);
    n_pre = (pair ? line.cta_of(last) : line.worker_of(last)) - c0 + 1;
  }
  const int nt = own_tiles(a, b);
  const int own_p0 = line.prefix_end + sum_b * a.n_kv + g * seg_points(nt, kSingleCost) + kPieceCost;
  const int w0 = line.worker_of(own_p0);
  const int n = n_pre + line.worker_of(own_p0 + (nt - 1) * kSingleCost) - w0 + 1;

  float M = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += 32) {
    // lane j looks at piece j0 + j: its place in the workspace and its log-sum-exp
    long long at = -1, l_at = 0;
    const int j = j0 + lane;
    if (j < n) {
      const bool pre = j < n_pre;
      const int w = pre ? c0 + j : w0 + j - n_pre;
      int lo, hi;
      if (pre && pair) {
        lo = line.cut(w);
        hi = min(line.cut(w + 1), line.pair_end);
      } else {
        line.single_part(w >> 1, w & 1, &lo, &hi);
      }
      const int p0 = pre ? pre_p0 : own_p0;
      const int cost = pre ? pre_cost : kSingleCost, tiles = pre ? pl.prefix_tiles : nt;
      if (tile_at(lo, p0, cost, tiles) < tile_at(hi, p0, cost, tiles)) {
        if (!pre) {
          l_at = (static_cast<long long>(w) + static_cast<long long>(b) * a.n_kv + g) * G + i;
          at = pl.o0 + l_at * D;
          l_at += pl.l0;
        } else if (pair) {
          l_at = (static_cast<long long>(w) + seg) * (2 * BM) + row % (2 * BM);
          at = pl.o2 + l_at * D;
          l_at += pl.l2;
        } else {
          l_at = (static_cast<long long>(w) + seg) * pl.rows1 + row - pl.n_pairs * 2 * BM;
          at = pl.o1 + l_at * D;
          l_at += pl.l1;
        }
      }
    }
    const float l = at >= 0 ? ws[l_at] : -INFINITY;
    float m = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float m_new = fmaxf(M, m);
    const float m_ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(M - m_ref);
    const float wl = at >= 0 ? exp2f(l - m_ref) : 0.f;
    M = m_new;
    den = den * alpha + wl;  // of this lane's pieces
    acc.x *= alpha;
    acc.y *= alpha;
    acc.z *= alpha;
    acc.w *= alpha;
    const int nj = min(32, n - j0);
#pragma unroll 8
    for (int jj = 0; jj < nj; ++jj) {
      const long long p = __shfl_sync(0xffffffffu, at, jj);
      const float wj = __shfl_sync(0xffffffffu, wl, jj);
      if (p >= 0 && lane < D / 4) {
        const float4 v = *reinterpret_cast<const float4*>(ws + p + 4 * lane);
        acc.x = fmaf(wj, v.x, acc.x);
        acc.y = fmaf(wj, v.y, acc.y);
        acc.z = fmaf(wj, v.z, acc.z);
        acc.w = fmaf(wj, v.w, acc.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  const float inv = 1.f / den;
  if (lane < D / 4)
    *reinterpret_cast<uint2*>(out + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && lane == 0) a.lse[bh] = (M + log2f(den)) * 0.69314718055994530942f;
}

// CTAs at most: the workspace is sized for this many (a GB300 has 152 SMs).
constexpr int kMaxCtas = 160;

PagedTcPlan make_plan(const PagedDecodeArgs& a, int ctas) {
  PagedTcPlan p{};
  const int G = a.n_h / a.n_kv;
  const long long rows = a.prefix_len > 0 ? static_cast<long long>(a.B) * G : 0;
  const int row_tiles = static_cast<int>((rows + BM - 1) / BM);
  p.ctas = ctas;
  p.n_pairs = row_tiles / 2;
  p.odd = row_tiles & 1;
  p.rows1 = p.odd ? static_cast<int>(rows - static_cast<long long>(p.n_pairs) * 2 * BM) : 0;
  p.prefix_tiles = static_cast<int>((static_cast<long long>(a.prefix_len) + BN - 1) / BN);
  const long long pieces2 = p.n_pairs ? kMaxCtas + static_cast<long long>(p.n_pairs) * a.n_kv : 0;
  const long long pieces1 = p.odd ? 2 * kMaxCtas + static_cast<long long>(a.n_kv) : 0;
  const long long pieces0 = 2 * kMaxCtas + static_cast<long long>(a.B) * a.n_kv;
  p.o2 = 0;
  p.o1 = p.o2 + pieces2 * 2 * BM * a.D_v;
  p.o0 = p.o1 + pieces1 * p.rows1 * a.D_v;
  p.l2 = p.o0 + pieces0 * G * a.D_v;
  p.l1 = p.l2 + pieces2 * 2 * BM;
  p.l0 = p.l1 + pieces1 * p.rows1;
  p.sums = (p.l0 + pieces0 * G + 3) & ~3LL;  // 16-byte aligned
  p.end = p.sums + a.B + 1;
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

template <int D>
cudaError_t launch(const PagedDecodeArgs& a, const RopeFreq& rope, const CUtensorMap* maps, const PagedTcPlan& pl,
                   cudaStream_t st, int* launches) {
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess) return e;
  paged_tc_kernel<D><<<pl.ctas, kThreads, Cfg<D>::kSmemBytes, st>>>(a, rope, pl, maps[0], maps[1]);
  *launches += 1;
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long grid = (static_cast<long long>(a.B) * a.n_h + kCombineWarps - 1) / kCombineWarps;
  paged_tc_combine_kernel<D><<<static_cast<unsigned>(grid), kCombineWarps * 32, 0, st>>>(a, pl);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace

bool decode_paged_tc_supported(const PagedDecodeArgs& a, bool bf16, int rope_offset, int rope_dims, bool rope) {
  const int G = a.n_h / a.n_kv;
  if (!(bf16 && a.D_qk == a.D_v && (a.D_qk == 64 || a.D_qk == 128) && G <= BM &&
        (!rope || (rope_offset == 0 && rope_dims == a.D_qk))))
    return false;
  // the line of tiles in 32-bit points: B * n_kv * keys up to some 3e10 (a table far wider than a cache's pages)
  const PagedTcPlan p = make_plan(a, 1);
  const long long own = ((static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len + BN - 1) / BN;
  const double points = static_cast<double>(a.n_kv) *
                        ((static_cast<double>(p.n_pairs) * kPairCost + p.odd * kSingleCost) * p.prefix_tiles +
                         (p.n_pairs + p.odd + static_cast<double>(a.B)) * kPieceCost +
                         static_cast<double>(a.B) * own * kSingleCost);
  return points < 2147483647.0;
}

size_t decode_paged_tc_workspace(const PagedDecodeArgs& a) {
  return static_cast<size_t>(make_plan(a, kMaxCtas).end) * sizeof(float);
}

cudaError_t launch_decode_paged_tc(const PagedDecodeArgs& a, const RopeFreq& rope, const CUtensorMap* maps,
                                   int num_sms, cudaStream_t st, int* launches) {
  // no more CTAs than the call can have tiles
  const long long own = ((static_cast<long long>(a.max_blocks) << a.page_shift) - a.prefix_len + BN - 1) / BN;
  const PagedTcPlan p = make_plan(a, 1);
  const long long most = static_cast<long long>(a.n_kv) *
                         (static_cast<long long>(p.n_pairs + p.odd) * p.prefix_tiles + own * a.B);
  long long ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (most < ctas) ctas = most > 0 ? most : 1;
  const PagedTcPlan pl = make_plan(a, static_cast<int>(ctas));
  return a.D_qk == 64 ? launch<64>(a, rope, maps, pl, st, launches) : launch<128>(a, rope, maps, pl, st, launches);
}

}  // namespace attn
