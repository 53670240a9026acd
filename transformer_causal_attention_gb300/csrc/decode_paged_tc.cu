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
// after request, KV head fastest) - weighted kPairCost : kSingleCost, and the line is
// cut into equal parts, one per CTA (one persistent CTA per SM).  A CTA's single tiles
// are cut once more, into halves for its two workers.  Cuts fall anywhere, also inside
// a request: each (worker, segment) piece writes one normalised partial and its
// log-sum-exp, and the combine kernel merges the pieces of a row.  So the SMs finish
// together whatever the lengths are, without a counter in memory, and partials are few.
// Where a piece's partial goes needs no table either: walking the line, each step to
// the next piece raises the worker's index or the segment's, so their sum numbers the
// pieces.  Only the requests' places on the line come from the lengths: every CTA sums
// them at its start (384 threads), CTA 0 leaves the sums for the combine kernel.
//
// A CTA (384 threads): warps 0 and 2 load K and V tiles by TMA, one box per page and
// 64 dims (a page is part of a tile, the tile, or twice the tile), the lanes of the warp
// issuing one box each and holding the next tile's page indices; warp 1 issues the MMAs;
// warp 3 clears value rows behind a segment's last key, which may hold anything; warps
// 4-7 and 8-11 are the two workers' softmax.  The workers run separate pieces (their
// tiles alternate in the K and V rings), so that one's MMAs and loads fill the other's
// softmax and piece ends; on pair tiles they hold the two row tiles.
// TMEM: S/P of the workers in columns [0, 128) and [128, 256), O behind them.
#include <math.h>

#include <atomic>

#include "kernels.h"

namespace attn {
namespace {

constexpr int BM = 128;  // rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kPairCost = 2, kSingleCost = 1;

// Register split as in prefill_tc.cu: a softmax thread holds a row of 128 scores.
constexpr int kLaunchRegs = 168;
constexpr int kRegsCtl = 152, kRegsSoftmax = 176;
constexpr int kRegsNeeded = 4 * 32 * kRegsCtl + 8 * 32 * kRegsSoftmax;
static_assert(kRegsNeeded <= kThreads * kLaunchRegs, "register split exceeds the launch's pool");

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kBlocks = D / 64;             // 64-dim column blocks of a tile
  static constexpr int kBlockBytes = BM * 128;       // one column block (128 rows x 128 bytes, swizzled)
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kKStages = D == 128 ? 2 : 5;
  static constexpr int kVStages = D == 128 ? 3 : 6;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kVStages * kTileBytes;
  static constexpr int kFreqOff = kBarOff + 512;     // RoPE frequencies, hi then lo words
  static constexpr int kSmemBytes = kFreqOff + D * 4 + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kOCol = 256;             // O of worker w at kOCol + w D
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, true);
};

struct Bars {
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], v_fixed[6];
  uint64_t q_ready[2], s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t fin;
  long long line[2];       // scan results: tiles before a worker's first request, per KV head
  long long warp_sum[kThreads / 32];
  int start_b[2];          // the request in which a worker's single tiles begin
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

}  // namespace

// The cut of a call that does not depend on the lengths, and the layout of its workspace.
struct PagedTcPlan {
  int ctas;
  int n_pairs;      // pairs of 128-row tiles of a KV head's prefix rows
  int odd;          // 1: one more row tile, of rows1 rows
  int rows1;
  int prefix_tiles; // key tiles of the prefix
  // float offsets into the workspace: partial outputs and log-sum-exps of pair pieces [256 rows],
  // single prefix pieces [rows1] and own pieces [G]; then (long long) B + 1 tile counts
  long long o2, o1, o0, l2, l1, l0, sums, end;
};

namespace {

__host__ __device__ __forceinline__ long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// The line of tiles and its cut, once the sum of the requests' own tiles (per KV head) is known.
struct Line {
  long long pair_tiles, single_prefix, total;  // tiles; total in cost units
  __device__ __forceinline__ Line(const PagedTcPlan& p, int n_kv, long long own) {
    pair_tiles = static_cast<long long>(p.n_pairs) * n_kv * p.prefix_tiles;
    single_prefix = static_cast<long long>(p.odd) * n_kv * p.prefix_tiles;
    total = pair_tiles * kPairCost + (single_prefix + own * n_kv) * kSingleCost;
  }
  // The line's tiles that start in [0, x): the first pair / single tile at or behind point x.
  __device__ __forceinline__ long long pair_at(long long x) const {
    return min(ceil_div(x, kPairCost), pair_tiles);
  }
  __device__ __forceinline__ long long single_at(long long x) const {
    return max(0LL, ceil_div(x - pair_tiles * kPairCost, kSingleCost));
  }
  __device__ __forceinline__ long long cut(int c, int ctas) const { return total * c / ctas; }
  // The CTA whose part holds point x.
  __device__ __forceinline__ int cta_of(long long x, int ctas) const {
    return static_cast<int>(ceil_div((x + 1) * ctas, total) - 1);
  }
  // Worker w of CTA c takes single tiles [lo, hi).
  __device__ __forceinline__ void singles(int c, int w, int ctas, long long* lo, long long* hi) const {
    const long long a = single_at(cut(c, ctas)), b = single_at(cut(c + 1, ctas));
    const long long mid = a + (b - a + 1) / 2;
    *lo = w ? mid : a;
    *hi = w ? b : mid;
  }
};

__device__ __forceinline__ int own_tiles(const PagedDecodeArgs& a, int b) {
  const int L = paged_len(a, b);
  return L > a.prefix_len ? (L - a.prefix_len + BN - 1) / BN : 0;
}

// A piece: tiles [t, t_end) of one segment for one worker (or, on pair tiles, both).
enum : int { kPair = 0, kPrefix = 1, kOwn = 2 };
struct Piece {
  int kind, b, g, row0, n_rows;  // own: request b; prefix: rows row0.. of KV head g
  int t, t_end, keys;            // keys of the whole segment: tile t holds min(128, keys - 128 t) of them
  long long slot;
};

// A walk along one worker's part of the line.
struct Walk {
  long long p, p_end;        // pair tiles of the CTA
  long long j, j_end, base;  // single tiles of the worker; base: the first one of request b
  int b, w;
};

template <bool PAIRS>
__device__ __forceinline__ bool next_piece(const PagedDecodeArgs& a, const PagedTcPlan& pl, Walk& w, Piece& u) {
  if (PAIRS) {
    if (w.p >= w.p_end) return false;
    const int seg = static_cast<int>(w.p / pl.prefix_tiles);
    u.kind = kPair;
    u.t = static_cast<int>(w.p - static_cast<long long>(seg) * pl.prefix_tiles);
    u.t_end = static_cast<int>(min(static_cast<long long>(pl.prefix_tiles), u.t + w.p_end - w.p));
    u.g = seg / pl.n_pairs;
    u.row0 = (seg % pl.n_pairs) * 2 * BM + w.w * BM;
    u.n_rows = min(BM, a.B * (a.n_h / a.n_kv) - u.row0);
    u.keys = a.prefix_len;
    u.b = 0;
    u.slot = static_cast<long long>(blockIdx.x) + seg;
    w.p += u.t_end - u.t;
    return true;
  }
  if (w.j >= w.j_end) return false;
  const long long own0 = static_cast<long long>(pl.odd) * a.n_kv * pl.prefix_tiles;
  const int worker = 2 * static_cast<int>(blockIdx.x) + w.w;
  if (w.j < own0) {
    u.kind = kPrefix;
    u.g = static_cast<int>(w.j / pl.prefix_tiles);
    u.t = static_cast<int>(w.j - static_cast<long long>(u.g) * pl.prefix_tiles);
    u.t_end = static_cast<int>(min(static_cast<long long>(pl.prefix_tiles), u.t + w.j_end - w.j));
    u.row0 = pl.n_pairs * 2 * BM;
    u.n_rows = pl.rows1;
    u.keys = a.prefix_len;
    u.b = 0;
    u.slot = static_cast<long long>(worker) + u.g;
  } else {
    int nt = own_tiles(a, w.b);
    while (w.j - own0 - w.base >= static_cast<long long>(nt) * a.n_kv) {
      w.base += static_cast<long long>(nt) * a.n_kv;
      nt = own_tiles(a, ++w.b);
    }
    const long long r = w.j - own0 - w.base;
    u.kind = kOwn;
    u.b = w.b;
    u.g = static_cast<int>(r / nt);
    u.t = static_cast<int>(r - static_cast<long long>(u.g) * nt);
    u.t_end = static_cast<int>(min(static_cast<long long>(nt), u.t + w.j_end - w.j));
    u.row0 = 0;
    u.n_rows = a.n_h / a.n_kv;
    u.keys = paged_len(a, w.b) - a.prefix_len;
    u.slot = static_cast<long long>(worker) + static_cast<long long>(w.b) * a.n_kv + u.g;
  }
  w.j += u.t_end - u.t;
  return true;
}

__device__ __forceinline__ int tile_keys(const Piece& u, int t) { return min(BN, u.keys - t * BN); }

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

// Byte offset of the 16-byte chunk c (dims 8 c ..) of row r of a K-major, 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// One loading warp's view of a stream of tiles: the piece, its tile, and in lane l < pages per
// tile the index of the tile's l-th page (loaded a tile ahead).
template <bool PAIRS>
struct Stream {
  Walk w;
  Piece u;
  int t;
  bool live;
  int id;

  __device__ __forceinline__ void fetch(const PagedDecodeArgs& a, int lane) {
    if (!live) return;
    const int* tbl = u.kind == kOwn ? a.block_table + static_cast<long long>(u.b) * a.max_blocks +
                                          (a.prefix_len >> a.page_shift)
                                    : a.prefix_pages;
    const int key = t * BN + (lane << a.page_shift);
    id = (lane == 0 || (lane << a.page_shift) < BN) && key < u.keys ? tbl[key >> a.page_shift] : -1;
  }
  __device__ __forceinline__ void start(const PagedDecodeArgs& a, const PagedTcPlan& pl, const Walk& walk, int lane) {
    w = walk;
    live = next_piece<PAIRS>(a, pl, w, u);
    t = live ? u.t : 0;
    fetch(a, lane);
  }
  __device__ __forceinline__ void advance(const PagedDecodeArgs& a, const PagedTcPlan& pl, int lane) {
    if (++t == u.t_end) {
      live = next_piece<PAIRS>(a, pl, w, u);
      t = live ? u.t : 0;
    }
    fetch(a, lane);
  }
};

struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ RopeFreq f,
                    const __grid_constant__ PagedTcPlan pl, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOff);
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
      mbar_init(&bars->q_ready[w], 128);
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->p_full[w], 128);
      mbar_init(&bars->o_done[w], 1);
      mbar_init(&bars->o_empty[w], 128);
      bars->line[w] = 0;
      bars->start_b[w] = 0;
    }
    mbar_init(&bars->fin, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }

  // ---- the requests' places on the line: thread i sums the own tiles of requests [i s, (i + 1) s)
  const int strip = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, static_cast<int>(threadIdx.x) * strip), b_hi = min(a.B, b_lo + strip);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += own_tiles(a, b);
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) bars->warp_sum[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long own = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += bars->warp_sum[i];
    own += bars->warp_sum[i];
  }
  const Line line(pl, a.n_kv, own);
  Walk walk[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    walk[w].w = w;
    walk[w].p = line.pair_at(line.cut(blockIdx.x, pl.ctas));
    walk[w].p_end = line.pair_at(line.cut(blockIdx.x + 1, pl.ctas));
    line.singles(blockIdx.x, w, pl.ctas, &walk[w].j, &walk[w].j_end);
    // the thread whose requests hold the worker's first own tile finds it
    const long long first = max(walk[w].j - line.single_prefix, 0LL);
    if (walk[w].j < walk[w].j_end && first >= before * a.n_kv && first < (before + mine) * a.n_kv) {
      long long at = before;
      int b = b_lo;
      for (int nt = own_tiles(a, b); first >= (at + nt) * a.n_kv; nt = own_tiles(a, ++b)) at += nt;
      bars->line[w] = at * a.n_kv;
      bars->start_b[w] = b;
    }
  }
  if (blockIdx.x == 0) {
    long long* const sums = reinterpret_cast<long long*>(static_cast<float*>(a.workspace) + pl.sums);
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      sums[b] = at;
      at += own_tiles(a, b);
    }
    if (threadIdx.x == 0) sums[a.B] = own;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    walk[w].base = bars->line[w];
    walk[w].b = bars->start_b[w];
  }
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort_flag, a.status, a.wait_limit_ns};

  if (warp < 4) {
    setmaxnreg_dec<kRegsCtl>();
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
      Ring r;
      uint32_t issued = 0, last_ph = 0;
      // one tile: lane l loads column block l / boxes of page l mod boxes
      auto load = [&](const Piece& u, int t, int id) -> bool {
        if (!warp_wait(&empty[r.st], r.ph ^ 1, wc)) return false;
        const int n = tile_keys(u, t);
        const int n_boxes = (n + (1 << box_shift) - 1) >> box_shift;  // pages without keys are not loaded
        if (lane == 0) mbar_arrive_expect_tx(&full[r.st], static_cast<uint32_t>(n_boxes * C::kBlocks) << (box_shift + 7));
        __syncwarp();
        const int box = lane & (boxes - 1), blk = lane / boxes;
        const int page = __shfl_sync(0xffffffffu, id, box);
        if (blk < C::kBlocks && box < n_boxes)
          tma_load_4d(ring + r.st * C::kTileBytes + blk * C::kBlockBytes + (box << (box_shift + 7)), map, &full[r.st],
                      blk * 64, u.g, (t * BN) & ((1 << a.page_shift) - 1), page);
        issued |= 1u << r.st;
        last_ph = (last_ph & ~(1u << r.st)) | (r.ph << r.st);
        r.next(n_stages);
        return true;
      };
      bool ok = true;
      {
        Stream<true> s;
        s.start(a, pl, walk[0], lane);
        while (ok && s.live) {
          const Piece u = s.u;
          const int t = s.t, id = s.id;
          s.advance(a, pl, lane);
          ok = load(u, t, id);
        }
      }
      Stream<false> s0, s1;
      s0.start(a, pl, walk[0], lane);
      s1.start(a, pl, walk[1], lane);
      while (ok && (s0.live || s1.live)) {
        if (s0.live) {
          const Piece u = s0.u;
          const int t = s0.t, id = s0.id;
          s0.advance(a, pl, lane);
          ok = load(u, t, id);
        }
        if (ok && s1.live) {
          const Piece u = s1.u;
          const int t = s1.t, id = s1.id;
          s1.advance(a, pl, lane);
          ok = load(u, t, id);
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
        uint32_t pph = 0, qph = 0, oph = 0, fix_ph = 0;  // parities, one bit per worker (fix_ph: per stage)
        auto issue_qk = [&](int w) {
          const uint64_t a0 = q_desc0 + ((w * C::kTileBytes) >> 4);
          const uint64_t b0 = k_desc0 + ((kr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4;
            mma_ss(tmem + w * 128u, a0 + off, b0 + off, C::kIdescQK, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full[w]);
        };
        auto issue_pv = [&](int w, bool accumulate) {
          const uint64_t b0 = v_desc0 + ((vr.st * C::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + C::kOCol + w * D, tmem + w * 128u + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescPV,
                   (accumulate || kk > 0) ? 1u : 0u);
        };
        auto wait_q = [&](int w) -> bool {
          const bool ok = mbar_wait(&bars->q_ready[w], (qph >> w) & 1u, wc);
          qph ^= 1u << w;
          return ok;
        };
        auto wait_k = [&]() -> bool { return mbar_wait(&bars->k_full[kr.st], kr.ph, wc); };
        auto wait_v = [&](int n) -> bool {  // n keys of the tile are real; fewer than 128: the rest is cleared first
          if (!mbar_wait(&bars->v_full[vr.st], vr.ph, wc)) return false;
          if (n == BN) return true;
          const bool ok = mbar_wait(&bars->v_fixed[vr.st], (fix_ph >> vr.st) & 1u, wc);
          fix_ph ^= 1u << vr.st;
          return ok;
        };
        auto wait_p = [&](int w, bool first) -> bool {  // P of the tile, and a free O for a piece's first
          if (!mbar_wait(&bars->p_full[w], (pph >> w) & 1u, wc)) return false;
          pph ^= 1u << w;
          if (first) {
            if (!mbar_wait(&bars->o_empty[w], ((oph >> w) & 1u) ^ 1u, wc)) return false;
            oph ^= 1u << w;
          }
          return true;
        };
        {
          // pair tiles: both workers' rows on each K/V tile
          Walk wk = walk[0];
          Piece u;
          bool live = next_piece<true>(a, pl, wk, u);
          int t = live ? u.t : 0;
          bool first = true;  // t is its piece's first tile
          if (live) {
            if (!wait_k()) goto mma_done;
            for (int w = 0; w < 2; ++w) {
              if (!wait_q(w)) goto mma_done;
              tc_fence_after();
              issue_qk(w);
            }
            mma_commit(&bars->k_empty[kr.st]);
            kr.next(C::kKStages);
          }
          while (live) {
            const bool last = t + 1 == u.t_end;
            const int n = tile_keys(u, t);
            bool more = !last;
            Piece nu = u;
            if (last) more = next_piece<true>(a, pl, wk, nu);
            if (!wait_v(n)) goto mma_done;
            for (int w = 0; w < 2; ++w) {
              if (!wait_p(w, first)) goto mma_done;
              tc_fence_after();
              issue_pv(w, !first);
              if (last) mma_commit(&bars->o_done[w]);
              if (w == 1) {
                mma_commit(&bars->v_empty[vr.st]);
                vr.next(C::kVStages);
              }
              if (more) {
                if (w == 0 && !wait_k()) goto mma_done;
                if (last && !wait_q(w)) goto mma_done;
                tc_fence_after();
                issue_qk(w);
              }
            }
            if (more) {
              mma_commit(&bars->k_empty[kr.st]);
              kr.next(C::kKStages);
            }
            live = more;
            first = last;
            if (last) {
              u = nu;
              t = u.t;
            } else {
              ++t;
            }
          }
        }
        {
          // single tiles: the workers take turns, each P V followed by its next Q K
          Walk w0 = walk[0], w1 = walk[1];
          Piece u0, u1;
          bool live0 = next_piece<false>(a, pl, w0, u0), live1 = next_piece<false>(a, pl, w1, u1);
          int t0 = live0 ? u0.t : 0, t1 = live1 ? u1.t : 0;
          bool first0 = true, first1 = true;
          auto qk_turn = [&](int w, bool new_piece) -> bool {
            if (!wait_k()) return false;
            if (new_piece && !wait_q(w)) return false;
            tc_fence_after();
            issue_qk(w);
            mma_commit(&bars->k_empty[kr.st]);
            kr.next(C::kKStages);
            return true;
          };
          auto turn = [&](int w, Walk& wk, Piece& u, int& t, bool& live, bool& first) -> bool {
            const bool last = t + 1 == u.t_end;
            if (!wait_v(tile_keys(u, t))) return false;
            if (!wait_p(w, first)) return false;
            tc_fence_after();
            issue_pv(w, !first);
            if (last) mma_commit(&bars->o_done[w]);
            mma_commit(&bars->v_empty[vr.st]);
            vr.next(C::kVStages);
            ++t;
            if (last) {
              live = next_piece<false>(a, pl, wk, u);
              t = live ? u.t : 0;
            }
            first = last;
            return !live || qk_turn(w, last);
          };
          if (live0 && !qk_turn(0, true)) goto mma_done;
          if (live1 && !qk_turn(1, true)) goto mma_done;
          while (live0 || live1) {
            if (live0 && !turn(0, w0, u0, t0, live0, first0)) goto mma_done;
            if (live1 && !turn(1, w1, u1, t1, live1, first1)) goto mma_done;
          }
        }
      mma_done:
        // every MMA issued so far completes before TMEM is released
        mma_commit(&bars->fin);
        drain_wait(&bars->fin, 0, a.wait_limit_ns);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ value rows behind a segment's end
      Ring r;
      auto pass = [&](int n) -> bool {
        if (!warp_wait(&bars->v_full[r.st], r.ph, wc)) return false;
        if (n < BN) {
          // rows n.. were not loaded or hold no token: their weights are 0, and 0 times anything must be 0
          uint8_t* const v = smem + C::kVOff + r.st * C::kTileBytes;
          for (int i = lane; i < (BN - n) * 8; i += 32) {
            const int row = n + (i >> 3);
#pragma unroll
            for (int blk = 0; blk < C::kBlocks; ++blk)
              *reinterpret_cast<uint4*>(v + blk * C::kBlockBytes + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->v_fixed[r.st]);
        }
        if (lane == 0) mbar_arrive(&bars->v_empty[r.st]);
        r.next(C::kVStages);
        return true;
      };
      bool ok = true;
      Walk w0 = walk[0], w1 = walk[1];
      Piece u0, u1;
      while (ok && next_piece<true>(a, pl, w0, u0))
        for (int t = u0.t; ok && t < u0.t_end; ++t) ok = pass(tile_keys(u0, t));
      bool live0 = next_piece<false>(a, pl, w0, u0), live1 = next_piece<false>(a, pl, w1, u1);
      int t0 = live0 ? u0.t : 0, t1 = live1 ? u1.t : 0;
      while (ok && (live0 || live1)) {
        if (live0) {
          ok = pass(tile_keys(u0, t0));
          if (++t0 == u0.t_end) {
            live0 = next_piece<false>(a, pl, w0, u0);
            t0 = live0 ? u0.t : 0;
          }
        }
        if (ok && live1) {
          ok = pass(tile_keys(u1, t1));
          if (++t1 == u1.t_end) {
            live1 = next_piece<false>(a, pl, w1, u1);
            t1 = live1 ? u1.t : 0;
          }
        }
      }
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
    uint8_t* const q_smem = smem + C::kQOff + w * C::kTileBytes;
    const int G = a.n_h / a.n_kv;
    float* const ws = static_cast<float*>(a.workspace);
    Walk wk = w ? walk[1] : walk[0];
    uint32_t sph = 0, n_done = 0;

    auto next = [&](Piece& u) -> bool {
      return next_piece<true>(a, pl, wk, u) || next_piece<false>(a, pl, wk, u);
    };
    // The piece's query rows into shared memory, each rotated at its request's last position; the
    // last piece's Q K have completed.  One thread per (row, chunks c and c + D / 16).
    auto prepare_q = [&](const Piece& u) {
      constexpr int kPairsOfChunks = D / 16;
      for (int idx = r; idx < u.n_rows * kPairsOfChunks; idx += 128) {
        const int i = idx / kPairsOfChunks, c = idx % kPairsOfChunks;
        const int b = u.kind == kOwn ? u.b : (u.row0 + i) / G;
        const int h = u.g * G + (u.kind == kOwn ? i : (u.row0 + i) % G);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<long long>(b) * a.n_h + h) * D;
        float x0[8], x1[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(q + c * 8), x0);
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(q + D / 2 + c * 8), x1);
        if (f.n_pairs) {  // the rotated span is the whole head (decode_paged_tc_supported)
          const int pos = max(paged_len(a, b), 1) - 1;
          if (f.half) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float sn, cs;
              rope_sincos_fast(pos, f_hi[c * 8 + e], f_lo[c * 8 + e], &sn, &cs);
              rotate_pair(x0[e], x1[e], sn, cs);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float sn, cs;
              rope_sincos_fast(pos, f_hi[c * 4 + e], f_lo[c * 4 + e], &sn, &cs);
              rotate_pair(x0[2 * e], x0[2 * e + 1], sn, cs);
              rope_sincos_fast(pos, f_hi[D / 4 + c * 4 + e], f_lo[D / 4 + c * 4 + e], &sn, &cs);
              rotate_pair(x1[2 * e], x1[2 * e + 1], sn, cs);
            }
          }
        }
        *reinterpret_cast<uint4*>(q_smem + chunk_off(i, c)) = f32_to_bf16x8(x0);
        *reinterpret_cast<uint4*>(q_smem + chunk_off(i, c + kPairsOfChunks)) = f32_to_bf16x8(x1);
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_ready[w]);
    };

    Piece u;
    bool live = next(u);
    if (live) prepare_q(u);
    while (live) {
      const bool active = quad * 32 < u.n_rows;  // this warp holds rows of the piece
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
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
        const bool seen = m_run != -INFINITY;
        float alpha = 1.f;
        if (need) {
          if (seen) alpha = fast_exp2(m_run - mx);
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
      Piece nu = u;
      const bool more = next(nu);
      if (more) prepare_q(nu);

      // epilogue: the piece's normalised partial and its log-sum-exp
      if (!warp_wait(&bars->o_done[w], n_done & 1, wc)) break;
      ++n_done;
      if (active) {
        tc_fence_after();
        const int rows = u.kind == kPair ? 2 * BM : u.kind == kPrefix ? pl.rows1 : G;
        const long long row = u.slot * rows + (u.kind == kPair ? w * BM : 0) + r;
        float* const po = ws + (u.kind == kPair ? pl.o2 : u.kind == kPrefix ? pl.o1 : pl.o0) + row * D;
        const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orow[32];
          tmem_ld32(o_addr + c * 32, orow);
          tmem_wait_ld();
          if (r < u.n_rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(po + c * 32 + e) =
                  make_float4(__uint_as_float(orow[e]) * inv_l, __uint_as_float(orow[e + 1]) * inv_l,
                              __uint_as_float(orow[e + 2]) * inv_l, __uint_as_float(orow[e + 3]) * inv_l);
          }
        }
        if (r < u.n_rows)
          ws[(u.kind == kPair ? pl.l2 : u.kind == kPrefix ? pl.l1 : pl.l0) + row] = m_run + log2f(l_run);
        tc_fence_before();
      }
      mbar_arrive(&bars->o_empty[w]);
      u = nu;
      live = more;
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
// last; a CTA or worker between them whose part of the line holds no tile wrote none.
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
  const long long* const sums = reinterpret_cast<const long long*>(ws + pl.sums);
  const Line line(pl, a.n_kv, sums[a.B]);
  // the row's segments: [first, last] tile of the prefix (pair or single) and of its own keys
  const long long row = static_cast<long long>(b) * G + i;  // among the KV head's prefix rows
  const bool pair = row < static_cast<long long>(pl.n_pairs) * 2 * BM;
  long long pf = 0, own_f;
  int c0 = 0, n_pre = 0;  // first CTA (pair) or worker (single) of the prefix pieces, and how many to look at
  auto worker_of = [&](long long j) {  // the worker that holds single tile j
    const int c = line.cta_of(line.pair_tiles * kPairCost + j * kSingleCost, pl.ctas);
    long long lo, hi;
    line.singles(c, 1, pl.ctas, &lo, &hi);
    return 2 * c + (j >= lo ? 1 : 0);
  };
  if (pl.prefix_tiles > 0) {
    const long long seg = pair ? static_cast<long long>(g) * pl.n_pairs + row / (2 * BM) : g;
    pf = seg * pl.prefix_tiles;
    const long long pe = pf + pl.prefix_tiles - 1;
    if (pair) {
      c0 = line.cta_of(pf * kPairCost, pl.ctas);
      n_pre = line.cta_of(pe * kPairCost, pl.ctas) - c0 + 1;
    } else {
      c0 = worker_of(pf);
      n_pre = worker_of(pe) - c0 + 1;
    }
  }
  const long long nt = (L - a.prefix_len + BN - 1) / BN;
  own_f = line.single_prefix + sums[b] * a.n_kv + g * nt;
  const int w0 = worker_of(own_f);
  const int n = n_pre + worker_of(own_f + nt - 1) - w0 + 1;

  float M = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += 32) {
    // lane j looks at piece j0 + j: its place in the workspace and its log-sum-exp
    long long at = -1, l_at = 0;
    const int j = j0 + lane;
    if (j < n_pre && pair) {
      const int c = c0 + j;
      const long long lo = line.pair_at(line.cut(c, pl.ctas)), hi = line.pair_at(line.cut(c + 1, pl.ctas));
      if (max(lo, pf) < min(hi, pf + pl.prefix_tiles)) {
        const long long seg = pf / pl.prefix_tiles;
        l_at = (c + seg) * (2 * BM) + row % (2 * BM);
        at = pl.o2 + l_at * D;
        l_at += pl.l2;
      }
    } else if (j < n) {
      const bool pre = j < n_pre;
      const int w = pre ? c0 + j : w0 + j - n_pre;
      const long long f = pre ? pf : own_f, e = f + (pre ? pl.prefix_tiles : nt);
      long long lo, hi;
      line.singles(w >> 1, w & 1, pl.ctas, &lo, &hi);
      if (max(lo, f) < min(hi, e)) {
        l_at = pre ? (static_cast<long long>(w) + g) * pl.rows1 + row - static_cast<long long>(pl.n_pairs) * 2 * BM
                   : (static_cast<long long>(w) + static_cast<long long>(b) * a.n_kv + g) * G + i;
        at = (pre ? pl.o1 : pl.o0) + l_at * D;
        l_at += pre ? pl.l1 : pl.l0;
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
    den = den * alpha + wl;
    acc.x *= alpha;
    acc.y *= alpha;
    acc.z *= alpha;
    acc.w *= alpha;
    const int nj = min(32, n - j0);
#pragma unroll 4
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
  // (den of a lane holds only its own pieces' weights, rescaled alike)
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

// False if the sizes pass what the kernel's indices hold.
PagedTcPlan make_plan(const PagedDecodeArgs& a, int ctas) {
  PagedTcPlan p{};
  const int G = a.n_h / a.n_kv;
  const long long rows = a.prefix_len > 0 ? static_cast<long long>(a.B) * G : 0;
  const int row_tiles = static_cast<int>((rows + BM - 1) / BM);
  p.ctas = ctas;
  p.n_pairs = row_tiles / 2;
  p.odd = row_tiles & 1;
  p.rows1 = p.odd ? static_cast<int>(rows - static_cast<long long>(p.n_pairs) * 2 * BM) : 0;
  p.prefix_tiles = (a.prefix_len + BN - 1) / BN;
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
  p.end = p.sums + 2 * (static_cast<long long>(a.B) + 1);
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
  return bf16 && a.D_qk == a.D_v && (a.D_qk == 64 || a.D_qk == 128) && G <= BM &&
         (!rope || (rope_offset == 0 && rope_dims == a.D_qk));
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
