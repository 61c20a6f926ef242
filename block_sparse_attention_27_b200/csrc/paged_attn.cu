// paged_attn.cu -- dsa_window_attn and dsa_kv4_attn: softmax attention of a block's
// queries over a paged cache, in bf16 with a sliding window and sinks or in 4 bits,
// and over the block's own tokens.
//
//   x_j = q.k_j / sqrt(d) over the visible keys j,  o = sum_j e^(x_j - m) v_j / l,
//   l = sum_j e^(x_j - m),  lse = m + ln l
//
// A unit is up to 128 query rows (token, head of one KV head's group) and their keys in
// tiles of 128: pages that hold a visible token, then block tokens.  The grid is one CTA
// per SM, and each CTA walks through units without stopping between them.  With few
// units, all units' tiles in a row are cut into equal shares, so that sequences of any
// lengths load the SMs alike; a unit that a share's border cuts leaves (O, m, l) of each
// piece in fp32 in the workspace, and paged_merge joins the pieces in order.  With many
// units (kManyUnits per CTA) each CTA takes whole ones.
//
// Warps:
//   0        K tiles (TMA boxes, or 16-byte asynchronous copies for pages under 64
//            tokens: a box costs the TMA unit about 90 ns whatever its size, and 32 boxes
//            of 2 KB per tile held decoding at 3.1 TB/s), the tiles' positions
//   1        TMEM; the MMAs
//   2..9     two softmax groups of 128 threads, a thread per row, alternate tiles
//   10, 11   V tiles; the queries
//   4-bit cache: 0 the queries, 10..12 and 13..15 unpack K and V rows into bf16 tiles
//
//   S = Q K^T (128 x 128) into one of three TMEM buffers, P = 2^(S - m) in bf16 over its
//   first 64 columns, O += P V (TMEM).  S runs two tiles ahead of P.
// A row's reference maximum m is common to the groups (shared memory): the group of tile
// k takes it from the group of tile k - 1 and moves it only when its tile beats it by
// 2^8, so O is rarely rescaled.  Sums, maxima and outputs are held in fp32, P alone in
// bf16: one MMA takes both operands in one type, and V is bf16.
#include <climits>
#include <type_traits>

#include "paged.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kBN = 128;  // keys of a tile
constexpr int kRowsPerTile = 128;
constexpr int kNever = INT_MAX;  // position of a key that takes no part
constexpr float kRescaleLog2 = 8.f;
constexpr int kTabs = 8;        // tiles whose positions are kept: six are in flight at most
constexpr int kMinTiles = 1;    // least tiles of a share
// Whole units above kManyUnits per CTA and above kMaxShared in all; equal shares of all tiles below.
// Shares against whole units, us, 8 KV heads of 4 query heads:
//   one token each over 4-bit prefixes of 1K to 8K: 16 sequences 47, 76; 64: 150, 194; 192: 409,
//     459; 193: 411, 494; 256: 537, 581; 400: 834, 835; all of 4K: 64: 126, 130; 193: 350, 345;
//     400: 710, 705
//   one token each through a window of 4096 over 700 to 8K: 64: 162, 170; 193: 458, 467; 400: 900, 872
//   32 tokens each over 4-bit prefixes of 300 to 4K: 8: 45, 73; 32: 137, 139; 74: 187, 140; 147: 434,
//     371; 193: 562, 514; through a window of 1024: 32: 74, 47; 147: 209, 161; 300: 362, 329
// So shares pay for ragged single tokens until far more units than these limits let through, and
// for blocks only while units are fewer than CTAs, or their lengths differ widely.
constexpr int kManyUnits = 8;
constexpr int kMaxShared = 1536;

// A wait in few instructions (these kernels have many, and code that outgrows the
// instruction cache costs them at every tile): a short spin in place, the bounded wait in
// a function of its own.
__device__ __noinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return mbar_wait(bar, parity, WaitCtx{abort, status});
}
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, const WaitCtx &ctx) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_long(bar, parity, ctx.abort, ctx.status);
}

template <int D, bool KV4>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = KV4 ? 2 : D == 128 ? 3 : 5;
  static constexpr int kThreads = KV4 ? 512 : 384;
  static constexpr uint32_t kHalf = 128u * 128u;           // 128 rows x 128 B
  static constexpr uint32_t kTile = kHalves * kHalf;       // one K or V tile, or Q
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kTile;
  static constexpr uint32_t kOffV = kOffK + kStages * kTile;
  // 4-bit cache: packed tiles on their way in, three each for K and V: codes, then scales
  static constexpr int kRawSlots = 3;
  static constexpr uint32_t kRawCodes = kBN * D / 2;
  static constexpr uint32_t kRaw = kRawCodes + kBN * (D / kKv4Group) * 2;
  static constexpr uint32_t kOffRaw = kOffV + kStages * kTile;
  static constexpr uint32_t kOffBar = kOffRaw + (KV4 ? 2 * kRawSlots * kRaw : 0);
  static constexpr int kNumBars = 4 * kStages + kTabs + 24;
  static constexpr uint32_t kOffTab = kOffBar + kNumBars * 8;      // per tile: 8 positions, flags, end
  static constexpr uint32_t kOffMisc = kOffTab + kTabs * 40;       // TMEM address, abort flag, scan result
  static constexpr uint32_t kOffM = kOffMisc + 32;                 // [128] reference maxima
  static constexpr uint32_t kOffL = kOffM + 512;                   // [128] sums on their way between groups
  static constexpr uint32_t kOffStop = kOffL + 512;                // [3] stops of the walk
  static constexpr uint32_t kAlloc = kOffStop + 3 * 96 + 1024;     // room to align the base to 1 KB
  static constexpr uint32_t kTmemO = 3 * kBN;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kAlloc <= 232448, "shared memory of a CTA");
};

// A piece of a unit in the workspace: which, and whether it holds the unit's first or
// last tile.
struct Piece {
  int unit, begins, ends, pad;
};

struct Params {
  Shape sh;
  PagedArgs a;
  int bpt;        // block tokens of a row tile
  int rowtiles;
  int units;
  int shared_out; // 1: equal shares of all tiles, 0: whole units
  int box_blk;    // block tokens of one TMA box
  Piece *piece;   // [CTA][2]: the unit that the CTA's share enters in its middle, the one it leaves
  float4 *part_o;  // [CTA][2][D/4][rows] x 4 columns
  float2 *part_ml;
};

// What a unit attends to: a list of pages and two ranges of block tokens.
struct Keys {
  int s, h, b0, rows;  // sequence, KV head, first token, query rows
  int n, nb;           // prefix and block tokens
  int nsp, wp0, npg;   // pages: sinks' pages 0..nsp-1, then wp0.. ; npg in all (or idx entries)
  int pt;              // tiles of pages
  int ua, ub0, ub;     // block tokens [0, ua) and [ub0, ub)
  int ta, tiles;       // tiles of the first range; tiles in all
};

// Rows' limits: key position j takes part iff j < end && (j < sk || (lb <= j && j <= hi)).
struct Limits {
  int lb, hi, sk;
};

__device__ __forceinline__ int clamp_int(long long x) {
  return (int)max((long long)-INT_MAX, min((long long)INT_MAX - 1, x));
}

template <bool KV4>
__device__ __forceinline__ Limits row_limits(const PagedArgs &a, int n, int b) {
  if (KV4) return Limits{INT_MIN, INT_MAX - 1, 0};
  const long long p = (long long)n + b;
  return Limits{clamp_int(p - a.window + 1), a.causal ? (int)p : clamp_int(p + a.window - 1),
                a.causal ? (int)min((long long)a.sinks, p + 1) : a.sinks};
}

// Bits j < len whose position base + j (base >= 0) is below x.
__device__ __forceinline__ uint32_t below(int base, int x, uint32_t len) {
  const uint32_t c = x <= base ? 0u : min((uint32_t)x - (uint32_t)base, len);
  return c >= 32 ? 0xffffffffu : (1u << c) - 1u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Whether one key takes part.
__device__ __forceinline__ bool seen(int pos, int end, const Limits &w) {
  return pos < end && (pos < w.sk || (pos >= w.lb && pos <= w.hi));
}
__device__ __forceinline__ uint32_t visible(int base, uint32_t len, int end, const Limits &w) {
  if (base == kNever) return 0u;
  return below(base, end, len) & (below(base, w.sk, len) | (~below(base, w.lb, len) & below(base, w.hi + 1, len)));
}
// Bits j of word w below key k of the tile (0 <= k <= 128).
__device__ __forceinline__ uint32_t first_bits(int k, int w) {
  const int t = min(max(k - 32 * w, 0), 32);
  uint32_t m;
  asm("shl.b32 %0, 0xffffffff, %1;" : "=r"(m) : "r"(t));  // (a shift by 32 leaves 0)
  return ~m;
}
// Visible keys of a tile whose positions are base, base + 1, ...
__device__ __forceinline__ void visible128(int base, int end, const Limits &w, uint32_t (&bits)[4]) {
  auto at = [&](int x) { return x <= base ? 0 : (int)min((uint32_t)x - (uint32_t)base, (uint32_t)kBN); };
  const int ke = at(end), ks = at(w.sk), kl = at(w.lb), kh = at(w.hi + 1);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bits[i] = first_bits(ke, i) & (first_bits(ks, i) | (~first_bits(kl, i) & first_bits(kh, i)));
}
// The same for 32 keys of a tile whose pages start at the table's positions.
template <int PAGE>
__device__ __forceinline__ uint32_t visible32(const int *pos, int word, int end, const Limits &w) {
  if (PAGE == 16)
    return visible(pos[2 * word], 16, end, w) | (visible(pos[2 * word + 1], 16, end, w) << 16);
  const int base = pos[32 * word / PAGE];
  return base == kNever ? 0u : visible(base + 32 * word % PAGE, 32, end, w);
}

template <bool KV4, int PAGE>
__device__ __forceinline__ Keys unit_keys(const Params &prm, int unit, Limits &first, Limits &last, bool report) {
  constexpr int PPT = kBN / PAGE;
  const Shape &sh = prm.sh;
  const PagedArgs &a = prm.a;
  Keys ks;
  const int rt = unit % prm.rowtiles;
  ks.h = unit / prm.rowtiles % sh.Hkv;
  ks.s = unit / prm.rowtiles / sh.Hkv;
  ks.b0 = rt * prm.bpt;
  ks.n = clamp_prefix(a.n_ctx[ks.s], sh.max_pages, PAGE, a.status, report);
  ks.nb = block_tokens(a.n_new, ks.s, sh.B, a.status, report);
  const int b_end = min(ks.b0 + prm.bpt, ks.nb);  // the unit's tokens are [b0, b_end)
  ks.rows = max(0, b_end - ks.b0) * sh.G;
  first = row_limits<KV4>(a, ks.n, ks.b0);
  last = row_limits<KV4>(a, ks.n, max(ks.b0, b_end - 1));
  const int np = (ks.n + PAGE - 1) / PAGE;
  if (KV4) {
    ks.nsp = 0;
    ks.wp0 = 0;
    ks.npg = np;
    if (a.idx) {
      ks.npg = a.idx_cnt[(size_t)ks.s * sh.Hkv + ks.h];
      if (ks.npg < 0 || ks.npg > sh.kmax) {
        if (report) raise_status(a.status, kStatusBadIndex);
        ks.npg = max(0, min(ks.npg, sh.kmax));
      }
    }
    ks.ua = 0;
    ks.ub0 = 0;
    ks.ub = a.blk_k ? ks.nb : 0;
  } else {
    const int lb = max(0, first.lb);  // the lowest position that a window of the unit reaches
    ks.nsp = (min(min(a.sinks, ks.n), lb) + PAGE - 1) / PAGE;
    ks.wp0 = max(ks.nsp, lb / PAGE);
    // (a window that begins at or behind the prefix's end has no page, not the one it may end in)
    ks.npg = ks.nsp + (lb < ks.n ? max(0, np - ks.wp0) : 0);
    const int ue = a.blk_k ? (a.causal ? min(ks.nb, b_end) : ks.nb) : 0;
    ks.ua = max(0, min(ue, clamp_int((long long)last.sk - ks.n)));  // sinks that reach into the block
    ks.ub0 = max(ks.ua, clamp_int((long long)first.lb - ks.n));
    ks.ub = min(ue, clamp_int((long long)last.hi + 1 - ks.n));
    if (ks.ub0 >= ks.ub) ks.ub0 = ks.ub = 0;
  }
  ks.ta = (ks.ua + kBN - 1) / kBN;
  const int tb = ks.ta + (ks.ub - ks.ub0 + kBN - 1) / kBN;
  ks.pt = (ks.npg + PPT - 1) / PPT;
  if (ks.pt + tb == 0) ks.pt = 1;  // rows without a key: one tile without a page
  ks.tiles = ks.rows > 0 ? ks.pt + tb : 0;
  return ks;
}

// One stop of a CTA's walk through its units: tiles [t0, t0 + nt) of a unit.  One thread
// works it out, the others read it in shared memory.
template <bool KV4, int PAGE>
struct Stop {
  Keys ks;
  Limits first, last;
  int unit, t0, nt;  // nt = 0: the walk is over
  __device__ __forceinline__ bool begins() const { return t0 == 0; }
  __device__ __forceinline__ bool ends() const { return t0 + nt == ks.tiles; }

  // Page e of tile t: logical and physical; lp = -1 where the list has ended, phys = -1
  // where the page cannot be read.
  __device__ __forceinline__ void page_at(const Params &prm, int t, int e, int &lp, int &phys) const {
    constexpr int PPT = kBN / PAGE;
    const Shape &sh = prm.sh;
    const int i = t * PPT + e;
    lp = -1;
    phys = -1;
    if (t >= ks.pt || i >= ks.npg) return;
    if (KV4 && prm.a.idx) {
      lp = prm.a.idx[((size_t)ks.s * sh.Hkv + ks.h) * sh.kmax + i];
      if (lp < 0 || (long long)lp * PAGE >= ks.n) lp = -2;
    } else {
      lp = i < ks.nsp ? i : ks.wp0 + (i - ks.nsp);
    }
    if (lp >= 0) phys = (int)physical_page(sh, ks.s, lp);
  }
  // A page whose every token every row sees.
  __device__ __forceinline__ bool page_full(const Params &prm, int lp, int phys) const {
    const int pb = lp * PAGE;
    return phys >= 0 && pb + PAGE <= ks.n && (KV4 || pb + PAGE <= prm.a.sinks || pb >= last.lb);
  }
  // First block token of tile t >= pt, where its range ends (a tile of the first range
  // must not repeat tokens of the second), and whether every row sees all 128.
  __device__ __forceinline__ int blk_tile(int t, int &u_end, bool &full) const {
    const int i = t - ks.pt;
    const bool sink = i < ks.ta;
    const int u0 = sink ? i * kBN : ks.ub0 + (i - ks.ta) * kBN;
    const int p0 = ks.n + u0;
    u_end = sink ? ks.ua : ks.nb;
    full = u0 + kBN <= u_end && (sink ? p0 + kBN <= first.sk : p0 >= last.lb && p0 + kBN - 1 <= first.hi);
    return u0;
  }
  // Writes the table entry of tile t (a whole warp; lane e < PPT holds page e).
  __device__ __forceinline__ void put_table(const Params &prm, int *tab, int t, int lane, int lp, int phys) const {
    constexpr int PPT = kBN / PAGE;
    if (t >= ks.pt) {
      bool full;
      int u_end;
      const int u0 = blk_tile(t, u_end, full);
      if (lane == 0) {
        tab[0] = ks.n + u0;
        tab[8] = (full ? 1 : 0) | 2;
        tab[9] = ks.n + u_end;
      }
    } else {
      if (lane < PPT && lp != -1 && phys < 0) raise_status(prm.a.status, kStatusBadIndex);
      if (lane < PPT) tab[lane] = phys >= 0 ? lp * PAGE : kNever;
      const bool full = __all_sync(0xffffffffu, lane >= PPT || page_full(prm, lp, phys));
      const int lp0 = __shfl_sync(0xffffffffu, lp, 0);
      const bool row = __all_sync(0xffffffffu, lane >= PPT || (phys >= 0 && lp == lp0 + lane));
      if (lane == 0) {
        tab[8] = (full ? 1 : 0) | (row ? 4 : 0);  // 1: every row sees every key; 2: block tokens; 4: positions in a row
        tab[9] = ks.n;
      }
    }
  }
};

// The walk itself: from a share (see cta_share) to its stops.
template <bool KV4, int PAGE>
struct Walk {
  int u, off, left;  // next unit, its first tile, tiles left of the share
  __device__ __forceinline__ explicit Walk(const int *share) : u(share[0]), off(share[1]), left(share[2]) {}
  __device__ __forceinline__ bool next(const Params &prm, Stop<KV4, PAGE> &at) {
    while (u < prm.units && left > 0) {
      at.unit = u;
      at.ks = unit_keys<KV4, PAGE>(prm, u, at.first, at.last, !prm.shared_out);  // (the scan has reported bad lengths)
      at.t0 = off;
      at.nt = min(at.ks.tiles - off, left);
      off = 0;
      if (prm.shared_out) {
        left -= at.nt;
        ++u;
      } else {
        u += gridDim.x;
      }
      if (at.nt > 0) return true;
    }
    at.nt = 0;
    return false;
  }
};

// This CTA's share, by a scan over the units' tiles: share[0..2] = its first unit, the
// first tile of it, its number of tiles.  All threads; ends with a CTA barrier.  `sums`: an
// int per warp.
template <bool KV4, int PAGE, int THREADS>
__device__ __forceinline__ void cta_share(const Params &prm, int *share, int *sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    share[0] = prm.shared_out ? prm.units : (int)blockIdx.x;
    share[1] = 0;
    share[2] = prm.shared_out ? 0 : INT_MAX;
  }
  if (prm.shared_out) {
    const int per = (prm.units + THREADS - 1) / THREADS;  // units of a thread
    const int u0 = threadIdx.x * per, u1 = min(u0 + per, prm.units);
    int mine = 0;
    // two rounds over the thread's units: their sum, then (after the scan) the one that the
    // share begins in
    int at = 0, lo = 0, hi = 0;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      const bool look = round == 0 || (lo >= at && lo < at + mine);
      const int sum0 = mine;
#pragma unroll 1
      for (int u = u0; look && u < u1; ++u) {
        Limits x, y;
        const int n = round == 1 && per == 1 ? sum0 : unit_keys<KV4, PAGE>(prm, u, x, y, blockIdx.x == 0).tiles;
        if (round == 0) {
          mine += n;
        } else {
          if (lo >= at && lo < at + n) {
            share[0] = u;
            share[1] = lo - at;
            share[2] = hi - lo;
          }
          at += n;
        }
      }
      if (round == 1) break;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      before += w < warp ? sums[w] : 0;
      total += sums[w];
    }
    const int shares = max(1, min((int)gridDim.x, total / kMinTiles)), c = blockIdx.x;
    at = before + upto - mine;  // first tile of this thread's units
    lo = c < shares ? (int)((long long)total * c / shares) : INT_MAX;
    hi = c < shares ? (int)((long long)total * (c + 1) / shares) : INT_MAX;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int PAGE, bool KV4>
__global__ void __launch_bounds__(Cfg<D, KV4>::kThreads, 1)
    paged_attn(const __grid_constant__ Params prm, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,  // boxes of a page, or of a tile's pages
               const __grid_constant__ CUtensorMap bkmap, const __grid_constant__ CUtensorMap bvmap) {
  using C = Cfg<D, KV4>;
  constexpr int ST = C::kStages;
  constexpr int PPT = kBN / PAGE;      // pages of a tile
  constexpr bool kBoxes = PAGE >= 64;  // bf16 pages come by TMA
  constexpr uint32_t kLoaders = KV4 ? 96 : 32;  // threads that fill K, and that fill V
  extern __shared__ unsigned char smem_raw[];
  const Shape &sh = prm.sh;
  const PagedArgs &a = prm.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *smem = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + C::kOffBar + 8u * (uint32_t)i; };
  auto k_full = [&](int st) { return bar(st); };
  auto k_empty = [&](int st) { return bar(ST + st); };
  auto v_full = [&](int st) { return bar(2 * ST + st); };
  auto v_empty = [&](int st) { return bar(3 * ST + st); };
  auto tab_full = [&](int k) { return bar(4 * ST + k % kTabs); };
  constexpr int kB0 = 4 * ST + kTabs;
  auto s_full = [&](int k) { return bar(kB0 + k % 3); };
  auto p_full = [&](int k) { return bar(kB0 + 3 + k % 3); };
  auto pv_done = [&](int k) { return bar(kB0 + 6 + (k & 1)); };
  auto decided = [&](int k) { return bar(kB0 + 8 + (k & 1)); };
  const uint32_t q_full = bar(kB0 + 10), q_empty = bar(kB0 + 11), o_full = bar(kB0 + 12), o_free = bar(kB0 + 13);
  // softmax threads among themselves, the loaders of K and of V among themselves (4-bit cache), the last MMA
  const uint32_t meet = bar(kB0 + 14), drain = bar(kB0 + 17);
  auto stop_full = [&](int it) { return bar(kB0 + 18 + it % 3); };
  auto stop_empty = [&](int it) { return bar(kB0 + 21 + it % 3); };
  static_assert(sizeof(Stop<KV4, PAGE>) <= 96, "slot of a stop");
  auto stop_at = [&](int it) { return reinterpret_cast<Stop<KV4, PAGE> *>(smem + C::kOffStop + (it % 3) * 96); };
  auto loaders = [&](bool isv) { return bar(kB0 + 15 + (isv ? 1 : 0)); };
  auto table = [&](int k) { return reinterpret_cast<int *>(smem + C::kOffTab + (k % kTabs) * 40); };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
  int *scan = reinterpret_cast<int *>(smem + C::kOffMisc + 8);  // first unit, its first tile, tiles of the share
  float *m_ref = reinterpret_cast<float *>(smem + C::kOffM), *l_x = reinterpret_cast<float *>(smem + C::kOffL);
  const WaitCtx ctx{abort_flag, a.status};
  volatile int never = 0;
  const WaitCtx drain_ctx{&never, a.status};
  const int aw = (prm.bpt * sh.G + 31) / 32;  // warps of a group that hold rows; the others rest

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int st = 0; st < ST; ++st) {
      mbar_init(k_full(st), kLoaders);
      mbar_init(k_empty(st), 1);
      mbar_init(v_full(st), kLoaders);
      mbar_init(v_empty(st), 1);
    }
#pragma unroll 1
    for (int k = 0; k < kTabs; ++k) mbar_init(tab_full(k), 1);
    for (int k = 0; k < 3; ++k) {
      mbar_init(s_full(k), 1);
      mbar_init(p_full(k), 32 * aw);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(pv_done(k), 1);
      mbar_init(decided(k), 32 * aw);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 64 * aw);
    mbar_init(meet, 64 * aw);
    mbar_init(loaders(false), kLoaders);
    mbar_init(loaders(true), kLoaders);
    mbar_init(drain, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(stop_full(i), 1);
      mbar_init(stop_empty(i), 1 + 2 * aw + 2 * kLoaders / 32);  // the issuer, softmax warps, loaders' warps
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&qmap);
  }
  if (warp == 1) {
    tmem_alloc(base + C::kOffMisc, C::kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();

  cta_share<KV4, PAGE, C::kThreads>(prm, scan, reinterpret_cast<int *>(m_ref));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc);
  // The role's next stop: waits for it, and (done) gives the last one's slot back.  False at
  // the end of the walk, and where a wait gave up.
  auto arrive_at = [&](int it) {
    return mbar_wait_short(stop_full(it), (it / 3) & 1, ctx) && stop_at(it)->nt > 0;
  };
  auto leave = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(stop_empty(it));
  };

  // Parity waits.  A wait names one of a barrier's phases, and must be made when the
  // phase before it has completed and the one after it cannot have.  k counts the CTA's
  // tiles over all its units.
  //   k_full, v_full (k)   the stage's next fill follows k_empty / v_empty of tile k,
  //                        committed after the MMAs that follow the issuer's wait.  Softmax
  //                        threads wait for v_full(k) before P(k), which PV(k) follows.
  //                        The fill before is done: the issuer waited for it, and a softmax
  //                        thread, which has S(k), knows PV(k - 3) done, so V(k - 3) and what
  //                        was before it.  With two stages (4-bit cache) the fill before
  //                        is V(k - 2), which may be missing still: there it waits for
  //                        PV(k - 2) first, which needs nothing of tile k but S(k).
  //   k_empty, v_empty     a stage's next commit needs the fill that follows the wait.
  //   tab_full (k)         slot k's next fill is tile k + 8; its loader has waited for S of
  //                        tile k + 8 - ST, k + 3 at the least, which needs PV(k), so P(k).
  //   s_full, p_full (k)   three of each: S(k + 3) is sent after PV(k), P(k + 3) follows it.
  //   pv_done (k)          two, alternating: the issuer waits for PV(k) before S(k + 3), when
  //                        PVs up to k are out.  A softmax thread waits for PV(k - 1) before
  //                        it decides tile k; PV(k + 1) needs that decision, and PV(k - 3)
  //                        was done before S(k) was sent.
  //   decided (k)          two: the group of tile k + 1 waits for it unless a unit begins
  //                        there; the next one, k + 2, needs the decision on k + 1.  Before
  //                        a unit both groups have met after the last PV, so none is skipped
  //                        that has not completed.
  //   q_full, q_empty, o_full, o_free   once per stop, each after the one before it.
  //   stop_full, stop_empty (it)   three slots: the one of stop it + 3 is written after
  //                        every role has left stop it.  The issuer reads stop it + 2 at most
  //                        while PV of stop it, which others wait for, is still to be sent.
  // No role waits for what follows its own step.  PV(k) is sent after S(k + 2), so with stops of
  // one tile PV of stop it needs K of stop it + 2, and nothing of stop it + 3: that one is
  // written when stop it has been left, which its PV comes before.  So a loader must not hold
  // back a tile while it waits for a stop: copied tiles are announced one tile late, but
  // the last of a stop before the loader waits for the next (a table entry, a tile by TMA or a
  // 4-bit tile is announced in its own step).  Within a stop, K(k - 1) is announced once S(k - ST)
  // is done and V(k - 1) once PV(k - ST) is: both come before the S and PV that need them.
  if (KV4 ? warp == 0 : warp == 11) {
    // ------------------------------------------------- the walk, and queries --
    if (lane == 0) {
      Walk<KV4, PAGE> walk(scan);
      int loaded = 0;
      for (int it = 0;; ++it) {
        if (it >= 3 && !mbar_wait_short(stop_empty(it), ((it / 3) - 1) & 1, ctx)) break;
        Stop<KV4, PAGE> &at = *stop_at(it);
        const bool more = walk.next(prm, at);
        mbar_arrive(stop_full(it));
        if (!more) break;
        if (it > 0 && !mbar_wait_short(q_empty, (it - 1) & 1, ctx)) break;
        mbar_arrive_expect_tx(q_full, (uint32_t)prm.bpt * sh.G * 128u * C::kHalves);
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(base + C::kOffQ + hf * C::kHalf, &qmap, q_full, hf * 64, at.ks.h * sh.G, at.ks.s * sh.B + at.ks.b0);
        loaded = it + 1;
      }
      if (loaded > 0) mbar_wait_short(q_full, (loaded - 1) & 1, drain_ctx);  // a copy in flight lands before the CTA ends
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t q_lo = sdesc_lo(base + C::kOffQ, 16), k_lo = sdesc_lo(base + C::kOffK, 16),
                     v_lo = sdesc_lo(base + C::kOffV, C::kHalf);
      constexpr uint32_t ids = idesc_bf16(128, kBN, false, false);
      constexpr uint32_t ido = idesc_bf16(128, D, false, true);
      // S runs two tiles, so up to two stops, ahead of PV: the tile counts of stops between
      int s_it = 0, s_left = 0, ks = 0, counts[4] = {0, 0, 0, 0};
      bool more = true, ok = true;
      // S of the next tile of the walk, if there is one
      auto issue_s = [&]() {
        if (s_left == 0) {
          if (!more) return true;
          if (!mbar_wait_short(stop_full(s_it), (s_it / 3) & 1, ctx)) return false;
          s_left = stop_at(s_it)->nt;
          mbar_arrive(stop_empty(s_it));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i == (s_it & 3)) counts[i] = s_left;
          more = s_left > 0;
          if (!more) return true;
          if (!mbar_wait_short(q_full, s_it & 1, ctx)) return false;
          ++s_it;
        }
        const int st = ks % ST;
        if (!mbar_wait_short(k_full(st), (ks / ST) & 1, ctx)) return false;
        // P of tile ks - 3 lies in the same columns: its PV must be done
        if (ks >= 3 && !mbar_wait_short(pv_done(ks - 3), ((ks - 3) >> 1) & 1, ctx)) return false;
        tc_fence_after();
        const uint32_t sk = k_lo + st * (C::kTile >> 4), ds = tmem + (ks % 3) * kBN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t step = ((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4;
          umma_bf16_w(ds, q_lo + step, sk + step, hi, ids, kk > 0 ? 1u : 0u);
        }
        umma_commit(s_full(ks));
        umma_commit(k_empty(st));
        ++ks;
        if (--s_left == 0) umma_commit(q_empty);
        return true;
      };
      ok = issue_s() && issue_s();
      int k = 0;
      for (int it = 0; ok; ++it) {
        int nt = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == (it & 3)) nt = counts[i];
        if (it >= s_it || nt == 0) break;
        for (int j = 0; ok && j < nt; ++j, ++k) {
          const int st = k % ST;
          ok = issue_s() && mbar_wait_short(p_full(k), (k / 3) & 1, ctx) && mbar_wait_short(v_full(st), (k / ST) & 1, ctx);
          // the epilogue of the unit before has read O
          if (ok && j == 0 && it > 0) ok = mbar_wait_short(o_free, (it - 1) & 1, ctx);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = v_lo + st * (C::kTile >> 4), pa = tmem + (k % 3) * kBN;
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            umma_bf16_ts_w(tmem + C::kTmemO, pa + kk * 8, sv + kk * (16 * 128 >> 4), hi, ido, (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(pv_done(k));
          umma_commit(v_empty(st));
        }
        if (ok) umma_commit(o_full);
      }
      umma_commit(drain);  // every issued MMA completes before TMEM and the tiles are released
      mbar_wait_short(drain, 0, drain_ctx);
    }
    __syncwarp();
  } else if (warp >= 2 && warp < 10) {
    // ---------------------------------------------------------- softmax groups --
    const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    if (quarter < aw) {
      const uint32_t lt = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t oc = lt + C::kTmemO;
      bool alive = true;
      int k0 = 0, it = 0, met = 0;  // first tile of the unit, units done, meetings
      // all softmax threads; a bounded wait, unlike a named barrier
      auto meet_all = [&]() {
        mbar_arrive(meet);
        alive = __all_sync(0xffffffffu, mbar_wait_short(meet, met & 1, ctx));
        ++met;
        return alive;
      };
      if (prm.shared_out && warp == 2 + ((4 - 2) & 3) && lane == 0) {  // the warp of group 0 with row 0
        prm.piece[2 * blockIdx.x].unit = -1;
        prm.piece[2 * blockIdx.x + 1].unit = -1;
      }
      for (; __all_sync(0xffffffffu, arrive_at(it)); leave(it), ++it) {
        const Stop<KV4, PAGE> &at = *stop_at(it);
        const Keys &ks = at.ks;
        const int rows = ks.rows;
        float m_used = -INFINITY, l = 0.f;
        const int k1 = k0 + at.nt;
        for (int k = k0 + ((k0 ^ g) & 1); k < k1; k += 2) {
          const uint32_t sc = lt + (k % 3) * kBN;
          alive = __all_sync(0xffffffffu, mbar_wait_short(tab_full(k), (k / kTabs) & 1, ctx) && mbar_wait_short(s_full(k), (k / 3) & 1, ctx));
          if (!alive) break;
          tc_fence_after();
          const int *tab = table(k);
          const int flags = tab[8];
          uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
          if (!(flags & 1)) {
            const bool blk = flags & 2;
            const int end = tab[9], st = k % ST;
            const Limits mine = row_limits<KV4>(a, ks.n, ks.b0 + r / sh.G);
            const Limits all{at.first.lb, at.last.hi, at.last.sk};  // keys that some row may see
            if (flags & 6) {  // a block tile, or pages in a row
              visible128(tab[0], end, mine, bits);
            } else {
#pragma unroll 1
              for (int w = 0; w < 4; ++w) {
                const uint32_t b = visible32<PAGE>(tab, w, end, mine);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (i == w) bits[i] = b;
              }
            }
            // Value rows that no row of the unit sees are zeroed: 0 * stale data must not reach O.
            // (In a 4-bit tile of pages they are zeros already.)
            if (!KV4 || blk) {
              // with fewer than three stages V(k - ST) may not be there yet: see v_full above
              if (ST < 3 && k >= ST) alive = __all_sync(0xffffffffu, mbar_wait_short(pv_done(k - ST), ((k - ST) >> 1) & 1, ctx));
              if (alive) alive = __all_sync(0xffffffffu, mbar_wait_short(v_full(st), (k / ST) & 1, ctx));
              if (!alive) break;
#pragma unroll 1
              for (int key = quarter * 32 + lane; key < kBN; key += 32 * aw) {
                const int from = blk ? tab[0] : tab[key / PAGE];
                if (from != kNever && seen(from + (blk ? key : key % PAGE), end, all)) continue;
                unsigned char *row = smem + C::kOffV + st * C::kTile + key * 128;
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
                  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + hf * C::kHalf + c * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
          }
          // The row's scores, all 128 in registers; with the 4-bit cache's warps beside it a
          // thread has 128 registers: it holds the first 64, and reads the others twice.
          constexpr int kHold = KV4 ? 64 : 128;
          uint32_t x[kHold];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if constexpr (KV4) {
            tmem_ld64(sc, x);
          } else {
            tmem_ld64x2(sc, *reinterpret_cast<uint32_t(*)[64]>(&x[0]), sc + 64, *reinterpret_cast<uint32_t(*)[64]>(&x[64]));
          }
          auto hide = [&](uint32_t *y, int w) {  // scores of 32 keys that take no part: -inf
            if (bits[w] == ~0u) return;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((bits[w] >> j) & 1u)) y[j] = 0xff800000u;
          };
#pragma unroll
          for (int w = 0; w < kHold / 32; ++w) hide(x + 32 * w, w);
#pragma unroll
          for (int j = 0; j < kHold; j += 2) mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
          if constexpr (KV4) {
#pragma unroll
            for (int w = 2; w < 4; ++w) {
              uint32_t y[32];
              tmem_ld32(sc + 32 * w, y);
              hide(y, w);
#pragma unroll
              for (int j = 0; j < 32; j += 2) mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
            }
          }
          const float tmax = r < rows ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sh.sl2 : -INFINITY;
          // the reference so far, from the group of the tile before; a row past the unit's keeps none
          float m_prev = -INFINITY;
          if (k > k0) {
            alive = __all_sync(0xffffffffu, mbar_wait_short(decided(k - 1), ((k - 1) >> 1) & 1, ctx));
            if (!alive) break;
            m_prev = m_ref[r];
          }
          const bool need = tmax > m_prev + kRescaleLog2 || (m_prev == -INFINITY && tmax > -INFINITY);
          const float m_now = need ? tmax : m_prev;
          if (k > k0 && __any_sync(0xffffffffu, need)) {  // O holds the unit's earlier tiles
            alive = __all_sync(0xffffffffu, mbar_wait_short(pv_done(k - 1), ((k - 1) >> 1) & 1, ctx));
            if (!alive) break;
            tc_fence_after();
            const float alpha = !need ? 1.f : m_prev == -INFINITY ? 0.f : fast_exp2(m_prev - m_now);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(oc + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(oc + c0, o);
            }
            tc_fence_before();
          }
          if (need || k == k0) m_ref[r] = m_now;
          mbar_arrive(decided(k));
          if (m_now != m_used) {
            l *= m_used == -INFINITY ? 0.f : fast_exp2(m_used - m_now);
            m_used = m_now;
          }
          const float mu = m_used == -INFINITY ? 0.f : m_used;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 scale2 = make_float2(sh.sl2, sh.sl2), mu2 = make_float2(-mu, -mu);
          auto emit = [&](const uint32_t *y, int w) {  // 32 probabilities, over S columns already read
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 e = fma2(make_float2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), scale2, mu2);
              const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              sum[j & 1] = add2(sum[j & 1], p);
              pk[j] = pack_bf16x2(p.x, p.y);
            }
            tmem_st16_async(sc + 16 * w, pk);
          };
#pragma unroll
          for (int w = 0; w < kHold / 32; ++w) emit(x + 32 * w, w);
          if constexpr (KV4) {
            tmem_ld64(sc + 64, x);
#pragma unroll
            for (int w = 2; w < 4; ++w) {
              hide(x + 32 * (w - 2), w);
              emit(x + 32 * (w - 2), w);
            }
          }
          tmem_wait_st();
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tc_fence_before();
          mbar_arrive(p_full(k));
        }
        if (!alive) break;
        // ---- the unit's rows: both groups' sums on the common reference, O from TMEM, a
        //      group per half of the columns
        alive = __all_sync(0xffffffffu, mbar_wait_short(o_full, it & 1, ctx));
        if (!alive) break;
        tc_fence_after();
        // m_ref is final once the last tile is decided (its barrier's next phase is a tile of
        // the next stop, which this thread has not begun)
        alive = __all_sync(0xffffffffu, mbar_wait_short(decided(k1 - 1), ((k1 - 1) >> 1) & 1, ctx));
        if (!alive) break;
        const float M = m_ref[r];
        if (m_used != M) l *= m_used == -INFINITY ? 0.f : fast_exp2(m_used - M);
        if (g == 1) l_x[r] = l;
        if (!meet_all()) break;
        if (g == 0) l_x[r] = l = l + l_x[r];
        if (!meet_all()) break;
        const float L = g == 0 ? l : l_x[r];
        const bool has = L != 0.f;  // a NaN sum counts
        const bool whole = at.begins() && at.ends();
        const int slot = 2 * blockIdx.x + (at.begins() ? 1 : 0);
        const bool mine_row = r < rows;
        const size_t orow = ((size_t)ks.s * sh.B + ks.b0 + r / sh.G) * sh.Hq + (size_t)ks.h * sh.G + r % sh.G;
        const size_t prow = (size_t)slot * ((size_t)prm.bpt * sh.G) + r;
        const float wt = whole ? (has ? 1.f / L : 0.f) : 1.f;
        if (g == 0 && mine_row) {
          if (!whole) {
            prm.part_ml[prow] = make_float2(M, L);
          } else if (sh.lse_out) {
            sh.lse_out[orow] = has ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
          }
        }
        if (!whole && warp == 4 && lane == 0) prm.piece[slot] = Piece{at.unit, at.begins(), at.ends(), 0};
#pragma unroll 1
        for (int i0 = 0; i0 < D / 2; i0 += 32) {
          const int c0 = g * (D / 2) + i0;
          uint32_t o[32];
          tmem_ld32(oc + c0, o);
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = has ? __uint_as_float(o[i]) * wt : 0.f;
          if (mine_row && whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.o_out + orow * D + c0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                  pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
          } else if (mine_row) {
            const int rpt = prm.bpt * sh.G;
            float4 *dst = prm.part_o + ((size_t)slot * (D / 4) + c0 / 4) * rpt + r;  // a warp's rows side by side
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i * rpt] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
          __syncwarp();  // the TMEM loads are warp-collective
        }
        tc_fence_before();
        mbar_arrive(o_free);
        k0 = k1;
      }
    }
  } else if (!KV4) {
    // ------------------------------------------------- bf16 tiles: K or V --
    const bool isv = warp == 10;
    const CUtensorMap *map = isv ? &vmap : &kmap, *bmap = isv ? &bvmap : &bkmap;
    const __nv_bfloat16 *cache = isv ? a.v : a.k;
    auto full = [&](int st) { return isv ? v_full(st) : k_full(st); };
    auto empty = [&](int st) { return isv ? v_empty(st) : k_empty(st); };
    const uint32_t ring = base + (isv ? C::kOffV : C::kOffK);
    int k = 0, told = 0;  // tiles issued; tiles announced (copies by threads are, one tile late)
    bool ok = true;
    auto announce_last = [&]() {
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(full((k - 1) % ST));
      told = k;
    };
    for (int it = 0; ok && __all_sync(0xffffffffu, arrive_at(it)); leave(it), ++it) {
      const Stop<KV4, PAGE> &at = *stop_at(it);
      const Keys &ks = at.ks;
      const int nt = at.nt, t0 = at.t0;
      int lp = -1, phys = -1;
      if (lane < PPT) at.page_at(prm, t0, lane, lp, phys);
      for (int j = 0; j < nt; ++j, ++k) {
        const int st = k % ST, t = t0 + j;
        int lp1 = -1, phys1 = -1;  // the next tile's pages, fetched before this tile's wait
        if (j + 1 < nt && lane < PPT) at.page_at(prm, t + 1, lane, lp1, phys1);
        if (k >= ST) ok = __all_sync(0xffffffffu, mbar_wait_short(empty(st), ((k / ST) - 1) & 1, ctx));
        if (!ok) break;
        if (!isv) {
          at.put_table(prm, table(k), t, lane, lp, phys);
          __syncwarp();
          if (lane == 0) mbar_arrive(tab_full(k));
        }
        const uint32_t dst = ring + st * C::kTile;
        const int p0 = __shfl_sync(0xffffffffu, phys, 0);
        const bool run = !kBoxes && __all_sync(0xffffffffu, lane >= PPT || (phys >= 0 && phys == p0 + lane));
        bool by_tma = t >= ks.pt;
        if (t >= ks.pt) {
          int u_end;
          bool f;
          const int u0 = at.blk_tile(t, u_end, f);
          if (lane == 0) {
            mbar_arrive_expect_tx(full(st), (uint32_t)prm.box_blk * 128u * C::kHalves);
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_3d(dst + hf * C::kHalf, bmap, full(st), hf * 64, ks.h, ks.s * sh.B + u0);
          } else {
            mbar_arrive(full(st));
          }
        } else if (run) {  // the tile's pages lie one after the other: one box per half
          by_tma = true;
          if (lane == 0) {
            mbar_arrive_expect_tx(full(st), C::kTile);
            for (int hf = 0; hf < C::kHalves; ++hf) tma_load_4d(dst + hf * C::kHalf, map, full(st), hf * 64, 0, ks.h, p0);
          } else {
            mbar_arrive(full(st));
          }
        } else if (kBoxes) {
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, lane < PPT && phys >= 0)) * PAGE * 128u * C::kHalves;
          if (lane == 0)
            mbar_arrive_expect_tx(full(st), bytes);
          else
            mbar_arrive(full(st));
          __syncwarp();
          const int e = lane % PPT, hf = lane / PPT;
          const int ph = __shfl_sync(0xffffffffu, phys, e);
          if (hf < C::kHalves && ph >= 0)
            tma_load_2d(dst + hf * C::kHalf + e * PAGE * 128u, map, full(st), hf * 64, (int)(((long long)ph * sh.Hkv + ks.h) * PAGE));
        } else {
          // 16 bytes a lane; D / 8 lanes hold a row
          constexpr int LPR = D / 8;
          const int cr = lane % LPR, row0 = lane / LPR;
          const uint32_t dcol = (cr >> 3) * C::kHalf;
#pragma unroll 1
          for (int e = 0; e < PPT; ++e) {
            const int ph = __shfl_sync(0xffffffffu, phys, e);
            if (ph < 0) continue;
            const __nv_bfloat16 *src = cache + (((long long)ph * sh.Hkv + ks.h) * PAGE + row0) * D + cr * 8;
#pragma unroll
            for (int i = 0; i < PAGE / (32 / LPR); ++i) {
              const int key = e * PAGE + i * (32 / LPR) + row0;
              cp_async16(dst + dcol + sw128_offset(key, cr & 7), src + (long long)i * (32 / LPR) * D);
            }
          }
        }
        if (!kBoxes) {
          cp_async_commit();
          if (k > 0) {  // the tile before has landed: announce it (unless TMA does)
            cp_async_wait<1>();
            if (told < k) {
              fence_proxy_async_smem();
              mbar_arrive(full((k - 1) % ST));
            }
          }
          told = by_tma ? k + 1 : k;  // tiles whose arrivals are made
        }
        lp = lp1;
        phys = phys1;
      }
      // The next stop may not come before the MMAs on this one's last tile: unless it is there,
      // that tile is announced now.
      if (!kBoxes && ok && told < k && !__all_sync(0xffffffffu, mbar_test(stop_full(it + 1), ((it + 1) / 3) & 1))) announce_last();
    }
    if (!kBoxes && told < k) announce_last();
    // copies in flight land before the CTA's shared memory is released
    if (lane == 0)
      for (int j = max(0, k - ST); j < k; ++j) mbar_wait_short(full(j % ST), (j / ST) & 1, drain_ctx);
    __syncwarp();
  } else {
    // ------------------------------------------- 4-bit rows into bf16 tiles --
    // Three warps each for K and V.  Packed tiles come in by 16-byte asynchronous copies, two
    // tiles ahead; a lane then turns 16 bytes (a group of 32 values) at a time into 64 bytes
    // of a swizzled row.  A warp alone on its scheduler waits for most of its instructions:
    // unpacking took 2.7 of 4.1 thousand cycles a tile in two warps.
    const bool isv = warp >= 13;
    const int tid = threadIdx.x - (isv ? 416 : 320);
    constexpr int GR = D / kKv4Group;            // groups of a row
    constexpr int CH = kBN * GR / 64;            // 16-byte copies of each of 64 threads
    const uint8_t *codes = isv ? a.kv4.v : a.kv4.k;
    const __nv_bfloat16 *scales = isv ? a.kv4.vs : a.kv4.ks;
    const CUtensorMap *bmap = isv ? &bvmap : &bkmap;
    auto full = [&](int st) { return isv ? v_full(st) : k_full(st); };
    auto empty = [&](int st) { return isv ? v_empty(st) : k_empty(st); };
    const uint32_t ring = isv ? C::kOffV : C::kOffK;
    const uint32_t rawring = C::kOffRaw + (isv ? C::kRawSlots * C::kRaw : 0);
    int k = 0, gathered = 0;
    bool ok = true;
    auto gather = [&]() {  // the three warps; a bounded wait, unlike a named barrier
      mbar_arrive(loaders(isv));
      ok = __all_sync(0xffffffffu, mbar_wait_short(loaders(isv), gathered & 1, ctx));
      ++gathered;
      return ok;
    };
    for (int it = 0; ok && __all_sync(0xffffffffu, arrive_at(it)); leave(it), ++it) {
      const Stop<KV4, PAGE> &at = *stop_at(it);
      const Keys &ks = at.ks;
      const int nt = at.nt, t0 = at.t0;
      // pages of the tiles j, j + 1, j + 2 of the piece: lane e holds page e
      int lp[3], ph[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        lp[i] = ph[i] = -1;
        if (i < nt && lane < PPT) at.page_at(prm, t0 + i, lane, lp[i], ph[i]);
      }
      // PAGE / 2 of 64 threads bring a page: its codes are consecutive, 16 bytes a thread and step
      auto load = [&](int slot, int phys) {
        const int e = tid / (PAGE / 2), at0 = tid % (PAGE / 2);
        const int p = __shfl_sync(0xffffffffu, phys, e & 31);
        if (tid < 64 && p >= 0) {
          const uint32_t dst = base + rawring + slot * C::kRaw + e * (PAGE * D / 2) + at0 * 16;
          const uint8_t *src = codes + ((long long)p * sh.Hkv + ks.h) * (PAGE * D / 2) + at0 * 16;
#pragma unroll
          for (int i = 0; i < CH; ++i) cp_async16(dst + i * (PAGE / 2) * 16, src + i * (PAGE / 2) * 16);
          if (at0 < PAGE * GR / 8)
            cp_async16(base + rawring + slot * C::kRaw + C::kRawCodes + e * (PAGE * GR * 2) + at0 * 16,
                       scales + ((long long)p * sh.Hkv + ks.h) * (PAGE * GR) + at0 * 8);
        }
        cp_async_commit();
      };
      if (!gather()) break;  // all three warps have read the piece before
      load(k % 3, ph[0]);
      load((k + 1) % 3, ph[1]);
      for (int j = 0; j < nt; ++j, ++k) {
        const int st = k % ST, t = t0 + j;
        const bool blk = t >= ks.pt;
        int lp3 = -1, ph3 = -1;
        if (j + 3 < nt && lane < PPT) at.page_at(prm, t + 3, lane, lp3, ph3);
        cp_async_wait<1>();
        if (!gather()) break;  // everybody's part of tile j is there, and tile j - 1 is read
        load((k + 2) % 3, ph[2]);
        if (k >= ST) ok = __all_sync(0xffffffffu, mbar_wait_short(empty(st), ((k / ST) - 1) & 1, ctx));
        if (!ok) break;
        if (warp == 12) {  // of K's warps the one with a pass less to unpack
          at.put_table(prm, table(k), t, lane, lp[0], ph[0]);
          __syncwarp();
          if (lane == 0) mbar_arrive(tab_full(k));
        }
        if (blk) {
          if (tid == 0) {
            int u_end;
            bool f;
            const int u0 = at.blk_tile(t, u_end, f);
            mbar_arrive_expect_tx(full(st), (uint32_t)prm.box_blk * 128u * C::kHalves);
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_3d(base + ring + st * C::kTile + hf * C::kHalf, bmap, full(st), hf * 64, ks.h, ks.s * sh.B + u0);
          } else {
            mbar_arrive(full(st));
          }
        } else {
          // A warp's pass is 32 groups of 32 / GR keys, one a lane; the swizzle of a lane's row
          // is the same in every pass.  (d = 128: eight lanes are four keys x two groups of one
          // half, so that their stores meet eight different banks of 16 bytes.)
          constexpr int kKeys = 32 / GR, kPasses = kBN / kKeys;
          const int key0 = GR == 4 ? ((lane >> 4) & 1) * 4 + ((lane >> 1) & 3) : lane / GR;
          const int grp = GR == 4 ? ((lane >> 3) & 1) * 2 + (lane & 1) : lane % GR, at0 = key0 * GR + grp;
          const unsigned char *src = smem + rawring + (k % 3) * C::kRaw;
          unsigned char *dst = smem + ring + st * C::kTile + (grp / 2) * C::kHalf;
          const bool whole = __all_sync(0xffffffffu, lane >= PPT || (ph[0] >= 0 && (lp[0] + 1) * PAGE <= ks.n));
          auto unpack = [&](int i, bool on) {
            uint4 w = *reinterpret_cast<const uint4 *>(src + (at0 + 32 * i) * 16);
            const __nv_bfloat16 sc = *reinterpret_cast<const __nv_bfloat16 *>(src + C::kRawCodes + (at0 + 32 * i) * 2);
            __nv_bfloat162 s8, m24;
            kv4_constants(__bfloat162bfloat162(sc), s8, m24);
            if (!on) {  // code 8 with scale 0 is the value 0
              w = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
              s8 = m24 = __float2bfloat162_rn(0.f);
            }
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4 *>(dst + i * kKeys * 128 + sw128_offset(key0, (grp % 2) * 4 + q)) =
                  make_uint4(kv4_pair(ww[q], 0, s8, m24), kv4_pair(ww[q], 1, s8, m24), kv4_pair(ww[q], 2, s8, m24),
                             kv4_pair(ww[q], 3, s8, m24));
          };
          if (whole) {
#pragma unroll 2
            for (int i = tid >> 5; i < kPasses; i += 3) unpack(i, true);
          } else {
#pragma unroll 1
            for (int i = tid >> 5; i < kPasses; i += 3) {
              const int key = key0 + i * kKeys;
              const int p = __shfl_sync(0xffffffffu, ph[0], key / PAGE), q = __shfl_sync(0xffffffffu, lp[0], key / PAGE);
              unpack(i, p >= 0 && q * PAGE + key % PAGE < ks.n);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(full(st));
        }
        lp[0] = lp[1]; ph[0] = ph[1];
        lp[1] = lp[2]; ph[1] = ph[2];
        lp[2] = lp3; ph[2] = ph3;
      }
      cp_async_wait<0>();
    }
    if (tid == 0)  // copies in flight land before the CTA's shared memory is released
      for (int j = max(0, k - ST); j < k; ++j) mbar_wait_short(full(j % ST), (j / ST) & 1, drain_ctx);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------- few rows ----
// Units of at most 16 query rows (decoding) are bound by the cache's bytes: a 128-row MMA
// would idle on them.  Here every warp works alone on 16 keys at a time, which come into its
// own ring in shared memory several steps ahead, with mma.m16n8k16:
//   S^T = K Q^T  (16 keys x 8 rows; the order of the contraction over d is free, so a
//                 lane's K fragments are 16 contiguous bytes)
//   O^T += V^T P^T  (d x 8 rows; the order of d over the M rows is free, so a lane's V
//                 fragments are D/8 contiguous values of four keys, pairs of keys
//                 interleaved by byte permutes, while still packed in the 4-bit cache)
// P goes from the accumulators' layout to the operand's by a transposing 8x8 move.  P is
// taken as the sum of two bf16 numbers (17 bits): the second product is free here.
// A lane owns the maxima and sums of the rows 2t, 2t + 1 of its column.
constexpr int kFewRows = 16;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 keys on their way into fragments.
template <int D>
struct KeysBf16 {
  uint32_t k[2][D / 8], v[4][D / 16];
  // K of keys g, g + 8: chunks t, t + 4, .. of 16 bytes; V of keys 2t, 2t+1, 2t+8, 2t+9: D/8 values
  __device__ __forceinline__ void load_k(const __nv_bfloat16 *row, long long stride, int g, int t, uint32_t on) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if ((on >> (g + 8 * i)) & 1u) x = reinterpret_cast<const uint4 *>(row + (g + 8 * i) * stride)[t + 4 * c];
        k[i][4 * c] = x.x; k[i][4 * c + 1] = x.y; k[i][4 * c + 2] = x.z; k[i][4 * c + 3] = x.w;
      }
  }
  __device__ __forceinline__ void load_v(const __nv_bfloat16 *row, long long stride, int g, int t, uint32_t on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * t + (i & 1) + 4 * (i & 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if ((on >> key) & 1u) x = reinterpret_cast<const uint4 *>(row + key * stride + (D / 8) * g)[c];
        v[i][4 * c] = x.x; v[i][4 * c + 1] = x.y; v[i][4 * c + 2] = x.z; v[i][4 * c + 3] = x.w;
      }
    }
  }
  // first element of the four of a lane in step j of the contraction
  static __device__ __forceinline__ int k_at(int t, int j) { return (t + 4 * (j >> 1)) * 8 + 4 * (j & 1); }
  __device__ __forceinline__ void k_frag(int j, uint32_t (&a)[4]) const {
    a[0] = k[0][2 * j]; a[1] = k[1][2 * j]; a[2] = k[0][2 * j + 1]; a[3] = k[1][2 * j + 1];
  }
  __device__ __forceinline__ void v_frag(int i, uint32_t (&a)[4]) const {
    a[0] = __byte_perm(v[0][i], v[1][i], 0x5410);
    a[1] = __byte_perm(v[0][i], v[1][i], 0x7632);
    a[2] = __byte_perm(v[2][i], v[3][i], 0x5410);
    a[3] = __byte_perm(v[2][i], v[3][i], 0x7632);
  }
};
// The same fragments out of a warp's ring in shared memory.  A slot holds 16 keys: K rows,
// then V rows, of a bf16 cache in 16-byte chunks whose places are permuted by row so that
// the lanes' 16-byte reads spread over the banks.
template <int D>
struct RingBf16 {
  static constexpr int kRow = 2 * D, kSide = 16 * kRow, kSlot = 2 * kSide;
  static constexpr int kChunks = D / 8;  // of a row
  static __device__ __forceinline__ int k_place(int key, int c) { return key * kRow + ((c ^ ((key & 1) << 2)) << 4); }
  static __device__ __forceinline__ int v_place(int key, int c) {
    return key * kRow + ((c ^ ((key & 2) << 1) ^ ((key & 4) >> 2)) << 4);
  }
  static __device__ __forceinline__ void fetch(uint32_t dst, const PagedArgs &a, long long row, int lane) {
#pragma unroll
    for (int i = 0; i < 16 * kChunks / 32; ++i) {
      const int e = lane + 32 * i, key = e / kChunks, c = e % kChunks;
      cp_async16(dst + k_place(key, c), a.k + (row + key) * D + 8 * c);
      cp_async16(dst + kSide + v_place(key, c), a.v + (row + key) * D + 8 * c);
    }
  }
  static __device__ __forceinline__ int k_at(int t, int j) { return KeysBf16<D>::k_at(t, j); }
  const unsigned char *at;
  int g, t;
  uint4 w[2];
  __device__ __forceinline__ void k_begin() {}
  __device__ __forceinline__ void k_frag(int j, uint32_t (&a)[4]) {
    if ((j & 1) == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = *reinterpret_cast<const uint4 *>(at + k_place(g + 8 * i, t + 2 * j));
    }
    if ((j & 1) == 0) {
      a[0] = w[0].x; a[1] = w[1].x; a[2] = w[0].y; a[3] = w[1].y;
    } else {
      a[0] = w[0].z; a[1] = w[1].z; a[2] = w[0].w; a[3] = w[1].w;
    }
  }
  uint4 v[4];
  uint32_t on;
  __device__ __forceinline__ void v_begin(uint32_t on_) { on = on_; }
  __device__ __forceinline__ void v_frag(int i, uint32_t (&a)[4]) {
    if ((i & 3) == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int key = 2 * t + (q & 1) + 4 * (q & 2);
        v[q] = *reinterpret_cast<const uint4 *>(at + kSide + v_place(key, (D / 64) * g + (i >> 2)));
        if (!((on >> key) & 1u)) v[q] = make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = (i & 3) == 0 ? v[q].x : (i & 3) == 1 ? v[q].y : (i & 3) == 2 ? v[q].z : v[q].w;
    a[0] = __byte_perm(x[0], x[1], 0x5410);
    a[1] = __byte_perm(x[0], x[1], 0x7632);
    a[2] = __byte_perm(x[2], x[3], 0x5410);
    a[3] = __byte_perm(x[2], x[3], 0x7632);
  }
};
template <int D>
struct RingKv4 {
  static constexpr int GR = D / kKv4Group;
  static constexpr int kCodes = 16 * D / 2, kScales = 16 * GR * 2;  // bytes of a side
  static constexpr int kSide = kCodes + kScales, kSlot = 2 * kSide;
  static __device__ __forceinline__ void fetch(uint32_t dst, const PagedArgs &a, long long row, int lane) {
#pragma unroll
    for (int i = 0; i < kCodes / 512; ++i) {
      const int e = 16 * (lane + 32 * i);
      cp_async16(dst + e, a.kv4.k + row * (D / 2) + e);
      cp_async16(dst + kSide + e, a.kv4.v + row * (D / 2) + e);
    }
    const int side = lane >> 4, e = 16 * (lane & 15);
    if (e < kScales)
      cp_async16(dst + side * kSide + kCodes + e, reinterpret_cast<const unsigned char *>((side ? a.kv4.vs : a.kv4.ks) + row * GR) + e);
  }
  static __device__ __forceinline__ int k_at(int t, int j) { return (D / 4) * t + 4 * j; }
  const unsigned char *at;
  int g, t;
  uint32_t k[2][D / 32], v[4][D / 64];
  __nv_bfloat162 s8[2], m24[2];
  static __device__ __forceinline__ uint32_t scale(const unsigned char *p) { return *reinterpret_cast<const uint16_t *>(p); }
  __device__ __forceinline__ void constants(int i, uint32_t lo, uint32_t hi) {
    const uint32_t x = lo | (hi << 16);
    kv4_constants(*reinterpret_cast<const __nv_bfloat162 *>(&x), s8[i], m24[i]);
  }
  __device__ __forceinline__ void k_begin() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = g + 8 * i;
      const unsigned char *p = at + key * (D / 2) + t * (D / 8);
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        k[i][0] = x.x; k[i][1] = x.y; k[i][2] = x.z; k[i][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        k[i][0] = x.x; k[i][1] = x.y;
      }
      const uint32_t sc = scale(at + kCodes + 2 * (key * GR + t * (D / 4) / kKv4Group));
      constants(i, sc, sc);
    }
  }
  __device__ __forceinline__ void k_frag(int j, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = kv4_pair(k[i][j >> 1], 2 * (j & 1), s8[i], m24[i]);
      a[i + 2] = kv4_pair(k[i][j >> 1], 2 * (j & 1) + 1, s8[i], m24[i]);
    }
  }
  __device__ __forceinline__ void v_begin(uint32_t on) {
    uint32_t sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * t + (i & 1) + 4 * (i & 2);
      const unsigned char *p = at + kSide + key * (D / 2) + g * (D / 16);
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        v[i][0] = x.x; v[i][1] = x.y;
      } else {
        v[i][0] = *reinterpret_cast<const uint32_t *>(p);
      }
      sc[i] = scale(at + kSide + kCodes + 2 * (key * GR + g * (D / 8) / kKv4Group));
      if (!((on >> key) & 1u)) {  // code 8 with scale 0 is the value 0
        sc[i] = 0;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) v[i][w] = 0x88888888u;
      }
    }
    constants(0, sc[0], sc[1]);
    constants(1, sc[2], sc[3]);
  }
  __device__ __forceinline__ void v_frag(int i, uint32_t (&a)[4]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t x = v[2 * p][i >> 2], y = v[2 * p + 1][i >> 2];
      a[2 * p] = kv4_pair(__byte_perm(x, y, 0x5410), i & 3, s8[p], m24[p]);
      a[2 * p + 1] = kv4_pair(__byte_perm(x, y, 0x7632), i & 3, s8[p], m24[p]);
    }
  }
};

// O^T and the statistics of a warp's keys, for 8 * NT rows.
template <int D, int NT>
struct FewState {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];  // rows 8 n + 2t, 8 n + 2t + 1; l of this lane's keys
};

// One step: 16 keys of fragments `f`; `hid` bit 4 n + 2 i + e: key g + 8 i is hidden from row 8 n + 2t + e.
template <int D, int NT, class F>
__device__ __forceinline__ void few_scores(F &f, const uint2 *qf, int lane, float (&x)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
  f.k_begin();
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    uint32_t a[4];
    f.k_frag(j, a);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 b = qf[(n * (D / 16) + j) * 32 + lane];
      mma_bf16(x[n], a[0], a[1], a[2], a[3], b.x, b.y);
    }
  }
}
template <int D, int NT>
__device__ __forceinline__ void few_softmax(FewState<D, NT> &st, float (&x)[NT][4], uint32_t hid, float sl2,
                                            uint32_t (&ph)[NT][2], uint32_t (&pl)[NT][2]) {
  bool need = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[n][e] = (hid >> (4 * n + e)) & 1u ? -INFINITY : x[n][e] * sl2;
      need |= x[n][e] > st.m[n][e & 1] + kRescaleLog2 || (st.m[n][e & 1] == -INFINITY && x[n][e] > -INFINITY);
    }
  if (__any_sync(0xffffffffu, need)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = fmaxf(x[n][e], x[n][e + 2]);
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        const float mn = fmaxf(st.m[n][e], t);
        const float al = st.m[n][e] == -INFINITY ? 0.f : st.m[n][e] == mn ? 1.f : fast_exp2(st.m[n][e] - mn);
        st.m[n][e] = mn;
        st.l[n][e] *= al;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[n][i][e] *= al;
          st.o[n][i][e + 2] *= al;
        }
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float p[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float mu = st.m[n][e & 1] == -INFINITY ? 0.f : st.m[n][e & 1];
      p[e] = fast_exp2(x[n][e] - mu);
      st.l[n][e & 1] += p[e];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ph[n][i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
      const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ph[n][i]));
      q[2 * i] = p[2 * i] - hi.x;
      q[2 * i + 1] = p[2 * i + 1] - hi.y;
      pl[n][i] = transpose8(pack_bf16x2(q[2 * i], q[2 * i + 1]));
      ph[n][i] = transpose8(ph[n][i]);
    }
  }
}
template <int D, int NT, class F>
__device__ __forceinline__ void few_values(F &f, FewState<D, NT> &st, const uint32_t (&ph)[NT][2], const uint32_t (&pl)[NT][2]) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t a[4];
    f.v_frag(i, a);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma_bf16(st.o[n][i], a[0], a[1], a[2], a[3], ph[n][0], ph[n][1]);
      mma_bf16(st.o[n][i], a[0], a[1], a[2], a[3], pl[n][0], pl[n][1]);
    }
  }
}

template <int D, bool KV4, int NT>
struct FewCfg {
  using Ring = typename std::conditional<KV4, RingKv4<D>, RingBf16<D>>::type;
  // Two CTAs an SM.  The bf16 cache needs bytes in flight (8 warps x 3 steps of 8 KB an SM),
  // the 4-bit one warps to unpack (16, 4 steps of 2.3 KB each); with 16 rows these want more
  // registers than two CTAs leave.
  static constexpr int kPerSm = KV4 && NT == 2 ? 1 : 2;
  static constexpr int kWarps = KV4 ? 8 : 4, kSteps = KV4 ? 4 : 3;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerTile = 8 / kWarps;                          // steps of a warp per tile
  static constexpr uint32_t kQ = 0;                                    // fragments [NT][D/16][32] x 8 bytes
  static constexpr uint32_t kML = kQ + NT * (D / 16) * 32 * 8;          // [warps][8 NT rows] (m, l)
  static constexpr uint32_t kRing = kML + kWarps * 8 * NT * 8;         // [warps][steps] slots
  static constexpr uint32_t kO = kRing;                                // [warps][8 NT rows][D + 4], after the ring's use
  static constexpr int kRow = D + 4;                                   // spreads the rows over the banks
  static constexpr uint32_t kRingBytes = kWarps * kSteps * Ring::kSlot, kOBytes = kWarps * 8 * NT * kRow * 4;
  static constexpr uint32_t kBytes = kRing + (kRingBytes > kOBytes ? kRingBytes : kOBytes);
};

template <int D, int PAGE, bool KV4, int NT>
__global__ void __launch_bounds__(FewCfg<D, KV4, NT>::kThreads, FewCfg<D, KV4, NT>::kPerSm) paged_few(const __grid_constant__ Params prm) {
  using M = FewCfg<D, KV4, NT>;
  constexpr int W = M::kWarps;
  extern __shared__ unsigned char smem_raw[];
  uint2 *qf = reinterpret_cast<uint2 *>(smem_raw + M::kQ);
  float2 *ml = reinterpret_cast<float2 *>(smem_raw + M::kML);
  float *ow = reinterpret_cast<float *>(smem_raw + M::kO);
  __shared__ int scan[3], sums[W];
  __shared__ Stop<KV4, PAGE> at;  // the current stop, read where it is needed: registers are short
  const Shape &sh = prm.sh;
  const PagedArgs &a = prm.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  grid_dep_wait();
  grid_dep_launch_dependents();
  cta_share<KV4, PAGE, M::kThreads>(prm, scan, sums);
  Walk<KV4, PAGE> way(scan);
  if (threadIdx.x == 0) {
    if (prm.shared_out) prm.piece[2 * blockIdx.x].unit = prm.piece[2 * blockIdx.x + 1].unit = -1;
  }
  for (;;) {
    if (threadIdx.x == 0) way.next(prm, at);
    __syncthreads();
    if (at.nt == 0) break;
    const Keys &ks = at.ks;
    // queries in the order of the contraction
    for (int e = threadIdx.x; e < NT * (D / 16) * 32; e += M::kThreads) {
      const int ln = e & 31, j = e / 32 % (D / 16), r = 8 * (e / 32 / (D / 16)) + (ln >> 2);
      uint2 q = make_uint2(0, 0);
      const int at = M::Ring::k_at(ln & 3, j);
      if (r < ks.rows)
        q = *reinterpret_cast<const uint2 *>(a.q + (((size_t)ks.s * sh.B + ks.b0 + r / sh.G) * sh.Hq + (size_t)ks.h * sh.G + r % sh.G) * D + at);
      qf[e] = q;
    }
    __syncthreads();
    FewState<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        st.m[n][e] = -INFINITY;
        st.l[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][i][e] = 0.f;
    }
    // which keys of the 16 at position `pos` (none at kNever) any row sees; bits of `hid` as above
    auto masks = [&](int pos, int end, uint32_t &on, uint32_t &hid) {
      on = 0xffffu;
      hid = 0;
      if (pos != kNever && pos + 16 <= end &&
          (KV4 || pos + 16 <= at.first.sk || (pos >= at.last.lb && pos + 15 <= at.first.hi)))
        return;
      on = visible(pos, 16, end, Limits{at.first.lb, at.last.hi, at.last.sk});
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = visible(pos, 16, end, row_limits<KV4>(a, ks.n, ks.b0 + (8 * n + 2 * t4 + e) / sh.G));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!((v >> (g + 8 * i)) & 1u)) hid |= 1u << (4 * n + 2 * i + e);
        }
    };
    // ---- tiles of pages.  Step i of a warp is 16 keys of tile i / kPerTile; the pages of 32
    //      steps are looked up at a time, a lane each.
    const int np = max(0, min(at.nt, ks.pt - at.t0)) * M::kPerTile, head = ks.h, n_ctx = ks.n;
    auto sub_of = [&](int i) { return warp + W * (i % M::kPerTile); };  // its place in the tile, in 16 keys
    int lps = -1, phs = -1;
    const uint32_t ring = smem_addr(smem_raw) + M::kRing + warp * (M::kSteps * M::Ring::kSlot);
    int pos_of = kNever;  // position of the first key of the step i with i % 32 = lane
    auto issue = [&](int i) {
      if (i < np) {
        if ((i & 31) == 0) {
          lps = phs = -1;
          const int e = i + lane;
          if (e < np) at.page_at(prm, at.t0 + e / M::kPerTile, 16 * sub_of(e) / PAGE, lps, phs);
          if (lps != -1 && phs < 0) raise_status(a.status, kStatusBadIndex);
        }
        const int lp = __shfl_sync(0xffffffffu, lps, i & 31), ph = __shfl_sync(0xffffffffu, phs, i & 31);
        const int in_page = 16 * sub_of(i) % PAGE;
        const int pos = ph >= 0 ? lp * PAGE + in_page : kNever;
        if (lane == (i & 31)) pos_of = pos;
        if (ph >= 0 && pos < n_ctx)
          M::Ring::fetch(ring + i % M::kSteps * M::Ring::kSlot, a, ((long long)ph * sh.Hkv + head) * PAGE + in_page, lane);
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < M::kSteps; ++i) issue(i);
#pragma unroll 1
    for (int i = 0; i < np; ++i) {
      uint32_t on, hid;
      masks(__shfl_sync(0xffffffffu, pos_of, i & 31), n_ctx, on, hid);
      cp_async_wait<M::kSteps - 1>();
      __syncwarp();  // every lane's part of the step is there
      if (on) {      // the same in every lane
        float x[NT][4];
        uint32_t ph[NT][2], pl[NT][2];
        typename M::Ring f;
        f.at = smem_raw + M::kRing + (warp * M::kSteps + i % M::kSteps) * M::Ring::kSlot;
        f.g = g;
        f.t = t4;
        few_scores<D, NT>(f, qf, lane, x);
        f.v_begin(on);
        few_softmax<D, NT>(st, x, hid, sh.sl2, ph, pl);
        few_values<D, NT>(f, st, ph, pl);
      }
      __syncwarp();  // every lane has read the slot
      issue(i + M::kSteps);
    }
    // ---- tiles of block tokens (bf16)
    for (int i = np; i < at.nt * M::kPerTile; ++i) {
      int u_end;
      bool fl;
      const int u = at.blk_tile(at.t0 + i / M::kPerTile, u_end, fl) + 16 * sub_of(i);
      if (u >= u_end) continue;
      uint32_t on0, hid0, ph[NT][2], pl[NT][2];
      masks(ks.n + u, ks.n + u_end, on0, hid0);
      if (!on0) continue;
      KeysBf16<D> b;
      const long long r0 = ((long long)ks.s * sh.B + u) * sh.Hkv + ks.h, stride = (long long)sh.Hkv * D;
      b.load_k(a.blk_k + r0 * D, stride, g, t4, on0);
      b.load_v(a.blk_v + r0 * D, stride, g, t4, on0);
      float x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        uint32_t fr[4];
        b.k_frag(jj, fr);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint2 q;
          if constexpr (KV4) {  // the stored queries follow the packed order: fetch these from memory
            const int r = 8 * n + g;
            q = make_uint2(0, 0);
            if (r < ks.rows)
              q = *reinterpret_cast<const uint2 *>(a.q + (((size_t)ks.s * sh.B + ks.b0 + r / sh.G) * sh.Hq + (size_t)ks.h * sh.G + r % sh.G) * D + KeysBf16<D>::k_at(t4, jj));
          } else {
            q = qf[(n * (D / 16) + jj) * 32 + lane];
          }
          mma_bf16(x[n], fr[0], fr[1], fr[2], fr[3], q.x, q.y);
        }
      }
      few_softmax<D, NT>(st, x, hid0, sh.sl2, ph, pl);
      few_values<D, NT>(b, st, ph, pl);
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings give way to the warps' O
    // ---- join the warps: sums over the lanes' keys, then (m, l, O) of each warp
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float &l = st.l[n][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = 8 * n + 2 * t4 + e;
        if (g == 0) ml[warp * 8 * NT + r] = make_float2(st.m[n][e], l);
        float *dst = ow + (warp * 8 * NT + r) * M::kRow + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[2 * i] = st.o[n][i][e];
          dst[2 * i + 1] = st.o[n][i][e + 2];
        }
      }
    __syncthreads();
    const bool whole = at.begins() && at.ends();
    const int slot = 2 * blockIdx.x + (at.begins() ? 1 : 0);
    if (!whole && threadIdx.x == 0) prm.piece[slot] = Piece{at.unit, at.begins(), at.ends(), 0};
    for (int e = threadIdx.x; e < ks.rows * (D / 4); e += M::kThreads) {
      // whole rows one after the other; a piece's side by side
      const int r = whole ? e / (D / 4) : e % ks.rows, c = (whole ? e % (D / 4) : e / ks.rows) * 4;
      float mx = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 v = ml[w * 8 * NT + r];
        if (v.y != 0.f) mx = fmaxf(mx, v.x);
      }
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 v = ml[w * 8 * NT + r];
        if (v.y == 0.f) continue;
        const float wt = v.x == -INFINITY ? 1.f : exp2f(v.x - mx);
        L = fmaf(wt, v.y, L);
        const float4 z = *reinterpret_cast<const float4 *>(ow + (w * 8 * NT + r) * M::kRow + c);
        y.x = fmaf(wt, z.x, y.x); y.y = fmaf(wt, z.y, y.y); y.z = fmaf(wt, z.z, y.z); y.w = fmaf(wt, z.w, y.w);
      }
      const size_t orow = ((size_t)ks.s * sh.B + ks.b0 + r / sh.G) * sh.Hq + (size_t)ks.h * sh.G + r % sh.G;
      const size_t prow = (size_t)slot * ((size_t)prm.bpt * sh.G) + r;
      if (whole) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint2 *>(a.o_out + orow * D + c) = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
        if (c == 0 && sh.lse_out) sh.lse_out[orow] = L != 0.f ? (mx + log2f(L)) * 0.6931471805599453f : -INFINITY;
      } else {
        prm.part_o[((size_t)slot * (D / 4) + c / 4) * (prm.bpt * sh.G) + r] = y;
        if (c == 0) prm.part_ml[prow] = make_float2(mx, L);
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of the units that shares cut: block x takes the unit that CTA x began and
// left (its later pieces are the first ones of CTAs x + 1, x + 2, ...); a thread has four
// columns of a row.  The pieces are joined in their order.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge(const __grid_constant__ Params prm) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const Shape &sh = prm.sh;
  const int rpt = prm.bpt * sh.G;  // rows of a unit
  const int lane = threadIdx.x & 31;
  const Piece p = prm.piece[2 * blockIdx.x + 1];
  if (p.unit < 0) return;
  // the pieces: slot 2 x + 1, then slots 2 (x + 1), ... to the one that ends the unit; a lane
  // looks at one each, so that the chain costs one round of loads per 32
  int count = 0;
  for (int i0 = 0;; i0 += 32) {
    const int c = blockIdx.x + i0 + lane;
    const bool ends = c > (int)gridDim.x || prm.piece[c == (int)blockIdx.x ? 2 * c + 1 : 2 * c].ends;
    const uint32_t found = __ballot_sync(0xffffffffu, ends);
    count += found ? __ffs(found) : 32;
    if (found) break;
  }
  count = min(count, (int)gridDim.x + 1 - (int)blockIdx.x);  // (a call that gave up may have left no end)
  const int rt = p.unit % prm.rowtiles, h = p.unit / prm.rowtiles % sh.Hkv, s = p.unit / prm.rowtiles / sh.Hkv;
  const int e = blockIdx.y * kMergeThreads + threadIdx.x, c4 = e / rpt, r = e % rpt;
  const int b = rt * prm.bpt + r / sh.G;
  if (c4 >= D / 4 || b >= block_tokens(prm.a.n_new, s, sh.B, prm.a.status, false)) return;
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < count; i0 += 8) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i >= count) continue;
      const size_t slot = i0 + i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i0 + i);
      ml[i] = prm.part_ml[slot * rpt + r];
      v[i] = prm.part_o[(slot * (D / 4) + c4) * rpt + r];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ml[i].y == 0.f) continue;  // a piece without a visible key holds zeros
      const float mn = fmaxf(M, ml[i].x);
      const float sc = M == -INFINITY ? 0.f : exp2f(M - mn), wt = ml[i].x == -INFINITY ? 1.f : exp2f(ml[i].x - mn);
      M = mn;
      L = fmaf(L, sc, wt * ml[i].y);
      o.x = fmaf(o.x, sc, wt * v[i].x); o.y = fmaf(o.y, sc, wt * v[i].y);
      o.z = fmaf(o.z, sc, wt * v[i].z); o.w = fmaf(o.w, sc, wt * v[i].w);
    }
  }
  const size_t orow = ((size_t)s * sh.B + b) * sh.Hq + (size_t)h * sh.G + r % sh.G;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<uint2 *>(prm.a.o_out + orow * D + 4 * c4) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (sh.lse_out && c4 == 0) sh.lse_out[orow] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

struct Geometry {
  int bpt, rowtiles, rows;  // rows of a unit
  long long units;
};
Geometry geometry(const Shape &sh) {
  Geometry g;
  g.bpt = std::min(kRowsPerTile / sh.G, sh.B);
  g.rowtiles = (sh.B + g.bpt - 1) / g.bpt;
  g.rows = g.bpt * sh.G;
  g.units = (long long)sh.S * sh.Hkv * g.rowtiles;
  return g;
}

PagedPlan make_plan(const Shape &sh, int sms, long long max_tiles, bool kv4) {
  const Geometry g = geometry(sh);
  PagedPlan p{};
  p.few = g.rows <= kFewRows;
  const int per_sm = !p.few ? 1 : kv4 ? (g.rows <= 8 ? FewCfg<128, true, 1>::kPerSm : FewCfg<128, true, 2>::kPerSm)
                                      : FewCfg<128, false, 1>::kPerSm;
  const int ctas = per_sm * sms;
  // Whole units where there are many, or where none is long enough to be cut, or where the tiles
  // of all, which the CTAs count in 32 bits, could be too many (a unit's ranges may each end in
  // a tile that max_tiles does not count).
  p.shared_out = g.units <= std::min((long long)kManyUnits * ctas, (long long)kMaxShared) && max_tiles > kMinTiles &&
                 g.units * (max_tiles + 4) <= INT_MAX;
  p.ctas = p.shared_out ? ctas : (int)std::min<long long>(ctas, g.units);
  p.launches = p.shared_out && ctas > 1 ? 2 : 1;
  // the same for every window, so that one workspace serves a model's layers
  p.total = kWorkspaceHeader + 2 * (size_t)ctas * (sizeof(Piece) + g.rows * ((size_t)sh.d * 4 + 8));
  return p;
}

template <int D, int PAGE, bool KV4, int NT>
cudaError_t launch_few(const Params &prm, const PagedPlan &plan, cudaStream_t stream) {
  constexpr auto kern = paged_few<D, PAGE, KV4, NT>;
  using M = FewCfg<D, KV4, NT>;
  cudaError_t err = set_smem_once<kern>(M::kBytes);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3((unsigned)plan.ctas), M::kThreads, M::kBytes, stream, prm);
}

template <int D, int PAGE, bool KV4>
cudaError_t launch_typed(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  using C = Cfg<D, KV4>;
  const Geometry g = geometry(sh);
  if (g.units > INT_MAX) return cudaErrorInvalidValue;
  Params prm{};
  prm.sh = sh;
  prm.a = a;
  prm.bpt = g.bpt;
  prm.rowtiles = g.rowtiles;
  prm.units = (int)g.units;
  prm.shared_out = plan.shared_out;
  prm.box_blk = std::min(kBN, (sh.B + 15) / 16 * 16);
  unsigned char *ws = reinterpret_cast<unsigned char *>(a.status) + kWorkspaceHeader;
  const size_t slots = 2 * (size_t)plan.ctas;
  prm.piece = reinterpret_cast<Piece *>(ws);
  prm.part_o = reinterpret_cast<float4 *>(ws + slots * sizeof(Piece));
  prm.part_ml = reinterpret_cast<float2 *>(prm.part_o + slots * g.rows * (D / 4));
  auto join = [&](cudaError_t e) {
    if (e != cudaSuccess || plan.launches == 1) return e;
    return launch_pdl(paged_merge<D>, dim3((unsigned)(plan.ctas - 1), (unsigned)((g.rows * (D / 4) + kMergeThreads - 1) / kMergeThreads)),
                      kMergeThreads, 0, stream, prm);
  };
  if (plan.few)
    return join(g.rows <= 8 ? launch_few<D, PAGE, KV4, 1>(prm, plan, stream) : launch_few<D, PAGE, KV4, 2>(prm, plan, stream));
  constexpr auto kern = paged_attn<D, PAGE, KV4>;
  cudaError_t err = set_smem_once<kern>(C::kAlloc);
  if (err != cudaSuccess) return err;
  CUtensorMap q{}, k{}, v{}, bk{}, bv{};
  const long long tokens = (long long)sh.S * sh.B;
  if ((err = make_q_tensor_map(&q, a.q, tokens, sh.Hq, D, sh.G, g.bpt)) != cudaSuccess) return err;
  if (!KV4 && PAGE < 64) {
    if ((err = make_kv_pages_tensor_map(&k, a.k, sh.n_phys, sh.Hkv, PAGE, D, kBN / PAGE)) != cudaSuccess) return err;
    if ((err = make_kv_pages_tensor_map(&v, a.v, sh.n_phys, sh.Hkv, PAGE, D, kBN / PAGE)) != cudaSuccess) return err;
  } else if (!KV4) {
    const long long nrows = sh.n_phys * sh.Hkv * PAGE;
    if ((err = make_kv_tensor_map(&k, a.k, nrows, D, PAGE)) != cudaSuccess) return err;
    if ((err = make_kv_tensor_map(&v, a.v, nrows, D, PAGE)) != cudaSuccess) return err;
  }
  if (a.blk_k) {
    if ((err = make_blk_tensor_map(&bk, a.blk_k, tokens, sh.Hkv, D, prm.box_blk)) != cudaSuccess) return err;
    if ((err = make_blk_tensor_map(&bv, a.blk_v, tokens, sh.Hkv, D, prm.box_blk)) != cudaSuccess) return err;
  }
  return join(launch_pdl(kern, dim3((unsigned)plan.ctas), C::kThreads, C::kAlloc, stream, prm, q, k, v, bk, bv));
}

template <bool KV4>
cudaError_t launch_any(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  if (sh.d == 128) {
    if (sh.P == 16) return launch_typed<128, 16, KV4>(sh, plan, a, stream);
    if (sh.P == 32) return launch_typed<128, 32, KV4>(sh, plan, a, stream);
    return launch_typed<128, 64, KV4>(sh, plan, a, stream);
  }
  if (sh.P == 16) return launch_typed<64, 16, KV4>(sh, plan, a, stream);
  if (sh.P == 32) return launch_typed<64, 32, KV4>(sh, plan, a, stream);
  return launch_typed<64, 64, KV4>(sh, plan, a, stream);
}

}  // namespace

PagedPlan plan_window(const Shape &sh, int num_sms, int window, int sinks) {
  const Geometry g = geometry(sh);
  const long long prefix = (long long)sh.max_pages * sh.P;
  const long long reach = std::min(prefix, (long long)window + sinks) + std::min((long long)sh.B, (long long)window + g.bpt);
  return make_plan(sh, num_sms, (reach + kBN - 1) / kBN, false);
}

PagedPlan plan_kv4(const Shape &sh, int num_sms, bool sparse) {
  const long long prefix = (long long)(sparse ? std::min(sh.kmax, sh.max_pages) : sh.max_pages) * sh.P;
  return make_plan(sh, num_sms, (prefix + kBN - 1) / kBN + (sh.B + kBN - 1) / kBN, true);
}

cudaError_t launch_window(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  return launch_any<false>(sh, plan, a, stream);
}
cudaError_t launch_kv4_attn(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  return launch_any<true>(sh, plan, a, stream);
}

}  // namespace dsa
