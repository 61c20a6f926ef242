// paged_attn.cu -- dsa_window_attn and dsa_kv4_attn: softmax attention of a block's
// queries over a paged cache, in bf16 with a sliding window and sinks or in 4 bits,
// and over the block's own tokens.
//
//   x_j = q.k_j / sqrt(d) over the visible keys j,  o = sum_j e^(x_j - m) v_j / l,
//   l = sum_j e^(x_j - m),  lse = m + ln l
//
// One CTA takes up to 128 query rows (token, head of one KV head's group) and a share
// of their keys in tiles of 128: pages that hold a visible token, then block tokens.
// Rows whose keys are shared out over several CTAs leave (O, m, l) in fp32 in the
// workspace, and paged_merge joins them.
//
// Warp roles: warp 0 loads the queries and (bf16 cache) the key tiles with TMA; warp 1
// owns TMEM and issues the MMAs; warps 2..9 are two softmax groups that take alternate
// tiles, a thread per row; warps 10..13 (4-bit cache) turn packed rows into bf16 tiles.
//   S = Q K^T (128 x 128, TMEM), P = 2^(S - m) in bf16 over S's first 64 columns,
//   O += P V (TMEM, one accumulator per group), joined at the end.
// The reference maximum of a row moves only when a tile beats it by 2^8, so O is
// rarely rescaled.  Sums and outputs are held in fp32, P alone in bf16 (the type of V,
// which one MMA takes both operands in).
#include <climits>

#include "paged.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kBN = 128;  // keys of a tile
constexpr int kRowsPerTile = 128;
constexpr int kNever = INT_MAX;  // position of a key that takes no part
constexpr float kRescaleLog2 = 8.f;

template <int D, bool KV4>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kThreads = KV4 ? 448 : 320;
  static constexpr uint32_t kHalf = 128u * 128u;           // 128 rows x 128 B
  static constexpr uint32_t kTile = kHalves * kHalf;       // one K or V tile, or Q
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kTile;
  static constexpr uint32_t kOffV = kOffK + kStages * kTile;
  static constexpr uint32_t kOffBar = kOffV + kStages * kTile;
  static constexpr int kNumBars = 4 * kStages + 8;
  static constexpr uint32_t kOffTab = kOffBar + kNumBars * 8;      // per stage: 8 positions, flags, end
  static constexpr uint32_t kOffMisc = kOffTab + kStages * 48;     // TMEM address, abort flag
  static constexpr uint32_t kAlloc = kOffMisc + 16 + 1024;         // room to align the base to 1 KB
  static constexpr uint32_t kOffML = kOffQ;                        // [2][128] (m, l) once Q is dead
  static constexpr uint32_t kTmemO = 2 * kBN;
  static constexpr uint32_t kTmemCols = 512;
};

struct Params {
  Shape sh;
  PagedArgs a;
  int bpt;        // block tokens of a row tile
  int rowtiles;
  int splits;
  int box_blk;    // block tokens of one TMA box
  float *part_o;  // [unit][split][rows][D]
  float2 *part_ml;
};

// What a CTA attends to: a list of pages and two ranges of block tokens.
struct Keys {
  int n, nb;          // prefix and block tokens
  int nsp, wp0, npg;  // pages: sinks' pages 0..nsp-1, then wp0.. ; npg in all (or idx entries)
  int pt;             // tiles of pages
  int ua, ub0, ub;    // block tokens [0, ua) and [ub0, ub)
  int ta, tiles;      // tiles of the first range; tiles in all
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

// Bits j < len whose position base + j is below x.
__device__ __forceinline__ uint32_t below(int base, int x, int len) {
  const int c = x <= base ? 0 : min((int)min((long long)x - base, (long long)len), len);
  return c >= 32 ? 0xffffffffu : (1u << c) - 1u;
}
__device__ __forceinline__ uint32_t visible(int base, int len, int end, const Limits &w) {
  if (base == kNever) return 0u;
  return below(base, end, len) & (below(base, w.sk, len) | (~below(base, w.lb, len) & below(base, w.hi + 1, len)));
}
// The same for 32 keys of a tile whose units of PAGE keys (or 128, a block tile) start at
// the table's positions.
template <int PAGE>
__device__ __forceinline__ uint32_t visible32(const int *pos, bool blk, int word, int end, const Limits &w) {
  if (blk) return visible(pos[0] + 32 * word, 32, end, w);
  if (PAGE == 16)
    return visible(pos[2 * word], 16, end, w) | (visible(pos[2 * word + 1], 16, end, w) << 16);
  const int base = pos[32 * word / PAGE];
  return base == kNever ? 0u : visible(base + 32 * word % PAGE, 32, end, w);
}

template <int D, int PAGE, bool KV4>
__global__ void __launch_bounds__(Cfg<D, KV4>::kThreads, 1)
    paged_attn(const __grid_constant__ Params prm, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ CUtensorMap kmap4, const __grid_constant__ CUtensorMap vmap4,
               const __grid_constant__ CUtensorMap bkmap, const __grid_constant__ CUtensorMap bvmap) {
  using C = Cfg<D, KV4>;
  constexpr int ST = C::kStages;
  constexpr int PPT = kBN / PAGE;  // pages of a tile
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
  auto s_full = [&](int g) { return bar(4 * ST + g); };
  auto p_full = [&](int g) { return bar(4 * ST + 2 + g); };
  auto pv_done = [&](int g) { return bar(4 * ST + 4 + g); };
  const uint32_t q_full = bar(4 * ST + 6), drain = bar(4 * ST + 7);
  auto table = [&](int st) { return reinterpret_cast<int *>(smem + C::kOffTab + st * 48); };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
  const WaitCtx ctx{abort_flag, a.status};
  volatile int never = 0;
  const WaitCtx drain_ctx{&never, a.status};

  // unit: (sequence, KV head, row tile, split)
  const int sp = blockIdx.x % prm.splits;
  const int unit = blockIdx.x / prm.splits;
  const int rt = unit % prm.rowtiles;
  const int h = unit / prm.rowtiles % sh.Hkv;
  const int s = unit / prm.rowtiles / sh.Hkv;
  const int b0 = rt * prm.bpt;
  const int rows_max = min(prm.bpt, sh.B - b0) * sh.G;  // before n_new
  const int active_warps = (rows_max + 31) / 32;        // of each softmax group

  if (threadIdx.x == 0) {
    for (int st = 0; st < ST; ++st) {
      mbar_init(k_full(st), KV4 ? 128 : 1);
      mbar_init(k_empty(st), 1);
      mbar_init(v_full(st), KV4 ? 128 : 1);
      mbar_init(v_empty(st), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(s_full(g), 1);
      mbar_init(p_full(g), 32 * active_warps);
      mbar_init(pv_done(g), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&qmap);
    if (!KV4) {
      tma_prefetch_map(&kmap);
      tma_prefetch_map(&vmap);
    }
  }
  if (warp == 1) {
    tmem_alloc(base + C::kOffMisc, C::kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();

  // ---- the keys of this row tile, and this split's tiles of them
  const bool reporter = threadIdx.x == 0 && h == 0 && rt == 0 && sp == 0;
  Keys ks;
  ks.n = clamp_prefix(a.n_ctx[s], sh.max_pages, PAGE, a.status, reporter);
  ks.nb = block_tokens(a.n_new, s, sh.B, a.status, reporter);
  const int b_end = min(b0 + prm.bpt, ks.nb);  // this tile's tokens are [b0, b_end)
  const int rows = max(0, b_end - b0) * sh.G;
  const int32_t *idx_head = nullptr;
  Limits first = row_limits<KV4>(a, ks.n, b0), last = row_limits<KV4>(a, ks.n, max(b0, b_end - 1));
  {
    const int np = (ks.n + PAGE - 1) / PAGE;
    if (KV4) {
      ks.nsp = 0;
      ks.wp0 = 0;
      ks.npg = np;
      if (a.idx) {
        idx_head = a.idx + ((size_t)s * sh.Hkv + h) * sh.kmax;
        ks.npg = a.idx_cnt[(size_t)s * sh.Hkv + h];
        if (ks.npg < 0 || ks.npg > sh.kmax) {
          if (threadIdx.x == 0 && rt == 0 && sp == 0) raise_status(a.status, kStatusBadIndex);
          ks.npg = max(0, min(ks.npg, sh.kmax));
        }
      }
      ks.ua = 0;
      ks.ub0 = 0;
      ks.ub = a.blk_k ? ks.nb : 0;
    } else {
      const int lb = max(0, first.lb);  // the lowest position that a window of the tile reaches
      ks.nsp = (min(min(a.sinks, ks.n), lb) + PAGE - 1) / PAGE;
      ks.wp0 = max(ks.nsp, lb / PAGE);
      ks.npg = ks.nsp + max(0, np - ks.wp0);
      const int ue = a.blk_k ? (a.causal ? min(ks.nb, b_end) : ks.nb) : 0;
      ks.ua = max(0, min(ue, clamp_int((long long)last.sk - ks.n)));  // sinks that reach into the block
      ks.ub0 = max(ks.ua, clamp_int((long long)first.lb - ks.n));
      ks.ub = min(ue, clamp_int((long long)last.hi + 1 - ks.n));
      if (ks.ub0 >= ks.ub) ks.ub0 = ks.ub = 0;
    }
    ks.pt = (ks.npg + PPT - 1) / PPT;
    ks.ta = (ks.ua + kBN - 1) / kBN;
    ks.tiles = rows > 0 ? ks.pt + ks.ta + (ks.ub - ks.ub0 + kBN - 1) / kBN : 0;
  }
  const int t0 = (int)((long long)ks.tiles * sp / prm.splits);
  const int nt = (int)((long long)ks.tiles * (sp + 1) / prm.splits) - t0;
  const int pend = ks.n;

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc);

  // page e of tile t (both counted from the list's start): logical and physical
  auto page_at = [&](int t, int e, int &lp, int &phys) {
    const int i = t * PPT + e;
    lp = -1;
    phys = -1;
    if (t >= ks.pt || i >= ks.npg) return;
    if (KV4 && idx_head) {
      lp = idx_head[i];
      if (lp < 0 || (long long)lp * PAGE >= ks.n) lp = -2;
    } else {
      lp = i < ks.nsp ? i : ks.wp0 + (i - ks.nsp);
    }
    if (lp >= 0) phys = (int)physical_page(sh, s, lp);
  };
  // a page whose every token every row sees
  auto page_full = [&](int lp, int phys) {
    const int pb = lp * PAGE;
    return phys >= 0 && pb + PAGE <= pend && (KV4 || pb + PAGE <= a.sinks || pb >= last.lb);
  };
  // first block token of tile t >= pt, where its range ends (a tile of the first range must
  // not repeat tokens of the second), and whether every row sees all 128
  auto blk_tile = [&](int t, int &u_end, bool &full) {
    const int i = t - ks.pt;
    const bool sink = i < ks.ta;
    const int u0 = sink ? i * kBN : ks.ub0 + (i - ks.ta) * kBN;
    const int p0 = ks.n + u0;
    u_end = sink ? ks.ua : ks.nb;
    full = u0 + kBN <= u_end && (sink ? p0 + kBN <= first.sk : p0 >= last.lb && p0 + kBN - 1 <= first.hi);
    return u0;
  };

  float m_used = -INFINITY, l = 0.f;
  bool alive = true;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer --
    if (lane == 0 && nt > 0) {
      mbar_arrive_expect_tx(q_full, (uint32_t)min(prm.bpt, sh.B) * sh.G * 128u * C::kHalves);
      for (int hf = 0; hf < C::kHalves; ++hf)
        tma_load_3d(base + C::kOffQ + hf * C::kHalf, &qmap, q_full, hf * 64, h * sh.G, s * sh.B + b0);
    }
    __syncwarp();
    if (!KV4) {
      int issued_k = 0, issued_v = 0;
      int lp = -1, phys = -1;
      if (nt > 0 && lane < PPT) page_at(t0, lane, lp, phys);
      for (int k = 0; k < nt; ++k) {
        const int st = k % ST, t = t0 + k;
        int lp1 = -1, phys1 = -1;  // the next tile's pages, fetched before this tile's waits
        if (k + 1 < nt && lane < PPT) page_at(t + 1, lane, lp1, phys1);
        const uint32_t sk = base + C::kOffK + st * C::kTile, sv = base + C::kOffV + st * C::kTile;
        const bool blk = t >= ks.pt;
        bool full = false;
        int u0 = 0, u_end = 0, nvalid = 0;
        bool run = false;
        if (blk) {
          u0 = blk_tile(t, u_end, full);
        } else {
          const bool listed = lane < PPT && lp != -1;
          if (listed && phys < 0) raise_status(a.status, kStatusBadIndex);
          nvalid = __popc(__ballot_sync(0xffffffffu, listed && phys >= 0));
          full = __all_sync(0xffffffffu, lane >= PPT || page_full(lp, phys)) && nvalid == PPT;
          const int p0 = __shfl_sync(0xffffffffu, phys, 0);
          run = nvalid == PPT && __all_sync(0xffffffffu, lane >= PPT || phys == p0 + lane);
        }
        const uint32_t bytes = (blk ? (uint32_t)prm.box_blk : (uint32_t)nvalid * PAGE) * 128u * C::kHalves;
        auto load = [&](uint32_t dst, uint32_t br, const CUtensorMap *m2, const CUtensorMap *m4, const CUtensorMap *mb) {
          if (lane == 0) mbar_arrive_expect_tx(br, bytes);
          __syncwarp();
          if (blk) {
            if (lane < C::kHalves) tma_load_3d(dst + lane * C::kHalf, mb, br, lane * 64, h, s * sh.B + u0);
          } else if (run) {
            const int p0 = __shfl_sync(0xffffffffu, phys, 0);
            if (lane < C::kHalves) tma_load_4d(dst + lane * C::kHalf, m4, br, lane * 64, 0, h, p0);
          } else {
            const int e = lane % PPT, hf = lane / PPT;
            const int ph = __shfl_sync(0xffffffffu, phys, e);
            if (hf < C::kHalves && ph >= 0)
              tma_load_2d(dst + hf * C::kHalf + e * PAGE * 128u, m2, br, hf * 64,
                          (int)(((long long)ph * sh.Hkv + h) * PAGE));
          }
        };
        if (k >= ST && !__all_sync(0xffffffffu, mbar_wait(k_empty(st), ((k / ST) - 1) & 1, ctx))) break;
        load(sk, k_full(st), &kmap, &kmap4, &bkmap);
        issued_k = k + 1;
        if (k >= ST && !__all_sync(0xffffffffu, mbar_wait(v_empty(st), ((k / ST) - 1) & 1, ctx))) break;
        int *tab = table(st);
        if (blk) {
          if (lane == 0) tab[0] = ks.n + u0;
        } else if (lane < PPT) {
          tab[lane] = phys >= 0 ? lp * PAGE : kNever;
        }
        if (lane == 0) {
          tab[8] = (full ? 1 : 0) | (blk ? 2 : 0);
          tab[9] = blk ? ks.n + u_end : ks.n;
        }
        __syncwarp();
        load(sv, v_full(st), &vmap, &vmap4, &bvmap);
        issued_v = k + 1;
        lp = lp1;
        phys = phys1;
      }
      // copies in flight land before the CTA's shared memory is released
      if (lane == 0) {
        for (int k = max(0, issued_k - ST); k < issued_k; ++k) mbar_wait(k_full(k % ST), (k / ST) & 1, drain_ctx);
        for (int k = max(0, issued_v - ST); k < issued_v; ++k) mbar_wait(v_full(k % ST), (k / ST) & 1, drain_ctx);
      }
    }
    if (lane == 0 && nt > 0) mbar_wait(q_full, 0, drain_ctx);
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer --
    // Every parity wait below is on the barrier's current or just completed phase:
    // a stage is refilled only after the commit that frees it, which follows the wait
    // for its fill; S of a group's next tile is sent after the wait for P of its last
    // one, and pv_done(g) is waited for once per phase, right where the S follows.
    if (lane == 0 && nt > 0) {
      constexpr uint32_t ids = idesc_bf16(128, kBN, false, false);
      constexpr uint32_t ido = idesc_bf16(128, D, false, true);
      auto issue_s = [&](int j) {
        const int st = j % ST, g = j & 1;
        if (!mbar_wait(k_full(st), (j / ST) & 1, ctx)) return false;
        // P of this group's previous tile lies in the same columns: its PV must be done
        if (j >= 2 && !mbar_wait(pv_done(g), ((j >> 1) - 1) & 1, ctx)) return false;
        tc_fence_after();
        const uint32_t sk = base + C::kOffK + st * C::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kHalf + (kk & 3) * 32;
          umma_bf16(tmem + g * kBN, sdesc_sw128(base + C::kOffQ + off, 16, 1024), sdesc_sw128(sk + off, 16, 1024), ids,
                    kk > 0 ? 1u : 0u);
        }
        umma_commit(s_full(g));
        umma_commit(k_empty(st));
        return true;
      };
      bool ok = mbar_wait(q_full, 0, ctx);
      for (int j = 0; ok && j < 2 && j < nt; ++j) ok = issue_s(j);
      for (int j = 0; ok && j < nt; ++j) {
        const int st = j % ST, g = j & 1;
        if (!mbar_wait(p_full(g), (j >> 1) & 1, ctx)) break;
        if (!mbar_wait(v_full(st), (j / ST) & 1, ctx)) break;
        tc_fence_after();
        const uint32_t sv = base + C::kOffV + st * C::kTile;
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          umma_bf16_ts(tmem + C::kTmemO + g * D, tmem + g * kBN + kk * 8, sdesc_sw128(sv + kk * 16 * 128, C::kHalf, 1024),
                       ido, (j > 1 || kk > 0) ? 1u : 0u);
        umma_commit(pv_done(g));
        umma_commit(v_empty(st));
        if (j + 2 < nt) ok = issue_s(j + 2);
      }
      umma_commit(drain);  // every issued MMA completes before TMEM is released
      mbar_wait(drain, 0, drain_ctx);
    }
    __syncwarp();
  } else if (warp < 10) {
    // ---------------------------------------------------------- softmax groups --
    const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    // the quarters of TMEM's lanes that hold rows; the other warps have nothing to do
    if (quarter < active_warps) {
      const uint32_t lt = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t sc = lt + g * kBN, oc = lt + C::kTmemO + g * D;
      const Limits mine = row_limits<KV4>(a, ks.n, b0 + r / sh.G);
      Limits all;  // keys that some row of the tile may see
      all.lb = first.lb;
      all.hi = last.hi;
      all.sk = last.sk;
      int m = 0;  // tiles this group has finished
      for (int k = g; k < nt; k += 2, ++m) {
        const int st = k % ST;
        alive = __all_sync(0xffffffffu, mbar_wait(s_full(g), m & 1, ctx));
        // the tile's table, and V for the rows zeroed below (its stage is refilled only
        // after this tile's P)
        alive = alive && __all_sync(0xffffffffu, mbar_wait(v_full(st), (k / ST) & 1, ctx));
        if (!alive) break;
        tc_fence_after();
        const int *tab = table(st);
        const int flags = tab[8];
        const bool blk = flags & 2;
        const int end = tab[9];
        uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
        if (!(flags & 1)) {
#pragma unroll
          for (int w = 0; w < 4; ++w) bits[w] = visible32<PAGE>(tab, blk, w, end, mine);
          // value rows that no row of the tile sees are zeroed: 0 * stale data must not reach O
          for (int key = quarter * 32 + lane; key < kBN; key += 32 * active_warps) {
            const uint32_t any = visible32<PAGE>(tab, blk, key >> 5, end, all);
            if ((any >> (key & 31)) & 1u) continue;
            unsigned char *row = smem + C::kOffV + st * C::kTile + key * 128;
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
              for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + hf * C::kHalf + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
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
        for (int j = 0; j < kHold; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(x[j]));
        if constexpr (KV4) {
#pragma unroll
          for (int w = 2; w < 4; ++w) {
            uint32_t y[32];
            tmem_ld32(sc + 32 * w, y);
            hide(y, w);
#pragma unroll
            for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(y[j]));
          }
        }
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sh.sl2;
        const bool need = tmax > m_used + kRescaleLog2 || (m_used == -INFINITY && tmax > -INFINITY);
        if (__any_sync(0xffffffffu, need)) {
          float alpha = 1.f;
          if (need) {
            alpha = m_used == -INFINITY ? 0.f : fast_exp2(m_used - tmax);
            m_used = tmax;
            l *= alpha;
          }
          if (m > 0) {  // PV of the group's previous tile is done: this tile's S was sent after it
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(oc + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(oc + c0, o);
            }
          }
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
        mbar_arrive(p_full(g));
      }
      if (alive && m > 0) {  // the issuer's one commit after its last MMA
        alive = __all_sync(0xffffffffu, mbar_wait(drain, 0, ctx));
        tc_fence_after();
      }
      if (!alive || m == 0) l = 0.f;
    }
  } else if (KV4) {
    // ------------------------------------------- packed rows into bf16 tiles --
    // 128 threads; chunk i of a thread is the 16 bytes (32 values, one scale) of group
    // tid % GR of key 128 / CH * i + tid / GR.  The packed rows of the next tile are
    // loaded before this tile's stage is waited for, its page ids one tile earlier.
    constexpr int GR = D / kKv4Group;  // groups of a row
    constexpr int CH = GR;             // chunks of a thread: 128 * GR / 128
    const int tid = threadIdx.x - 320;
    const int grp = tid % GR;
    struct Raw {
      uint4 k[CH], v[CH];
      __nv_bfloat16 ks[CH], vs[CH];
    };
    auto key_of = [&](int i) { return i * (kBN / CH) + tid / GR; };
    auto ids_of = [&](int t, int (&lp)[CH], int (&phys)[CH]) {
#pragma unroll
      for (int i = 0; i < CH; ++i) page_at(t, key_of(i) / PAGE, lp[i], phys[i]);
    };
    auto on = [&](int i, const int (&lp)[CH], const int (&phys)[CH]) {
      return phys[i] >= 0 && lp[i] * PAGE + key_of(i) % PAGE < pend;
    };
    auto fetch = [&](Raw &x, const int (&lp)[CH], const int (&phys)[CH]) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (!on(i, lp, phys)) continue;
        const long long row = ((long long)phys[i] * sh.Hkv + h) * PAGE + key_of(i) % PAGE;
        x.k[i] = __ldg(reinterpret_cast<const uint4 *>(a.kv4.k + row * (D / 2)) + grp);
        x.ks[i] = a.kv4.ks[row * GR + grp];
        x.v[i] = __ldg(reinterpret_cast<const uint4 *>(a.kv4.v + row * (D / 2)) + grp);
        x.vs[i] = a.kv4.vs[row * GR + grp];
      }
    };
    auto put = [&](uint32_t off, const uint4 (&w)[CH], const __nv_bfloat16 (&sc)[CH], const int (&lp)[CH], const int (&phys)[CH]) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int key = key_of(i);
        unsigned char *dst = smem + off + (grp / 2) * C::kHalf;
        const bool o = on(i, lp, phys);
        __nv_bfloat162 s8, m24;
        kv4_constants(sc[i], s8, m24);
        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 y = make_uint4(0, 0, 0, 0);
          if (o) y = make_uint4(kv4_pair(ww[c], 0, s8, m24), kv4_pair(ww[c], 1, s8, m24), kv4_pair(ww[c], 2, s8, m24), kv4_pair(ww[c], 3, s8, m24));
          *reinterpret_cast<uint4 *>(dst + sw128_offset(key, (grp % 2) * 4 + c)) = y;
        }
      }
    };
    Raw cur, nxt;
    int lp0[CH], ph0[CH], lp1[CH], ph1[CH];
    int issued = 0;
    bool ok = true;
    if (nt > 0) {
      ids_of(t0, lp0, ph0);
      fetch(cur, lp0, ph0);
      ids_of(t0 + 1, lp1, ph1);
    }
    for (int k = 0; ok && k < nt; ++k) {
      const int st = k % ST, t = t0 + k;
      const bool blk = t >= ks.pt;
      int lp2[CH], ph2[CH];
      fetch(nxt, lp1, ph1);
      ids_of(t + 2, lp2, ph2);
      int elp = -1, ephys = -1;  // the table's entry of this lane
      if (tid < PPT) page_at(t, tid, elp, ephys);
      bool full = false;
      int u0 = 0, u_end = 0;
      if (blk) u0 = blk_tile(t, u_end, full);
      if (k >= ST) ok = __all_sync(0xffffffffu, mbar_wait(k_empty(st), ((k / ST) - 1) & 1, ctx));
      if (!ok) break;
      const uint32_t bytes = (uint32_t)prm.box_blk * 128u * C::kHalves;
      const uint32_t ok_k = C::kOffK + st * C::kTile, ok_v = C::kOffV + st * C::kTile;
      if (blk) {
        if (tid == 0) {
          mbar_arrive_expect_tx(k_full(st), bytes);
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(base + ok_k + hf * C::kHalf, &bkmap, k_full(st), hf * 64, h, s * sh.B + u0);
        } else {
          mbar_arrive(k_full(st));
        }
      } else {
        put(ok_k, cur.k, cur.ks, lp0, ph0);
        fence_proxy_async_smem();
        mbar_arrive(k_full(st));
      }
      if (k >= ST) ok = __all_sync(0xffffffffu, mbar_wait(v_empty(st), ((k / ST) - 1) & 1, ctx));
      issued = k + 1;
      if (!ok) break;
      if (tid < 32) {
        int *tab = table(st);
        if (blk) {
          if (tid == 0) tab[0] = ks.n + u0;
        } else {
          if (elp != -1 && ephys < 0) raise_status(a.status, kStatusBadIndex);
          if (tid < PPT) tab[tid] = ephys >= 0 ? elp * PAGE : kNever;
          full = __all_sync(0xffffffffu, tid >= PPT || page_full(elp, ephys));
        }
        if (tid == 0) {
          tab[8] = (full ? 1 : 0) | (blk ? 2 : 0);
          tab[9] = blk ? ks.n + u_end : ks.n;
        }
        __syncwarp();
      }
      if (blk) {
        if (tid == 0) {
          mbar_arrive_expect_tx(v_full(st), bytes);
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(base + ok_v + hf * C::kHalf, &bvmap, v_full(st), hf * 64, h, s * sh.B + u0);
        } else {
          mbar_arrive(v_full(st));
        }
      } else {
        put(ok_v, cur.v, cur.vs, lp0, ph0);
        fence_proxy_async_smem();
        mbar_arrive(v_full(st));
      }
      cur = nxt;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        lp0[i] = lp1[i]; ph0[i] = ph1[i];
        lp1[i] = lp2[i]; ph1[i] = ph2[i];
      }
    }
    if (tid == 0) {  // copies in flight land before the CTA's shared memory is released
      for (int k = max(0, issued - ST); k < issued; ++k) {
        if (t0 + k < ks.pt) continue;
        mbar_wait(k_full(k % ST), (k / ST) & 1, drain_ctx);
        if (ok) mbar_wait(v_full(k % ST), (k / ST) & 1, drain_ctx);
      }
    }
  }

  // ---- join the groups and write the rows (or their share, for the merge)
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every MMA is done: Q, K and V are dead
  tc_fence_after();
  float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffML);
  if (warp >= 2 && warp < 10) ml[((warp - 2) >> 2) * 128 + (warp & 3) * 32 + lane] = make_float2(m_used, l);
  __syncthreads();
  if (warp >= 2 && warp < 10 && (warp & 3) < active_warps) {
    const int g = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lt = tmem + ((uint32_t)(quarter * 32) << 16) + C::kTmemO;
    const float2 x = ml[r], y = ml[128 + r];
    const bool hx = x.y != 0.f, hy = y.y != 0.f;  // a NaN sum counts as data
    const float M = fmaxf(hx ? x.x : -INFINITY, hy ? y.x : -INFINITY);
    const float M0 = M == -INFINITY ? 0.f : M;
    float wx = hx ? exp2f(x.x == -INFINITY ? 0.f : x.x - M0) : 0.f, wy = hy ? exp2f(y.x == -INFINITY ? 0.f : y.x - M0) : 0.f;
    const float L = (hx ? wx * x.y : 0.f) + (hy ? wy * y.y : 0.f);
    const bool warp_x = __any_sync(0xffffffffu, hx), warp_y = __any_sync(0xffffffffu, hy);
    const bool mine = r < rows;
    const size_t orow = ((size_t)s * sh.B + b0 + r / sh.G) * sh.Hq + (size_t)h * sh.G + r % sh.G;
    const size_t prow = ((size_t)unit * prm.splits + sp) * ((size_t)prm.bpt * sh.G) + r;
    const bool direct = prm.splits == 1;
    const float inv = L != 0.f ? 1.f / L : 0.f;
    if (mine && g == 0) {
      if (!direct) prm.part_ml[prow] = make_float2(M, L);
      if (direct && sh.lse_out)
        sh.lse_out[orow] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
    if (direct) {
      wx *= inv;
      wy *= inv;
    }
    for (int c0 = g * (D / 2); c0 < (g + 1) * (D / 2); c0 += 32) {  // each group half of the columns
      uint32_t u[32], v[32];
      if (warp_x && warp_y) {
        tmem_ld32x2(lt + c0, u, lt + D + c0, v);
      } else {
        if (warp_x) tmem_ld32(lt + c0, u);
        if (warp_y) tmem_ld32(lt + D + c0, v);
      }
      float o[32];
#pragma unroll
      for (int i = 0; i < 32; ++i)  // an accumulator without data is never touched
        o[i] = (hx ? wx * __uint_as_float(u[i]) : 0.f) + (hy ? wy * __uint_as_float(v[i]) : 0.f);
      if (mine && direct) {
        uint4 *dst = reinterpret_cast<uint4 *>(a.o_out + orow * D + c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                              pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
      } else if (mine && L != 0.f) {
        float4 *dst = reinterpret_cast<float4 *>(prm.part_o + prow * D + c0);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      __syncwarp();  // the TMEM loads are warp-collective
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the splits of each row: one warp per row, D/32 columns a lane.
constexpr int kMergeThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge(const __grid_constant__ Params prm) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const Shape &sh = prm.sh;
  const int lane = threadIdx.x & 31;
  const int rpt = prm.bpt * sh.G;  // rows of a unit
  const long long w = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int unit = (int)(w / rpt), r = (int)(w % rpt);
  const int rt = unit % prm.rowtiles, h = unit / prm.rowtiles % sh.Hkv, s = unit / prm.rowtiles / sh.Hkv;
  if (s >= sh.S) return;
  const int b = rt * prm.bpt + r / sh.G;
  if (b >= block_tokens(prm.a.n_new, s, sh.B, prm.a.status, false)) return;
  constexpr int E = D / 32;
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int sp = 0; sp < prm.splits; ++sp) {
    const size_t prow = ((size_t)unit * prm.splits + sp) * rpt + r;
    const float2 ml = prm.part_ml[prow];
    if (ml.y == 0.f) continue;  // no key, nothing written
    const float mn = fmaxf(M, ml.x);
    const float sc = M == -INFINITY ? 0.f : exp2f(M - mn), wt = ml.x == -INFINITY ? 1.f : exp2f(ml.x - mn);
    M = mn;
    L = fmaf(L, sc, wt * ml.y);
    const float *src = prm.part_o + prow * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], sc, wt * src[e]);
  }
  const size_t orow = ((size_t)s * sh.B + b) * sh.Hq + (size_t)h * sh.G + r % sh.G;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  uint32_t *dst = reinterpret_cast<uint32_t *>(prm.a.o_out + orow * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (sh.lse_out && lane == 0) sh.lse_out[orow] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
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

// Splits: the count whose waves of CTAs (one per SM) take the least time, a CTA
// costing its tiles plus a fixed part (set-up and epilogue), a split row the merge.
// The workspace holds the largest count a shape may get, whatever its window.
int max_splits(const Geometry &g, int sms) { return (int)std::max(1LL, std::min(64LL, 4LL * sms / g.units)); }
PagedPlan make_plan(const Shape &sh, int sms, long long max_tiles) {
  const Geometry g = geometry(sh);
  const int cap = max_splits(g, sms);
  PagedPlan p{1, 1, 0};
  long long best = -1;
  for (int sp = 1; sp <= cap && sp <= max_tiles; ++sp) {
    const long long waves = (g.units * sp + sms - 1) / sms;
    const long long cost = waves * ((max_tiles + sp - 1) / sp + 3) + (sp > 1 ? 2 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      p.splits = sp;
    }
  }
  p.launches = p.splits > 1 ? 2 : 1;
  p.total = kWorkspaceHeader;
  if (cap > 1) p.total += (size_t)g.units * cap * g.rows * ((size_t)sh.d * 4 + 8);
  return p;
}

template <int D, int PAGE, bool KV4>
cudaError_t launch_typed(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  using C = Cfg<D, KV4>;
  const Geometry g = geometry(sh);
  if (g.units * plan.splits > INT_MAX) return cudaErrorInvalidValue;
  Params prm{};
  prm.sh = sh;
  prm.a = a;
  prm.bpt = g.bpt;
  prm.rowtiles = g.rowtiles;
  prm.splits = plan.splits;
  prm.box_blk = std::min(kBN, (sh.B + 15) / 16 * 16);
  unsigned char *ws = reinterpret_cast<unsigned char *>(a.status) + kWorkspaceHeader;
  const size_t rows = (size_t)g.units * plan.splits * g.rows;
  prm.part_o = reinterpret_cast<float *>(ws);
  prm.part_ml = reinterpret_cast<float2 *>(ws + rows * D * 4);
  constexpr auto kern = paged_attn<D, PAGE, KV4>;
  cudaError_t err = set_smem_once<kern>(C::kAlloc);
  if (err != cudaSuccess) return err;
  CUtensorMap q{}, k{}, v{}, k4{}, v4{}, bk{}, bv{};
  const long long tokens = (long long)sh.S * sh.B;
  if ((err = make_q_tensor_map(&q, a.q, tokens, sh.Hq, D, sh.G, g.bpt)) != cudaSuccess) return err;
  if (!KV4) {
    const long long nrows = sh.n_phys * sh.Hkv * PAGE;
    if ((err = make_kv_tensor_map(&k, a.k, nrows, D, PAGE)) != cudaSuccess) return err;
    if ((err = make_kv_tensor_map(&v, a.v, nrows, D, PAGE)) != cudaSuccess) return err;
    if ((err = make_kv_pages_tensor_map(&k4, a.k, sh.n_phys, sh.Hkv, PAGE, D, kBN / PAGE)) != cudaSuccess) return err;
    if ((err = make_kv_pages_tensor_map(&v4, a.v, sh.n_phys, sh.Hkv, PAGE, D, kBN / PAGE)) != cudaSuccess) return err;
  }
  if (a.blk_k) {
    if ((err = make_blk_tensor_map(&bk, a.blk_k, tokens, sh.Hkv, D, prm.box_blk)) != cudaSuccess) return err;
    if ((err = make_blk_tensor_map(&bv, a.blk_v, tokens, sh.Hkv, D, prm.box_blk)) != cudaSuccess) return err;
  }
  err = launch_pdl(kern, dim3((unsigned)(g.units * plan.splits)), C::kThreads, C::kAlloc, stream, prm, q, k, v, k4, v4, bk, bv);
  if (err != cudaSuccess || plan.splits == 1) return err;
  const long long merge_rows = g.units * g.rows;
  return launch_pdl(paged_merge<D>, dim3((unsigned)((merge_rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32))),
                    kMergeThreads, 0, stream, prm);
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
  return make_plan(sh, num_sms, (reach + kBN - 1) / kBN);
}

PagedPlan plan_kv4(const Shape &sh, int num_sms, bool sparse) {
  const long long prefix = (long long)(sparse ? std::min(sh.kmax, sh.max_pages) : sh.max_pages) * sh.P;
  return make_plan(sh, num_sms, (prefix + kBN - 1) / kBN + (sh.B + kBN - 1) / kBN);
}

cudaError_t launch_window(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  return launch_any<false>(sh, plan, a, stream);
}
cudaError_t launch_kv4_attn(const Shape &sh, const PagedPlan &plan, const PagedArgs &a, cudaStream_t stream) {
  return launch_any<true>(sh, plan, a, stream);
}

}  // namespace dsa
