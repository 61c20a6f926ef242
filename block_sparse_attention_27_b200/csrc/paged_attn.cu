// paged_attn.cu -- dsa_window_attn and dsa_kv4_attn: softmax attention of a block's
// queries over a paged cache, in bf16 with a sliding window and sinks or in 4 bits,
// and over the block's own tokens.
//
// One warp per query row; a lane holds D/32 elements of the query and the output.
// One pass over the visible keys with the running maximum and sum of the softmax.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kRowThreads = 256;

struct RowState {
  float m = -INFINITY, l = 0.f;
};

template <int D, bool KV4>
__global__ void __launch_bounds__(kRowThreads) paged_attn(const Shape sh, const PagedArgs a) {
  constexpr int E = D / 32;  // elements of a lane
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);  // (s, b, hq)
  if (row >= (long long)sh.S * sh.B * sh.Hq) return;
  const int hq = (int)(row % sh.Hq);
  const long long t = row / sh.Hq;
  const int s = (int)(t / sh.B), b = (int)(t % sh.B), h = hq / sh.G;
  const bool lead = lane == 0 && b == 0;
  const int nb = block_tokens(a.n_new, s, sh.B, a.status, lead && hq == 0);
  if (b >= nb) return;
  const int n = clamp_prefix(a.n_ctx[s], sh.max_pages, sh.P, a.status, lead && hq == 0);
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[row * D + lane * E + e]) * sh.sl2;
    o[e] = 0.f;
  }
  RowState st;
  auto key = [&](const float (&k)[E], const float (&v)[E]) {
    float x = 0.f;
    for (int e = 0; e < E; ++e) x = fmaf(q[e], k[e], x);
    x = warp_sum(x);
    const float m = fmaxf(st.m, x);
    const float al = st.m == -INFINITY ? 0.f : exp2f(st.m - m), p = exp2f(x - m);
    st.m = m;
    st.l = fmaf(st.l, al, p);
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], al, p * v[e]);
  };
  const long long pos = (long long)n + b;
  auto seen = [&](long long j) {
    if (KV4) return true;
    const long long gap = pos > j ? pos - j : j - pos;
    return (j < a.sinks || gap < a.window) && (!a.causal || j <= pos);
  };
  auto page = [&](int lp, int j0, int j1) {
    const long long phys = physical_page(sh, s, lp);
    if (phys < 0) {
      if (lane == 0) raise_status(a.status, kStatusBadIndex);
      return;
    }
    for (int j = j0; j < j1; ++j) {
      if (!seen(j)) continue;
      const long long r = (phys * sh.Hkv + h) * sh.P + (j - lp * sh.P);
      float k[E], v[E];
      for (int e = 0; e < E; ++e) {
        const int x = lane * E + e;
        if constexpr (KV4) {
          const int sft = 4 * ((x % 8) >> 1) + 16 * (x & 1);
          const uint32_t wk = reinterpret_cast<const uint32_t *>(a.kv4.k + r * (D / 2))[x / 8];
          const uint32_t wv = reinterpret_cast<const uint32_t *>(a.kv4.v + r * (D / 2))[x / 8];
          k[e] = (float)((int)((wk >> sft) & 15u) - 8) * __bfloat162float(a.kv4.ks[r * (D / kKv4Group) + x / kKv4Group]);
          v[e] = (float)((int)((wv >> sft) & 15u) - 8) * __bfloat162float(a.kv4.vs[r * (D / kKv4Group) + x / kKv4Group]);
        } else {
          k[e] = __bfloat162float(a.k[r * D + x]);
          v[e] = __bfloat162float(a.v[r * D + x]);
        }
      }
      key(k, v);
    }
  };
  if (KV4 && a.idx) {
    const int32_t *idx = a.idx + ((size_t)s * sh.Hkv + h) * sh.kmax;
    int cnt = a.idx_cnt[(size_t)s * sh.Hkv + h];
    if (cnt < 0 || cnt > sh.kmax) {
      if (lane == 0) raise_status(a.status, kStatusBadIndex);
      cnt = max(0, min(cnt, sh.kmax));
    }
    for (int i = 0; i < cnt; ++i) {
      const int lp = idx[i];
      if (lp < 0 || lp >= (n + sh.P - 1) / sh.P) {
        if (lane == 0) raise_status(a.status, kStatusBadIndex);
        continue;
      }
      page(lp, lp * sh.P, min(n, (lp + 1) * sh.P));
    }
  } else {
    const long long low = KV4 ? 0 : max(0LL, pos - a.window + 1);
    const int sinks = KV4 ? 0 : (int)min((long long)a.sinks, min(low, (long long)n));
    for (int lp = 0; lp * sh.P < sinks; ++lp) page(lp, lp * sh.P, min(sinks, (lp + 1) * sh.P));
    for (int lp = (int)(low / sh.P); lp * sh.P < n; ++lp) page(lp, (int)max((long long)lp * sh.P, low), min(n, (lp + 1) * sh.P));
  }
  if (a.blk_k) {
    for (int u = 0; u < nb; ++u) {
      if (!seen((long long)n + u)) continue;
      const size_t r = (((size_t)s * sh.B + u) * sh.Hkv + h) * D + lane * E;
      float k[E], v[E];
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(a.blk_k[r + e]);
        v[e] = __bfloat162float(a.blk_v[r + e]);
      }
      key(k, v);
    }
  }
  const float inv = st.l > 0.f ? 1.f / st.l : 0.f;
  for (int e = 0; e < E; ++e) a.o_out[row * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
  if (sh.lse_out && lane == 0) sh.lse_out[row] = st.l > 0.f ? (st.m + log2f(st.l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool KV4>
cudaError_t launch_rows(const Shape &sh, const PagedArgs &a, cudaStream_t stream) {
  const long long rows = (long long)sh.S * sh.B * sh.Hq;
  return launch_pdl(paged_attn<D, KV4>, dim3((unsigned)((rows + kRowThreads / 32 - 1) / (kRowThreads / 32))), kRowThreads, 0,
                    stream, sh, a);
}

}  // namespace

PagedPlan plan_window(const Shape &, int, int, int) { return PagedPlan{1, 1, kWorkspaceHeader}; }
PagedPlan plan_kv4(const Shape &, int, bool) { return PagedPlan{1, 1, kWorkspaceHeader}; }

cudaError_t launch_window(const Shape &sh, const PagedPlan &, const PagedArgs &a, cudaStream_t stream) {
  return sh.d == 128 ? launch_rows<128, false>(sh, a, stream) : launch_rows<64, false>(sh, a, stream);
}
cudaError_t launch_kv4_attn(const Shape &sh, const PagedPlan &, const PagedArgs &a, cudaStream_t stream) {
  return sh.d == 128 ? launch_rows<128, true>(sh, a, stream) : launch_rows<64, true>(sh, a, stream);
}

}  // namespace dsa
