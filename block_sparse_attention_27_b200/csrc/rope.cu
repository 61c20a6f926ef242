// rope.cu -- dsa_qk_norm_rope: the norm of each head's query and key, the rotation
// by position and the append to the paged cache in one pass over the projections.
//
// D / 2V lanes hold one head's row, 2V values each (V = 4 or 8): for the half layout the values
// [V l, V l + V) and their partners [rot/2 + V l, ..), for the interleaved one 2V consecutive
// values; lanes past the rotated part hold the values from rot on.  So a rotation needs no
// exchange between lanes, and the mean square is one shuffle reduction.  cos and sin of a
// token's rot/2 angles are computed once per CTA into shared memory: the angle in turns in
// fp64 (positions of long contexts lose the fast pairs in fp32), reduced to half a turn, then
// sincospi in fp32.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kRopeThreads = 256;

template <int V>  // V bf16 values in one load
struct Halves;
template <>
struct Halves<4> { using type = uint2; };
template <>
struct Halves<8> { using type = uint4; };

template <int V>
__device__ __forceinline__ void unpack(const typename Halves<V>::type &lo, const typename Halves<V>::type &hi, float2 (&x)[V]) {
  const __nv_bfloat162 *u = reinterpret_cast<const __nv_bfloat162 *>(&lo), *v = reinterpret_cast<const __nv_bfloat162 *>(&hi);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    x[j] = __bfloat1622float2(u[j]);
    x[V / 2 + j] = __bfloat1622float2(v[j]);
  }
}

template <int V>
__device__ __forceinline__ typename Halves<V>::type pack(const float2 *x) {
  typename Halves<V>::type y;
  uint32_t *p = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) p[j] = pack_bf16x2(x[j].x, x[j].y);
  return y;
}

// A CTA takes TT tokens, or some of the passes over their rows: queries, keys and values each
// in passes of kRows rows (token, head), so that a pass knows its pointers, its weights and
// whether it rotates.  A prompt is bound by the latency of its loads and the instructions
// between them: 28K tokens of 28 + 4 heads took 142 us with the kinds mixed in one loop, 115
// with 2 x 4 values a lane and four tokens a CTA, 98 with 2 x 8 values, packed fp32 arithmetic
// and eight tokens (the floor is 70).  Four CTAs an SM (64 registers);
// three take 110 us, five spill and take 119, weights read from shared memory 124.
template <int D, bool INTERLEAVED, int TT, int V>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope(const Shape sh, const RopeArgs a, int passes_per_cta) {
  constexpr int kLanes = D / (2 * V);          // lanes of a row
  constexpr int kRows = kRopeThreads / kLanes;  // rows of a pass
  using Vec = typename Halves<V>::type;
  __shared__ __align__(16) float cosines[TT][D / 2], sines[TT][D / 2];
  __shared__ long long crow_of[TT];  // the token's row of head 0 in the cache (head h is h * P further), -1: none
  __shared__ int live[TT];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const int t0 = blockIdx.x * TT, tokens = min(TT, sh.S * sh.B - t0);
  for (int e = threadIdx.x; e < TT * (D / 2); e += kRopeThreads) {
    const int i = e / (D / 2), f = e % (D / 2), t = t0 + i;
    const bool in = i < tokens;
    const int s = in ? t / sh.B : 0, b = t - s * sh.B;
    if (f == 0) {
      int on = in && b < block_tokens(a.n_new, s, sh.B, a.status, in && b == 0 && blockIdx.y == 0);
      long long row = -1;
      if (on && (a.k_cache || a.v_cache)) {
        const int n = a.n_ctx[s];
        const long long at = (long long)n + b, phys = n < 0 ? -1 : physical_page(sh, s, at / sh.P);
        if (phys >= 0)
          row = phys * sh.Hkv * sh.P + at % sh.P;
        else if (blockIdx.y == 0)
          raise_status(a.status, kStatusBadIndex);
      }
      live[i] = on;
      crow_of[i] = row;
    }
    if (in && f < a.rot / 2) {
      const int pos = a.positions ? a.positions[t] : a.n_ctx[s] + b;
      double turns = (double)pos * (double)a.inv_freq[f] * 0.15915494309189533577;
      turns -= rint(turns);
      float sn, cn;
      sincospif((float)(2.0 * turns), &sn, &cn);
      cosines[i][f] = cn * a.scale;
      sines[i][f] = sn * a.scale;
    }
  }
  __syncthreads();
  const int l = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int turn = a.rot / (2 * V);  // lanes that rotate
  const int e0 = INTERLEAVED || l >= turn ? 2 * V * l : V * l;
  const int e1 = INTERLEAVED || l >= turn ? 2 * V * l + V : a.rot / 2 + V * l;
  const bool turns = l < turn;
  int done = 0;  // passes of the kinds before
  const int from = blockIdx.y * passes_per_cta, to = from + passes_per_cta;
  auto head_of = [&](int row, int heads, int &i) {  // row = token i of the CTA, head
    i = 0;
#pragma unroll
    for (int k = 1; k < TT; ++k) i += row >= k * heads;
    return row - i * heads;
  };
  auto kind = [&](int heads, const __nv_bfloat16 *in, long long stride, const __nv_bfloat16 *wt, __nv_bfloat16 *out,
                  __nv_bfloat16 *cache) {
    const int rows = tokens * heads, passes = (TT * heads + kRows - 1) / kRows;
    const int p0 = max(0, from - done), p1 = min(passes, to - done);
    done += passes;
    if (p0 >= p1) return;
    float2 w[V];
    if (wt) unpack<V>(*reinterpret_cast<const Vec *>(wt + e0), *reinterpret_cast<const Vec *>(wt + e1), w);
    Vec lo, hi;
    int i, h;
    bool on;
    auto load = [&](int p) {
      const int row = p * kRows + row0;
      h = head_of(row, heads, i);
      on = p < p1 && row < rows && live[i];
      lo = hi = Vec{};
      if (!on) return;
      const __nv_bfloat16 *src = in + (t0 + i) * stride + h * D;
      lo = *reinterpret_cast<const Vec *>(src + e0);
      hi = *reinterpret_cast<const Vec *>(src + e1);
    };
    load(p0);
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {  // whole warps: the reduction is a warp shuffle
      float2 x[V];
      unpack<V>(lo, hi, x);
      const int ic = i, hc = h;
      const bool was = on;
      load(p + 1);
      if (wt) {
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < V; ++j) sq = sm100::fma2(x[j], x[j], sq);
        float ss = sq.x + sq.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = sm100::mul2(x[j], sm100::mul2(w[j], inv2));
      }
      if (!was) continue;
      if (turns) {
        // angles V l .. V l + V - 1: of the half layout's pairs (x[j], x[V/2 + j]) two a step
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          const float4 c = *reinterpret_cast<const float4 *>(&cosines[ic][V * l + 4 * j]);
          const float4 n = *reinterpret_cast<const float4 *>(&sines[ic][V * l + 4 * j]);
          if constexpr (INTERLEAVED) {
            const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 u = x[4 * j + k];
              x[4 * j + k] = make_float2(u.x * cc[k] - u.y * nn[k], u.y * cc[k] + u.x * nn[k]);
            }
          } else {
            const float2 cc[2] = {{c.x, c.y}, {c.z, c.w}}, nn[2] = {{n.x, n.y}, {n.z, n.w}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 u = x[2 * j + k], v = x[V / 2 + 2 * j + k];
              x[2 * j + k] = sm100::fma2(u, cc[k], sm100::mul2(v, make_float2(-nn[k].x, -nn[k].y)));
              x[V / 2 + 2 * j + k] = sm100::fma2(v, cc[k], sm100::mul2(u, nn[k]));
            }
          }
        }
      }
      const Vec y0 = pack<V>(x), y1 = pack<V>(x + V / 2);
      if (out) {
        __nv_bfloat16 *dst = out + (long long)((t0 + ic) * heads + hc) * D;
        *reinterpret_cast<Vec *>(dst + e0) = y0;
        *reinterpret_cast<Vec *>(dst + e1) = y1;
      }
      if (cache && crow_of[ic] >= 0) {
        __nv_bfloat16 *dst = cache + (crow_of[ic] + hc * sh.P) * D;
        *reinterpret_cast<Vec *>(dst + e0) = y0;
        *reinterpret_cast<Vec *>(dst + e1) = y1;
      }
    }
  };
  if (a.q) kind(sh.Hq, a.q, a.q_stride, a.q_norm, a.q_out, nullptr);
  if (a.k) kind(sh.Hkv, a.k, a.k_stride, a.k_norm, a.k_out, a.k_cache);
  if (!a.v) return;
  // values: copied bit for bit, 16 bytes a load
  const int passes = (TT * sh.Hkv + kRows - 1) / kRows;
  for (int p = max(0, from - done); p < min(passes, to - done); ++p) {
    const int row = p * kRows + row0;
    int i;
    const int h = head_of(row, sh.Hkv, i);
    if (row >= tokens * sh.Hkv || !live[i]) continue;
    const __nv_bfloat16 *src = a.v + (t0 + i) * a.v_stride + h * D + 8 * l;
    __nv_bfloat16 *out = a.v_out ? a.v_out + (long long)((t0 + i) * sh.Hkv + h) * D + 8 * l : nullptr;
    __nv_bfloat16 *cache = a.v_cache && crow_of[i] >= 0 ? a.v_cache + (crow_of[i] + h * sh.P) * D + 8 * l : nullptr;
    uint4 y[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) y[j] = *reinterpret_cast<const uint4 *>(src + j * 8 * kLanes);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      if (out) *reinterpret_cast<uint4 *>(out + j * 8 * kLanes) = y[j];
      if (cache) *reinterpret_cast<uint4 *>(cache + j * 8 * kLanes) = y[j];
    }
  }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_d(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  constexpr int TT = 8;
  const long long tokens = (long long)sh.S * sh.B;
  auto passes = [&](int tt, int v) {
    const int rows = kRopeThreads / (D / (2 * v));
    auto of = [&](const void *in, int heads) { return in ? (tt * heads + rows - 1) / rows : 0; };
    return of(a.q, sh.Hq) + of(a.k, sh.Hkv) + of(a.v, sh.Hkv);
  };
  // Few tokens: a CTA per pass of one token, four values twice a lane.  More: eight tokens share
  // the angles and fill the passes, eight values twice a lane (16-byte loads; four where rot/2 is
  // no multiple of eight), and a CTA takes more than one pass once the SMs have three CTAs each.
  // 28 + 4 heads, single tokens against eight: 128 tokens 3.4 us against 3.9, 256 tokens 5.3
  // against 4.2, 4096 tokens 58 against 16.  All passes in one CTA: 512 tokens 8.2 us against 5.5;
  // one pass a CTA: 4096 tokens 32 against 16.
  if (tokens >= 148) {
    const int v = a.rot % 16 == 0 ? 8 : 4, all = passes(TT, v);
    const long long groups = (tokens + TT - 1) / TT;
    const int each = (int)min((long long)all, max(1LL, groups * all / (3 * 148)));
    const dim3 grid((unsigned)groups, (unsigned)((all + each - 1) / each));
    return v == 8 ? launch_pdl(qk_norm_rope<D, INTERLEAVED, TT, 8>, grid, kRopeThreads, 0, stream, sh, a, each)
                  : launch_pdl(qk_norm_rope<D, INTERLEAVED, TT, 4>, grid, kRopeThreads, 0, stream, sh, a, each);
  }
  return launch_pdl(qk_norm_rope<D, INTERLEAVED, 1, 4>, dim3((unsigned)tokens, (unsigned)passes(1, 4)), kRopeThreads, 0,
                    stream, sh, a, 1);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  if (sh.d == 128) return a.interleaved ? launch_d<128, true>(sh, a, stream) : launch_d<128, false>(sh, a, stream);
  return a.interleaved ? launch_d<64, true>(sh, a, stream) : launch_d<64, false>(sh, a, stream);
}

}  // namespace dsa
