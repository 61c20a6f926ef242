// rope.cu -- dsa_qk_norm_rope: the norm of each head's query and key, the rotation
// by position and the append to the paged cache in one pass over the projections.
//
// D/8 lanes hold one head's row, eight values each: for the half layout the values
// [4l, 4l+4) and their partners [rot/2 + 4l, ..), for the interleaved one eight
// consecutive values; lanes past the rotated part hold the values from rot on.  So a
// rotation needs no exchange between lanes, and the mean square is one shuffle
// reduction.  cos and sin of a token's rot/2 angles are computed once per CTA into
// shared memory: the angle in turns in fp64 (positions of long contexts lose the
// fast pairs in fp32), reduced to half a turn, then sincospi in fp32.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kRopeThreads = 256;

// A CTA takes TT tokens, or some of the passes over the rows of one: queries, keys and
// values each in passes of kRows rows (token, head), so that a pass knows its pointers, its
// weights and whether it rotates.  The kernel is bound by its instructions as soon as they
// are many (229 a row pair with the three kinds mixed in one loop: 142 us for 28K tokens).
template <int D, bool INTERLEAVED, int TT>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope(const Shape sh, const RopeArgs a, int passes_per_cta) {
  constexpr int kLanes = D / 8;                // lanes of a row
  constexpr int kRows = kRopeThreads / kLanes;  // rows of a pass
  __shared__ __align__(16) float2 cs[TT][D / 2];
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
      cs[i][f] = make_float2(cn * a.scale, sn * a.scale);
    }
  }
  __syncthreads();
  const int l = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int turn = a.rot / 8;  // lanes that rotate
  const int e0 = INTERLEAVED || l >= turn ? 8 * l : 4 * l;
  const int e1 = INTERLEAVED || l >= turn ? 8 * l + 4 : a.rot / 2 + 4 * l;
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
    float w[8];
    if (wt) {
      const uint2 w0 = *reinterpret_cast<const uint2 *>(wt + e0), w1 = *reinterpret_cast<const uint2 *>(wt + e1);
      const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&w0);
      const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(&w1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 f = __bfloat1622float2(p[j]), g = __bfloat1622float2(q[j]);
        w[2 * j] = f.x; w[2 * j + 1] = f.y;
        w[4 + 2 * j] = g.x; w[5 + 2 * j] = g.y;
      }
    }
    uint2 lo, hi;
    int i, h;
    bool on;
    auto load = [&](int p) {
      const int row = p * kRows + row0;
      h = head_of(row, heads, i);
      on = p < p1 && row < rows && live[i];
      lo = hi = make_uint2(0, 0);
      if (!on) return;
      const __nv_bfloat16 *src = in + (t0 + i) * stride + h * D;
      lo = *reinterpret_cast<const uint2 *>(src + e0);
      hi = *reinterpret_cast<const uint2 *>(src + e1);
    };
    load(p0);
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {  // whole warps: the reduction is a warp shuffle
      float x[8];
      {
        const __nv_bfloat162 *u = reinterpret_cast<const __nv_bfloat162 *>(&lo);
        const __nv_bfloat162 *v = reinterpret_cast<const __nv_bfloat162 *>(&hi);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = __bfloat1622float2(u[j]), g = __bfloat1622float2(v[j]);
          x[2 * j] = f.x; x[2 * j + 1] = f.y;
          x[4 + 2 * j] = g.x; x[5 + 2 * j] = g.y;
        }
      }
      const int ic = i, hc = h;
      const bool was = on;
      load(p + 1);
      if (wt) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= inv * w[j];
      }
      if (!was) continue;
      if (turns) {
        const float4 *c4 = reinterpret_cast<const float4 *>(&cs[ic][4 * l]);
        const float4 ca = c4[0], cb = c4[1];
        const float2 c[4] = {{ca.x, ca.y}, {ca.z, ca.w}, {cb.x, cb.y}, {cb.z, cb.w}};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float &u = INTERLEAVED ? x[2 * j] : x[j], &v = INTERLEAVED ? x[2 * j + 1] : x[4 + j];
          const float s = u * c[j].x - v * c[j].y, t = v * c[j].x + u * c[j].y;
          u = s;
          v = t;
        }
      }
      const uint2 y0 = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      const uint2 y1 = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      if (out) {
        __nv_bfloat16 *dst = out + (long long)((t0 + ic) * heads + hc) * D;
        *reinterpret_cast<uint2 *>(dst + e0) = y0;
        *reinterpret_cast<uint2 *>(dst + e1) = y1;
      }
      if (cache && crow_of[ic] >= 0) {
        __nv_bfloat16 *dst = cache + (crow_of[ic] + hc * sh.P) * D;
        *reinterpret_cast<uint2 *>(dst + e0) = y0;
        *reinterpret_cast<uint2 *>(dst + e1) = y1;
      }
    }
  };
  if (a.q) kind(sh.Hq, a.q, a.q_stride, a.q_norm, a.q_out, nullptr);
  if (a.k) kind(sh.Hkv, a.k, a.k_stride, a.k_norm, a.k_out, a.k_cache);
  if (!a.v) return;
  // values: copied bit for bit, 16 bytes a lane
  const int passes = (TT * sh.Hkv + kRows - 1) / kRows;
  for (int p = max(0, from - done); p < min(passes, to - done); ++p) {
    const int row = p * kRows + row0;
    int i;
    const int h = head_of(row, sh.Hkv, i);
    if (row >= tokens * sh.Hkv || !live[i]) continue;
    const uint4 y = *reinterpret_cast<const uint4 *>(a.v + (t0 + i) * a.v_stride + h * D + 8 * l);
    if (a.v_out) *reinterpret_cast<uint4 *>(a.v_out + (long long)((t0 + i) * sh.Hkv + h) * D + 8 * l) = y;
    if (a.v_cache && crow_of[i] >= 0) *reinterpret_cast<uint4 *>(a.v_cache + (crow_of[i] + h * sh.P) * D + 8 * l) = y;
  }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_d(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  constexpr int kRows = kRopeThreads / (D / 8);
  constexpr int TT = 4;
  const long long tokens = (long long)sh.S * sh.B;
  auto passes = [&](int tt) {
    auto of = [&](const void *in, int heads) { return in ? (tt * heads + kRows - 1) / kRows : 0; };
    return of(a.q, sh.Hq) + of(a.k, sh.Hkv) + of(a.v, sh.Hkv);
  };
  // Few tokens: a CTA per pass, so that many SMs share one step's block.  Many: four tokens a
  // CTA with all their passes (the angles once, the last pass of each kind fuller).
  if (tokens >= TT * 4 * 148)
    return launch_pdl(qk_norm_rope<D, INTERLEAVED, TT>, dim3((unsigned)((tokens + TT - 1) / TT)), kRopeThreads, 0, stream, sh, a,
                      passes(TT));
  return launch_pdl(qk_norm_rope<D, INTERLEAVED, 1>, dim3((unsigned)tokens, (unsigned)passes(1)), kRopeThreads, 0, stream, sh, a, 1);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  if (sh.d == 128) return a.interleaved ? launch_d<128, true>(sh, a, stream) : launch_d<128, false>(sh, a, stream);
  return a.interleaved ? launch_d<64, true>(sh, a, stream) : launch_d<64, false>(sh, a, stream);
}

}  // namespace dsa
