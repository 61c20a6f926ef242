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

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope(const Shape sh, const RopeArgs a, int rows_per_cta) {
  constexpr int kLanes = D / 8;               // lanes of a row
  constexpr int kRows = kRopeThreads / kLanes;  // rows of a pass
  __shared__ float2 cs[D / 2];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const int t = blockIdx.x;  // token
  const int s = t / sh.B, b = t % sh.B;
  if (b >= block_tokens(a.n_new, s, sh.B, a.status, b == 0 && blockIdx.y == 0 && threadIdx.x == 0)) return;
  const int pos = a.positions ? a.positions[t] : a.n_ctx[s] + b;
  if (threadIdx.x < a.rot / 2) {
    double turns = (double)pos * (double)a.inv_freq[threadIdx.x] * 0.15915494309189533577;
    turns -= rint(turns);
    float sn, cn;
    sincospif((float)(2.0 * turns), &sn, &cn);
    cs[threadIdx.x] = make_float2(cn * a.scale, sn * a.scale);
  }
  // the token's row in the cache
  long long crow = -1;  // row of head 0; head h is h * P further
  if (a.k_cache || a.v_cache) {
    const long long at = (long long)a.n_ctx[s] + b;
    const long long phys = a.n_ctx[s] < 0 ? -1 : physical_page(sh, s, at / sh.P);
    if (phys >= 0)
      crow = phys * sh.Hkv * sh.P + at % sh.P;
    else if (blockIdx.y == 0 && threadIdx.x == 0)
      raise_status(a.status, kStatusBadIndex);
  }
  __syncthreads();
  const int l = threadIdx.x % kLanes;
  const int turn = a.rot / 8;  // lanes that rotate
  const int e0 = INTERLEAVED || l >= turn ? 8 * l : 4 * l;
  const int e1 = INTERLEAVED || l >= turn ? 8 * l + 4 : a.rot / 2 + 4 * l;
  const int nq = a.q ? sh.Hq : 0, nk = a.k ? sh.Hkv : 0, nv = a.v ? sh.Hkv : 0;
  const int r1 = min(nq + nk + nv, (int)(blockIdx.y + 1) * rows_per_cta);
  // whole warps stay in the loop: the reduction below is a warp shuffle
  for (int r0 = blockIdx.y * rows_per_cta; r0 < r1; r0 += kRows) {
    const int r = r0 + threadIdx.x / kLanes;
    if (r0 + (int)(threadIdx.x & ~31) / kLanes >= r1) break;
    const bool on = r < r1;
    const int kind = r < nq ? 0 : r < nq + nk ? 1 : 2;
    const int h = kind == 0 ? r : kind == 1 ? r - nq : r - nq - nk;
    const __nv_bfloat16 *src = kind == 0   ? a.q + (long long)t * a.q_stride
                               : kind == 1 ? a.k + (long long)t * a.k_stride
                                           : a.v + (long long)t * a.v_stride;
    uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
    if (on) {
      lo = *reinterpret_cast<const uint2 *>(src + (long long)h * D + e0);
      hi = *reinterpret_cast<const uint2 *>(src + (long long)h * D + e1);
    }
    const __nv_bfloat16 *w = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    float x[8];
    {
      const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&lo);
      const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(&hi);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = __bfloat1622float2(p[i]), g = __bfloat1622float2(q[i]);
        x[2 * i] = f.x; x[2 * i + 1] = f.y;
        x[4 + 2 * i] = g.x; x[5 + 2 * i] = g.y;
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!on) continue;
    if (w) {
      const float inv = rsqrtf(ss * (1.f / D) + a.eps);
      const uint2 wl = *reinterpret_cast<const uint2 *>(w + e0), wh = *reinterpret_cast<const uint2 *>(w + e1);
      const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&wl);
      const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(&wh);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = __bfloat1622float2(p[i]), g = __bfloat1622float2(q[i]);
        x[2 * i] *= inv * f.x; x[2 * i + 1] *= inv * f.y;
        x[4 + 2 * i] *= inv * g.x; x[5 + 2 * i] *= inv * g.y;
      }
    }
    if (kind < 2 && l < turn) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = cs[4 * l + i];
        float &p = INTERLEAVED ? x[2 * i] : x[i], &q = INTERLEAVED ? x[2 * i + 1] : x[4 + i];
        const float u = p * c.x - q * c.y, v = q * c.x + p * c.y;
        p = u;
        q = v;
      }
    }
    if (kind < 2) {  // values are copied bit for bit
      lo = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      hi = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    __nv_bfloat16 *out = kind == 0   ? a.q_out + ((long long)t * sh.Hq + h) * D
                         : kind == 1 ? (a.k_out ? a.k_out + ((long long)t * sh.Hkv + h) * D : nullptr)
                                     : (a.v_out ? a.v_out + ((long long)t * sh.Hkv + h) * D : nullptr);
    if (out) {
      *reinterpret_cast<uint2 *>(out + e0) = lo;
      *reinterpret_cast<uint2 *>(out + e1) = hi;
    }
    __nv_bfloat16 *cache = kind == 1 ? a.k_cache : kind == 2 ? a.v_cache : nullptr;
    if (cache && crow >= 0) {
      cache += (crow + (long long)h * sh.P) * D;
      *reinterpret_cast<uint2 *>(cache + e0) = lo;
      *reinterpret_cast<uint2 *>(cache + e1) = hi;
    }
  }
}

template <int D>
cudaError_t launch_d(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  constexpr int kRows = kRopeThreads / (D / 8);
  const int rows = (a.q ? sh.Hq : 0) + (a.k ? sh.Hkv : 0) + (a.v ? sh.Hkv : 0);
  const long long tokens = (long long)sh.S * sh.B;
  const int chunks = (rows + kRows - 1) / kRows;
  const dim3 grid((unsigned)tokens, (unsigned)chunks, 1);
  return a.interleaved ? launch_pdl(qk_norm_rope<D, true>, grid, kRopeThreads, 0, stream, sh, a, kRows)
                       : launch_pdl(qk_norm_rope<D, false>, grid, kRopeThreads, 0, stream, sh, a, kRows);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const Shape &sh, const RopeArgs &a, cudaStream_t stream) {
  return sh.d == 128 ? launch_d<128>(sh, a, stream) : launch_d<64>(sh, a, stream);
}

}  // namespace dsa
