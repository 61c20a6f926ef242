// kv4.cu -- dsa_kv4_store and dsa_kv4_load: rows into and out of the 4-bit cache.
// Four lanes hold a group of 32 values, eight each: one packed word per lane.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kKv4Threads = 256;

// Scale of a group whose largest magnitude is amax: the smallest number of five
// significant bits that is at least amax / 7.  A true division: a product with 1/7
// would push exact multiples of 7 over their border.
__device__ __forceinline__ float kv4_scale(float amax) {
  if (!(amax < 1.329227996e36f)) return __int_as_float(0x7fc00000);  // 2^120 or more, or NaN
  if (amax < 7.888609052e-31f) return 0.f;                           // 2^-100
  return __uint_as_float((__float_as_uint(__fdiv_rn(amax, 7.f)) + 0x7ffffu) & ~0x7ffffu);
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads)
    kv4_store(const Shape sh, const Kv4 c, const __nv_bfloat16 *__restrict__ k, const __nv_bfloat16 *__restrict__ v,
              const int32_t *__restrict__ n_ctx, const int32_t *__restrict__ n_new, uint32_t *status) {
  constexpr int kLanes = D / 8;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const long long item = (long long)blockIdx.x * (kKv4Threads / kLanes) + threadIdx.x / kLanes;  // (token, k|v, head)
  const int l = threadIdx.x % kLanes;
  const long long t = item / (2 * sh.Hkv);
  const int r = (int)(item % (2 * sh.Hkv));
  const bool isv = r >= sh.Hkv;
  const int h = isv ? r - sh.Hkv : r;
  bool on = t < (long long)sh.S * sh.B;
  long long row = 0;
  if (on) {
    const int s = (int)(t / sh.B), b = (int)(t % sh.B);
    on = b < block_tokens(n_new, s, sh.B, status, b == 0 && r == 0 && l == 0);
    if (on) {
      const int n = n_ctx[s];
      const long long phys = n < 0 ? -1 : physical_page(sh, s, ((long long)n + b) / sh.P);
      if (phys < 0) {
        if (r == 0 && l == 0) raise_status(status, kStatusBadIndex);
        on = false;
      } else {
        row = (phys * sh.Hkv + h) * sh.P + (n + b) % sh.P;
      }
    }
  }
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (on) raw = *reinterpret_cast<const uint4 *>((isv ? v : k) + (t * sh.Hkv + h) * D + 8 * l);
  float x[8];
  const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(p[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(x[i]));
    bad |= x[i] != x[i];
  }
  if (bad) amax = INFINITY;  // fmaxf drops NaN
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const float s = kv4_scale(amax);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q = 8.f;
    if (s > 0.f) q += fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f);
    w |= (uint32_t)q << (4 * (i >> 1) + 16 * (i & 1));
  }
  if (!on) return;
  *reinterpret_cast<uint32_t *>((isv ? c.v : c.k) + row * (D / 2) + 4 * l) = w;
  if (l % 4 == 0) (isv ? c.vs : c.ks)[row * (D / kKv4Group) + l / 4] = __float2bfloat16_rn(s);
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads)
    kv4_load(const Shape sh, const Kv4 c, __nv_bfloat16 *__restrict__ k, __nv_bfloat16 *__restrict__ v,
             const int32_t *__restrict__ start, const int32_t *__restrict__ n_new, uint32_t *status) {
  constexpr int kLanes = D / 8;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const long long item = (long long)blockIdx.x * (kKv4Threads / kLanes) + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  const long long t = item / (2 * sh.Hkv);
  const int r = (int)(item % (2 * sh.Hkv));
  const bool isv = r >= sh.Hkv;
  const int h = isv ? r - sh.Hkv : r;
  if (t >= (long long)sh.S * sh.B) return;
  const int s = (int)(t / sh.B), b = (int)(t % sh.B);
  const bool lead = r == 0 && l == 0;
  if (b >= block_tokens(n_new, s, sh.B, status, lead && b == 0)) return;
  const int n = start[s];
  const long long phys = n < 0 ? -1 : physical_page(sh, s, ((long long)n + b) / sh.P);
  if (phys < 0) {
    if (lead) raise_status(status, kStatusBadIndex);
    return;
  }
  const long long row = (phys * sh.Hkv + h) * sh.P + (n + b) % sh.P;
  const uint32_t w = *reinterpret_cast<const uint32_t *>((isv ? c.v : c.k) + row * (D / 2) + 4 * l);
  __nv_bfloat162 s8, m24;
  kv4_constants((isv ? c.vs : c.ks)[row * (D / kKv4Group) + l / 4], s8, m24);
  *reinterpret_cast<uint4 *>((isv ? v : k) + (t * sh.Hkv + h) * D + 8 * l) =
      make_uint4(kv4_pair(w, 0, s8, m24), kv4_pair(w, 1, s8, m24), kv4_pair(w, 2, s8, m24), kv4_pair(w, 3, s8, m24));
}

template <int D>
unsigned rows_grid(const Shape &sh) {
  constexpr int kRows = kKv4Threads / (D / 8);
  return (unsigned)(((long long)sh.S * sh.B * 2 * sh.Hkv + kRows - 1) / kRows);
}

}  // namespace

cudaError_t launch_kv4_store(const Shape &sh, const Kv4 &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                             const int32_t *n_ctx, const int32_t *n_new, uint32_t *status, cudaStream_t stream) {
  return sh.d == 128 ? launch_pdl(kv4_store<128>, dim3(rows_grid<128>(sh)), kKv4Threads, 0, stream, sh, c, k, v, n_ctx, n_new, status)
                     : launch_pdl(kv4_store<64>, dim3(rows_grid<64>(sh)), kKv4Threads, 0, stream, sh, c, k, v, n_ctx, n_new, status);
}

cudaError_t launch_kv4_load(const Shape &sh, const Kv4 &c, __nv_bfloat16 *k, __nv_bfloat16 *v, const int32_t *start,
                            const int32_t *n_new, uint32_t *status, cudaStream_t stream) {
  return sh.d == 128 ? launch_pdl(kv4_load<128>, dim3(rows_grid<128>(sh)), kKv4Threads, 0, stream, sh, c, k, v, start, n_new, status)
                     : launch_pdl(kv4_load<64>, dim3(rows_grid<64>(sh)), kKv4Threads, 0, stream, sh, c, k, v, start, n_new, status);
}

}  // namespace dsa
