// kv4.cu -- dsa_kv4_store and dsa_kv4_load: rows into and out of the 4-bit cache.
// Four lanes hold a group of 32 values, eight each: one packed word per lane and group.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kKv4Threads = 256;

// Scale of a group whose largest magnitude has the bits amax (bf16): the smallest number of
// five significant bits that is at least amax / 7, 0 below 2^-100, NaN from 2^120 on (and for
// NaN).  The product with a seventh less 2^-20 of it stands for the division: with amax = A 2^e,
// A of eight bits, a quotient that is no five-bit number lies at least 1/255 above the border
// below it, and one that is falls under its border by less than rounding up puts back.
__device__ __forceinline__ float kv4_scale(uint32_t amax) {
  if (amax >= 0x7b80u) return __int_as_float(0x7fc00000);
  if (amax < 0x0d80u) return 0.f;
  constexpr float kSeventh = (1.f - 1.f / 1048576.f) / 7.f;
  return __uint_as_float((__float_as_uint(__uint_as_float(amax << 16) * kSeventh) + 0x7ffffu) & ~0x7ffffu);
}

// Word of codes and scale of a lane's eight values; the four lanes of a group come together.
__device__ __forceinline__ uint32_t kv4_codes(const uint4 &x, float &s) {
  // magnitudes order as their bits do, infinities and NaN above all numbers
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t big = __vmaxu2(__vmaxu2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu), __vmaxu2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu));
  big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 2));
  s = kv4_scale(max(big >> 16, big & 0xffffu));
  // Nearest integer to x / s, ties to even, without a division each.  x / s is half way between
  // integers or at least 2^-9 off (x has eight significant bits, s five, |x| <= 7 s), so
  // rounding the product with 1/s (two units off at most) to a multiple of 2^-11 first meets
  // the half-way quotients exactly and moves no other across.  The next sum rounds that to an
  // integer; four codes are then the digits of one fp32 integer, eight a word.
  const float inv = __fdividef(1.f, s);
  constexpr float kTo11 = 6144.f, kTo0 = 12582912.f;  // 1.5 2^12, 1.5 2^23: a unit is 2^-11, 1
  float2 digits = make_float2(kTo0 + 34952.f, kTo0 + 34952.f);  // 8 (1 + 16 + 256 + 4096)
  float place = 1.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 z = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
    const float2 y = sm100::fma2(z, make_float2(inv, inv), make_float2(kTo11, kTo11));
    const float2 m = sm100::add2(sm100::add2(y, make_float2(kTo0 - kTo11, kTo0 - kTo11)), make_float2(-kTo0, -kTo0));
    digits = sm100::fma2(m, make_float2(place, place), digits);
    place *= 16.f;
  }
  const uint32_t w = __byte_perm(__float_as_uint(digits.x), __float_as_uint(digits.y), 0x5410);
  return s > 0.f ? w : 0x88888888u;
}

// Walks a CTA's rows (token, K | V, head), kPass apart: TT tokens from t0, found once per
// token and kept in shared memory (looked up by every lane, they were most of the
// instructions that bound these kernels: 284 and 165 a lane and row).  A lane holds C chunks of
// eight values, kLanes chunks apart: four lanes a group, whole sectors a load, and what a row
// costs besides is shared by twice the values.  32K tokens of 8 heads, store and load: 87 us, 73 without
// a division and with packed arithmetic, 61 with two chunks a lane, 59.5 with two rows' loads ahead of
// their stores in the load (the floor is 44).
template <int D, int C>
struct Rows {
  static constexpr int kLanes = D / (8 * C), kPass = kKv4Threads / kLanes;
  int i, r, n, di, dr;  // token of the CTA, row of it, rows of a token; the step of one pass
  __device__ __forceinline__ Rows(int n_) : n(n_) {
    const int row = threadIdx.x / kLanes;
    i = row / n;
    r = row - i * n;
    di = kPass / n;
    dr = kPass - di * n;
  }
  __device__ __forceinline__ void step() {
    i += di;
    r += dr;
    if (r >= n) {
      r -= n;
      ++i;
    }
  }
};
// Row of head 0 in the cache of each of the CTA's tokens (head h is h * P further), -1: none.
template <int TT>
__device__ __forceinline__ void find_tokens(const Shape &sh, long long t0, const int32_t *first,
                                            const int32_t *n_new, uint32_t *status, long long (&rows)[TT]) {
  if (threadIdx.x < TT) {
    const long long t = t0 + threadIdx.x;
    long long row = -1;
    if (t < (long long)sh.S * sh.B) {
      const int s = (int)((unsigned)t / (unsigned)sh.B), b = (int)(t - (long long)s * sh.B);
      if (b < block_tokens(n_new, s, sh.B, status, b == 0)) {
        const int n = first[s];
        const long long at = (long long)n + b;
        const long long phys = n < 0 ? -1 : physical_page(sh, s, at / sh.P);
        if (phys < 0)
          raise_status(status, kStatusBadIndex);
        else
          row = phys * sh.Hkv * sh.P + at % sh.P;
      }
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
}

template <int D, int TT, int C>
__global__ void __launch_bounds__(kKv4Threads, 8)
    kv4_store(const Shape sh, const Kv4 c4, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
              const int32_t *n_ctx, const int32_t *n_new, uint32_t *status) {
  __shared__ long long rows[TT];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const long long t0 = (long long)blockIdx.x * TT;
  find_tokens<TT>(sh, t0, n_ctx, n_new, status, rows);
  Rows<D, C> at(2 * sh.Hkv);
  constexpr int kLanes = Rows<D, C>::kLanes;
  const int l = threadIdx.x % kLanes;
  uint4 next[C];
  auto load = [&]() {
#pragma unroll
    for (int c = 0; c < C; ++c) next[c] = make_uint4(0, 0, 0, 0);
    if (at.i >= TT || rows[at.i] < 0) return;
    const bool isv = at.r >= sh.Hkv;
    const uint4 *src = reinterpret_cast<const uint4 *>((isv ? v : k) + ((t0 + at.i) * sh.Hkv + (isv ? at.r - sh.Hkv : at.r)) * D) + l;
#pragma unroll
    for (int c = 0; c < C; ++c) next[c] = src[c * kLanes];
  };
  load();
  // whole warps go round: a group's maximum is a shuffle
#pragma unroll 1
  for (int done = 0; done < TT * 2 * sh.Hkv; done += Rows<D, C>::kPass) {
    uint4 raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = next[c];
    const int i = at.i, r = at.r;
    at.step();
    load();
    uint32_t w[C];
    float sc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = kv4_codes(raw[c], sc[c]);
    if (i >= TT || rows[i] < 0) continue;
    const bool isv = r >= sh.Hkv;
    const long long row = rows[i] + (isv ? r - sh.Hkv : r) * sh.P;
    uint8_t *codes = (isv ? c4.v : c4.k) + row * (D / 2) + 4 * l;
    __nv_bfloat16 *scales = (isv ? c4.vs : c4.ks) + row * (D / kKv4Group) + l / 4;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      *reinterpret_cast<uint32_t *>(codes + c * 4 * kLanes) = w[c];
      if (l % 4 == 0) scales[c * (kLanes / 4)] = __float2bfloat16_rn(sc[c]);
    }
  }
}

template <int D, int TT, int C>
__global__ void __launch_bounds__(kKv4Threads, 8)
    kv4_load(const Shape sh, const Kv4 c4, __nv_bfloat16 *k, __nv_bfloat16 *v, const int32_t *start,
             const int32_t *n_new, uint32_t *status) {
  __shared__ long long rows[TT];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch_dependents();
  const long long t0 = (long long)blockIdx.x * TT;
  find_tokens<TT>(sh, t0, start, n_new, status, rows);
  Rows<D, C> at(2 * sh.Hkv);
  constexpr int kLanes = Rows<D, C>::kLanes, kAhead = 2;
  const int l = threadIdx.x % kLanes;
  // Rows kAhead at a time: their loads go out before the first store, behind which the next rows'
  // loads stay.  64K tokens of 4 heads: 25.5 us; three rows 29.2, four 29.7 (no more registers with
  // six CTAs an SM: 29.2 and 29.6).
#pragma unroll 1
  while (at.i < TT) {
    uint32_t w[kAhead][C];
    __nv_bfloat16 sc[kAhead][C];
    __nv_bfloat16 *out[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      out[u] = nullptr;
      if (at.i < TT && rows[at.i] >= 0) {
        const bool isv = at.r >= sh.Hkv;
        const int h = isv ? at.r - sh.Hkv : at.r;
        const long long row = rows[at.i] + h * sh.P;
        const uint8_t *codes = (isv ? c4.v : c4.k) + row * (D / 2) + 4 * l;
        const __nv_bfloat16 *scales = (isv ? c4.vs : c4.ks) + row * (D / kKv4Group) + l / 4;
        out[u] = (isv ? v : k) + ((t0 + at.i) * sh.Hkv + h) * D + 8 * l;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          w[u][c] = *reinterpret_cast<const uint32_t *>(codes + c * 4 * kLanes);
          sc[u][c] = scales[c * (kLanes / 4)];
        }
      }
      at.step();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!out[u]) continue;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        __nv_bfloat162 s8, m24;
        kv4_constants(sc[u][c], s8, m24);
        *reinterpret_cast<uint4 *>(out[u] + c * 8 * kLanes) =
            make_uint4(kv4_pair(w[u][c], 0, s8, m24), kv4_pair(w[u][c], 1, s8, m24), kv4_pair(w[u][c], 2, s8, m24),
                       kv4_pair(w[u][c], 3, s8, m24));
      }
    }
  }
}

unsigned tokens_grid(const Shape &sh, int per) { return (unsigned)(((long long)sh.S * sh.B + per - 1) / per); }

// A token a CTA and eight values a lane while that is quicker, then four tokens, and eight once
// they fill the SMs (8 KV heads, store and load): 512 tokens 5.8, 6.0, 7.8 us; 1024 tokens 7.4, 6.6,
// 7.8; 2048 tokens 11.4, 8.4, 9.1; 8192 tokens 35.6, 19.9, 20.2; 32766 tokens 142, 70.3, 65.9.
int tokens_per_cta(const Shape &sh) {
  const long long tokens = (long long)sh.S * sh.B;
  return tokens >= 8 * 8 * 148 ? 8 : tokens >= 1024 ? 4 : 1;
}

}  // namespace

#define DSA_KV4_LAUNCH_D(kern, d, ...)                                                                        \
  switch (tokens_per_cta(sh)) {                                                                               \
    case 8: return launch_pdl(kern<d, 8, 2>, dim3(tokens_grid(sh, 8)), kKv4Threads, 0, stream, __VA_ARGS__);  \
    case 4: return launch_pdl(kern<d, 4, 2>, dim3(tokens_grid(sh, 4)), kKv4Threads, 0, stream, __VA_ARGS__);  \
    default: return launch_pdl(kern<d, 1, 1>, dim3(tokens_grid(sh, 1)), kKv4Threads, 0, stream, __VA_ARGS__); \
  }
#define DSA_KV4_LAUNCH(kern, ...)                          \
  if (sh.d == 128) DSA_KV4_LAUNCH_D(kern, 128, __VA_ARGS__) \
  DSA_KV4_LAUNCH_D(kern, 64, __VA_ARGS__)

cudaError_t launch_kv4_store(const Shape &sh, const Kv4 &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                             const int32_t *n_ctx, const int32_t *n_new, uint32_t *status, cudaStream_t stream) {
  DSA_KV4_LAUNCH(kv4_store, sh, c, k, v, n_ctx, n_new, status);
}

cudaError_t launch_kv4_load(const Shape &sh, const Kv4 &c, __nv_bfloat16 *k, __nv_bfloat16 *v, const int32_t *start,
                            const int32_t *n_new, uint32_t *status, cudaStream_t stream) {
  DSA_KV4_LAUNCH(kv4_load, sh, c, k, v, start, n_new, status);
}

}  // namespace dsa
