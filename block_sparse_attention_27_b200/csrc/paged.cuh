// paged.cuh -- what the operators beside the two passes share: the block's token
// counts, the lookup of a logical token in the paged cache, the 4-bit code.
//
// These kernels are launched as programmatic dependents: their blocks are resident while the
// kernel ahead still writes what they read after the dependency wait.  None of it is read-only
// for their life, which the read-only path (__ldg, const __restrict__ parameters) asks for, so
// every load here is a plain one.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace dsa {

// Tokens of sequence s's block that exist (n_new, else B).
__device__ __forceinline__ int block_tokens(const int32_t *n_new, int s, int B, uint32_t *status, bool report) {
  if (!n_new) return B;
  const int m = n_new[s];
  if (m < 0 || m > B) {
    if (report) raise_status(status, kStatusBadIndex);
    return m < 0 ? 0 : B;
  }
  return m;
}

// Physical page of logical page lp of sequence s, or -1 (not in the table, or an
// entry outside the cache).
__device__ __forceinline__ long long physical_page(const Shape &sh, int s, long long lp) {
  if (lp < 0 || lp >= sh.max_pages) return -1;
  const long long p = sh.page_table ? (long long)sh.page_table[(size_t)s * sh.max_pages + lp]
                                    : (long long)s * sh.max_pages + lp;
  return p >= 0 && p < sh.n_phys ? p : -1;
}

// 4-bit cache: a group is 32 values that share a scale of five significant bits,
// a word eight values (2i in bits 4i.., 2i + 1 in bits 16 + 4i..).
constexpr int kKv4Group = 32;

// Values 2i and 2i + 1 of a word as a bf16 pair.  (w shifted so that the codes sit in
// mantissa bits 3..6) | 0x4300 is 128 + 8 code; one fma with s/8 and -24 s gives
// (code - 8) s.  Both constants are exact (s has five significant bits, 24 s seven),
// and so is the result (|code - 8| <= 8: at most eight bits in all).
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, int i, __nv_bfloat162 s8, __nv_bfloat162 m24) {
  const uint32_t x = i == 0 ? w << 3 : w >> (4 * i - 3);
  const uint32_t y = (x & 0x00780078u) | 0x43004300u;
  __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&y), s8, m24);
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ void kv4_constants(__nv_bfloat162 s, __nv_bfloat162 &s8, __nv_bfloat162 &m24) {
  s8 = __hmul2(s, __float2bfloat162_rn(0.125f));
  m24 = __hmul2(s, __float2bfloat162_rn(-24.f));
}
__device__ __forceinline__ void kv4_constants(__nv_bfloat16 s, __nv_bfloat162 &s8, __nv_bfloat162 &m24) {
  const float f = __bfloat162float(s);
  s8 = __float2bfloat162_rn(f * 0.125f);
  m24 = __float2bfloat162_rn(f * -24.f);
}

// Launch as a programmatic dependent of the kernel ahead on the stream.
template <class K, class... A>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

}  // namespace dsa
