// Block-scaled e4m3 quantisation.
//
//   block b of block_rows x 128 elements (ragged at the right and bottom edge):
//     a = max(max_b |x|, 2^-100),  scale_b = a / 448,  code = e4m3(x * (448 / a))
//
// e4m3 holds magnitudes up to 448 with 4 significant bits, so the largest
// element of a block lands on 448 and every element is off by at most half a
// step, 2^-4 of its value (2^-10 in units of the scale below 2^-6). The
// maximum, the scale and the product are float; the one rounding to 8 bits is
// the conversion (nearest even). The floor 2^-100 keeps the quotient of an
// all-zero block finite: its codes are 0. A NaN in a block makes its scale
// and codes NaN; an infinity makes the scale infinite.
//
// The work is one pass: a lane holds 16 bytes of a row, 16 lanes hold the 128
// columns of a block, and the maximum is a shuffle over them (1-row blocks) or
// a shuffle and one exchange in shared memory (128-row blocks, whose elements
// stay in registers in between). HBM bandwidth bounds it: 3 bytes per bf16
// element.
#include "common.cuh"
#include "internal.h"

#include "fp8.cuh"

namespace uno {

namespace {

constexpr int kRowThreads = 256;
constexpr int kBlkThreads = 256;

// 8 consecutive elements as raw words, and as floats.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ float amax8(const Vec8<__nv_bfloat16>& v) {
  const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(abs_bf16x2(v.w.x), abs_bf16x2(v.w.y)),
                                    max_nan_bf16x2(abs_bf16x2(v.w.z), abs_bf16x2(v.w.w)));
  return max_nan(bf16_lo(m), bf16_hi(m));
}
__device__ __forceinline__ float amax8(const Vec8<float>& v) {
  float f[8];
  v.get(f);
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
  return m;
}

template <typename T>
__device__ __forceinline__ uint2 codes8(const Vec8<T>& v, float inv) {
  float f[8];
  v.get(f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= inv;
  return e4m3x8(f);
}

// 1 x 128 blocks: half a warp per block, kIter blocks in flight per half warp.
// scale of (row m, block b) at scales[m * ld_m + b * ld_b].
template <typename T, int kIter>
__global__ void __launch_bounds__(kRowThreads)
    quantize_rows_kernel(const T* __restrict__ x, uint32_t total, int K, uint32_t nkb, uint8_t* __restrict__ q,
                         float* __restrict__ scales, long long ld_m, long long ld_b) {
  const uint32_t half = threadIdx.x >> 4, l = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (kIter * (kRowThreads / 16)) + half;
  pdl_wait();
  Vec8<T> v[kIter];
  size_t off[kIter];
  bool in[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t b = first + i * (kRowThreads / 16), m = b / nkb;
    const int c = static_cast<int>((b - m * nkb) * 128 + l * 8);
    in[i] = b < total && c < K;
    off[i] = static_cast<size_t>(m) * K + c;
    if (in[i]) v[i].load(x + off[i]);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    float a = amax8(v[i]);
#pragma unroll
    for (int o = 8; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    a = max_nan(a, kAmaxFloor);
    if (in[i]) *reinterpret_cast<uint2*>(q + off[i]) = codes8(v[i], __fdiv_rn(kE4m3Max, a));
    const uint32_t b = first + i * (kRowThreads / 16);
    if (l == 0 && b < total) {
      const uint32_t m = b / nkb;
      scales[m * ld_m + (b - m * nkb) * ld_b] = __fdiv_rn(a, kE4m3Max);
    }
  }
}

// 128 x 128 blocks: one CTA each, the block in registers between the maximum
// and the conversion (8 vectors a thread).
template <typename T>
__global__ void __launch_bounds__(kBlkThreads)
    quantize_blocks_kernel(const T* __restrict__ x, long long M, int K, int nkb, uint8_t* __restrict__ q,
                           float* __restrict__ scales) {
  constexpr int kRows = kBlkThreads / 16, kIter = 128 / kRows;
  __shared__ float part[kBlkThreads / 32];
  const int kb = blockIdx.x % nkb;
  const long long m0 = static_cast<long long>(blockIdx.x / nkb) * 128;
  const int rr = threadIdx.x >> 4, c = kb * 128 + (threadIdx.x & 15) * 8;
  pdl_wait();
  Vec8<T> v[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long m = m0 + rr + i * kRows;
    if (m < M && c < K) v[i].load(x + m * K + c);
    else v[i].zero();
  }
  float a = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < kIter; ++i) a = max_nan(a, amax8(v[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBlkThreads / 32; ++w) a = max_nan(a, part[w]);
  const float inv = __fdiv_rn(kE4m3Max, a);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long m = m0 + rr + i * kRows;
    if (m < M && c < K) *reinterpret_cast<uint2*>(q + m * K + c) = codes8(v[i], inv);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = __fdiv_rn(a, kE4m3Max);
}

template <typename T>
uno_status rows_launch(const T* x, int64_t M, int64_t K, uint8_t* q, float* scales, int64_t ld_m,
                       int64_t ld_b, cudaStream_t s) {
  const int nkb = static_cast<int>((K + 127) / 128);
  constexpr int per = kRowThreads / 16;
  const int64_t blocks = M * nkb;
  // one block per half warp until the grid fills the device, then four in flight
  const bool wide = blocks >= static_cast<int64_t>(device_sm_count()) * per * 16;
  const int64_t grid = (blocks + per * (wide ? 4 : 1) - 1) / (per * (wide ? 4 : 1));
  if (blocks > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many blocks to quantise");
  const dim3 g(static_cast<unsigned>(grid)), b(kRowThreads);
  const uint32_t total = static_cast<uint32_t>(blocks), per_row = static_cast<uint32_t>(nkb);
  const long long lm = ld_m, lb = ld_b;
  const int k = static_cast<int>(K);
  const cudaError_t e =
      wide ? launch_kernel(quantize_rows_kernel<T, 4>, g, b, 0, s, 1, x, total, k, per_row, q, scales, lm, lb)
           : launch_kernel(quantize_rows_kernel<T, 1>, g, b, 0, s, 1, x, total, k, per_row, q, scales, lm, lb);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "row quantisation launch");
}

template <typename T>
uno_status blocks_launch(const T* x, int64_t M, int64_t K, uint8_t* q, float* scales, cudaStream_t s) {
  const int nkb = static_cast<int>((K + 127) / 128);
  const int64_t grid = (M + 127) / 128 * nkb;
  if (grid > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many blocks to quantise");
  const cudaError_t e =
      launch_kernel(quantize_blocks_kernel<T>, dim3(static_cast<unsigned>(grid)), dim3(kBlkThreads), 0,
                    s, 1, x, static_cast<long long>(M), static_cast<int>(K), nkb, q, scales);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "block quantisation launch");
}

}  // namespace

// The kernels here never trigger their dependents early: what they write may
// be a weight, which the GEMM kernels prefetch before they wait.
uno_status fp8_quantize_launch(uno_dtype dt, int64_t M, int64_t K, int block_rows, const void* x,
                               uint8_t* q, float* scales, int64_t ld_m, int64_t ld_b,
                               cudaStream_t s) {
  if (dt == UNO_F32) {
    const float* xf = static_cast<const float*>(x);
    return block_rows == 1 ? rows_launch(xf, M, K, q, scales, ld_m, ld_b, s)
                           : blocks_launch(xf, M, K, q, scales, s);
  }
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
  return block_rows == 1 ? rows_launch(xb, M, K, q, scales, ld_m, ld_b, s)
                         : blocks_launch(xb, M, K, q, scales, s);
}

}  // namespace uno
