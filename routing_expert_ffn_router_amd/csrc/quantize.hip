// A matrix to e4m3 with one power-of-two scale per block of 1 x 128 or 128 x 128 values.
//
//   s = 2^e, e the least integer >= -126 with max |x| <= 448 * 2^e over the block;  q = x / s.
// Dividing by a power of two is exact (e4m3's own rounding is the only one), so the result does
// not depend on how the division is carried out.  Bound by HBM: each value is read once and a
// byte written; a thread holds its values in registers between the maximum and the conversion
// (8191 x 4096 fp32 rows 31 us, 5.4 TB/s; eight weights of 14336 x 4096 bf16 246 us, 5.7 TB/s;
// 256 x 7168 bf16 rows 3.0 us, latency).
#include <algorithm>

#include "fp8_common.h"
#include "kernels.h"

namespace moe {

// Eight consecutive values from memory, as floats.
template <class T>
struct Load8;
template <>
struct Load8<bf16> {
  u32x4 v;
  __device__ inline void load(const bf16* p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  }
  __device__ inline void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
};
template <>
struct Load8<float> {
  u32x4 v[2];
  __device__ inline void load(const float* p) {
    v[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    v[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p) + 1);
  }
  __device__ inline void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i / 4][i % 4]);
  }
};

__device__ inline uint32_t max8(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  return m;
}

__device__ inline void store8(uint8_t* q, const float* f, int e, bool finite) {
  const float r = inv_scale(e);
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = finite ? pack_e4m3(f[4 * i] * r, f[4 * i + 1] * r, f[4 * i + 2] * r, f[4 * i + 3] * r)
                  : kNan4;
  *reinterpret_cast<u32x2*>(q) = w;
}

// Rows: the matrix is a list of rows * K / 128 groups of 128 values in memory order, and the
// scales a list in the same order.  Sixteen lanes hold a group (16 bytes of bf16, or 32 of fp32,
// each); U groups per lane are in flight.
template <class T, int U>
__global__ void __launch_bounds__(256)
quantize_rows_kernel(const T* __restrict__ x, int64_t groups, int scale_type,
                     uint8_t* __restrict__ q, void* __restrict__ scale) {
  const int sub = threadIdx.x & 15;
  const int64_t g0 = ((int64_t)blockIdx.x * U) * 16 + threadIdx.x / 16;
  Load8<T> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = min(g0 + u * 16, groups - 1);
    v[u].load(x + g * kScaleBlock + sub * 8);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * 16;
    if (g >= groups) return;
    float f[8];
    v[u].get(f);
    uint32_t m = max8(f);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 16));
    const bool finite = m < kInfBits;
    const int e = finite ? scale_exponent(m) : 0;
    store8(q + g * kScaleBlock + sub * 8, f, e, finite);
    if (sub == 0) store_scale(scale, g, scale_type, e, finite);
  }
}

// 128 x 128 blocks: one workgroup each; a thread holds eight pieces of eight values, sixteen
// rows apart, so that a wave reads whole cache lines of four rows at once.
template <class T>
__global__ void __launch_bounds__(256)
quantize_blocks_kernel(const T* __restrict__ x, int64_t K, int64_t kblocks, int scale_type,
                       uint8_t* __restrict__ q, void* __restrict__ scale) {
  __shared__ uint32_t wave_max[4];
  const int64_t b = blockIdx.x, rb = b / kblocks, cb = b - rb * kblocks;
  const int64_t at = (rb * 128 + threadIdx.x / 16) * K + cb * 128 + (threadIdx.x & 15) * 8;
  Load8<T> v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u].load(x + at + u * 16 * K);
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[8];
    v[u].get(f);
    m = max(m, max8(f));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if (lane_id() == 0) wave_max[threadIdx.x / 64] = m;
  __syncthreads();
  m = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
  const bool finite = m < kInfBits;
  const int e = finite ? scale_exponent(m) : 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[8];
    v[u].get(f);
    store8(q + at + u * 16 * K, f, e, finite);
  }
  if (threadIdx.x == 0) store_scale(scale, b, scale_type, e, finite);
}

template <class T>
static hipError_t run_quantize(int64_t rows, int64_t K, int64_t block_rows, int scale_type,
                               const T* x, uint8_t* q, void* scale, hipStream_t s) {
  const int64_t kblocks = K / kScaleBlock;
  if (block_rows == 128) {
    quantize_blocks_kernel<T><<<(unsigned)(rows / 128 * kblocks), 256, 0, s>>>(
        x, K, kblocks, scale_type, q, scale);
    return hipGetLastError();
  }
  const int64_t groups = rows * kblocks;
  // sixteen groups per block and step: one step where the blocks are few (256 x 7168 bf16 3.0
  // against 3.9 us, 1024 x 4096 3.9 against 4.4; 2048 x 4096 the same), else four in flight (8192 x
  // 4096 17.9 against 20.2 us)
  if (groups <= 32768)
    quantize_rows_kernel<T, 1><<<(unsigned)((groups + 15) / 16), 256, 0, s>>>(
        x, groups, scale_type, q, scale);
  else
    quantize_rows_kernel<T, 4><<<(unsigned)((groups + 63) / 64), 256, 0, s>>>(
        x, groups, scale_type, q, scale);
  return hipGetLastError();
}

hipError_t launch_quantize(int64_t rows, int64_t K, int64_t block_rows, int dtype,
                           int scale_type, const void* x, void* q, void* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == 1)
    return run_quantize(rows, K, block_rows, scale_type, (const bf16*)x, (uint8_t*)q, scale, s);
  return run_quantize(rows, K, block_rows, scale_type, (const float*)x, (uint8_t*)q, scale, s);
}

}  // namespace moe
