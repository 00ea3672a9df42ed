// The 2-norm over many gradients, and the gradients times a clipping factor.
//
//   norm = sqrt(sum over all tensors and values of g^2);  out = g * min(1, max_norm / norm).
//
// A launch takes the tensors' addresses and lengths in its arguments (no table in device memory,
// so nothing is copied and a captured launch holds its own), cut into chunks of 32 KB that the
// blocks take in turn.  Squares are summed in 64 bits: a value's square cannot overflow or vanish
// (an fp32 sum loses 1e20 and 1e-25), at no cost while HBM is the bound.  Each block leaves one
// sum, and a last launch adds them in one order, so a norm repeats bit for bit.
//   1.4 G bf16 values (2.8 GB): norm 490 us, 5.7 TB/s; clipping 1060 us, 5.3 TB/s.  320 small tensors: 56 us
// in six launches, beside about 160 us in which the host checks them and fills the arguments.  (Clipping
// from the last chunk to the first, which the norm has just read, is no faster: 1555 us either way for both.)
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

// 16 bytes at any element's address
template <class T>
struct Piece;
template <>
struct Piece<float> {
  typedef u32x4 type __attribute__((aligned(4)));
};
template <>
struct Piece<bf16> {
  typedef u32x4 type __attribute__((aligned(2)));
};

template <class T>
__device__ inline void unpack(const u32x4& v, float* f) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
}

constexpr int kChunkBytes = 32 * 1024, kClipThreads = 256;
constexpr int kChunkPieces = kChunkBytes / 16 / kClipThreads;  // a thread's pieces of a chunk

// Tensors of one launch; first[i]: chunks before tensor i.  n holds the length, and in its
// lowest bit the type (1: bf16).
template <int M>
struct NormBatch {
  static constexpr int kMost = M;
  const void* p[M];
  int64_t n2[M];
  int32_t first[M + 1];
  int32_t count;
};
using NormTensors = NormBatch<kNormTensors>;
struct ClipTensors {
  static constexpr int kMost = kClipTensors;
  const void* p[kClipTensors];
  void* o[kClipTensors];
  int64_t n2[kClipTensors];
  int32_t first[kClipTensors + 1];
  int32_t count;
};
static_assert(sizeof(NormTensors) <= 4000 && sizeof(ClipTensors) <= 4000, "kernel arguments");

// the tensor that holds a chunk
template <class B>
__device__ inline int tensor_of(const B& b, int chunk) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <class T>
__device__ inline double chunk_squares(const T* p, int n) {
  constexpr int V = 16 / sizeof(T);
  const int pieces = n / V, tid = threadIdx.x;
  double sum[2] = {0.0, 0.0};
  u32x4 v[kChunkPieces];
#pragma unroll
  for (int i = 0; i < kChunkPieces; ++i) {
    const int q = i * kClipThreads + tid;
    v[i] = u32x4{0, 0, 0, 0};
    if (q < pieces) v[i] = *reinterpret_cast<const typename Piece<T>::type*>(p + q * V);
  }
#pragma unroll
  for (int i = 0; i < kChunkPieces; ++i) {
    float f[V];
    unpack<T>(v[i], f);
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j & 1] = fma((double)f[j], (double)f[j], sum[j & 1]);
  }
  if (tid < n - pieces * V) {
    const double f = (double)Elt<T>::to_f32(p[pieces * V + tid]);
    sum[0] = fma(f, f, sum[0]);
  }
  return sum[0] + sum[1];
}

__device__ inline double shfl_xor_f64(double v, int m) {
  return __longlong_as_double((long long)shfl_xor_u64((uint64_t)__double_as_longlong(v), m));
}

// The block's sum, on thread 0.
template <int THREADS>
__device__ inline double block_sum(double v) {
  __shared__ double part[THREADS / kWave];
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += shfl_xor_f64(v, m);
  if (lane_id() == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < THREADS / kWave; ++w) sum += part[w];
  return sum;
}

__global__ void __launch_bounds__(kClipThreads)
norm_kernel(const NormTensors b, int chunks, double* __restrict__ partial) {
  double sum = 0.0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(b, c);
    const int64_t n = b.n2[t] >> 1;
    const char* p = static_cast<const char*>(b.p[t]);
    const int64_t at = (int64_t)(c - b.first[t]) * kChunkBytes;
    if (b.n2[t] & 1)
      sum += chunk_squares(reinterpret_cast<const bf16*>(p + at),
                           (int)min(n - at / 2, (int64_t)(kChunkBytes / 2)));
    else
      sum += chunk_squares(reinterpret_cast<const float*>(p + at),
                           (int)min(n - at / 4, (int64_t)(kChunkBytes / 4)));
  }
  sum = block_sum<kClipThreads>(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(1024)
norm_sum_kernel(const double* __restrict__ partial, int n, float* __restrict__ norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) sum += partial[i];
  sum = block_sum<1024>(sum);
  if (threadIdx.x == 0) *norm = (float)sqrt(sum);
}

template <class T>
__device__ inline void chunk_scaled(const T* p, T* o, int n, float factor) {
  constexpr int V = 16 / sizeof(T);
  const int pieces = n / V, tid = threadIdx.x;
  u32x4 v[kChunkPieces];
#pragma unroll
  for (int i = 0; i < kChunkPieces; ++i) {
    const int q = i * kClipThreads + tid;
    if (q < pieces) v[i] = *reinterpret_cast<const typename Piece<T>::type*>(p + q * V);
  }
#pragma unroll
  for (int i = 0; i < kChunkPieces; ++i) {
    const int q = i * kClipThreads + tid;
    if (q >= pieces) break;
    float f[V];
    unpack<T>(v[i], f);
    typedef T tx __attribute__((ext_vector_type(16 / sizeof(T))));
    tx r;
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = Elt<T>::from_f32(f[j] * factor);
    *reinterpret_cast<typename Piece<T>::type*>(o + q * V) = __builtin_bit_cast(u32x4, r);
  }
  const int q = pieces * V + tid;
  if (q < n) o[q] = Elt<T>::from_f32(Elt<T>::to_f32(p[q]) * factor);
}

// A factor of one leaves a tensor that is clipped in place unread.  A norm that is no number or
// infinite clips nothing.
__global__ void __launch_bounds__(kClipThreads)
clip_kernel(const ClipTensors b, int chunks, float max_norm, const float* __restrict__ norm) {
  const float size = *norm;
  const float factor =
      size > max_norm && size < __builtin_huge_valf() ? max_norm / size : 1.0f;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(b, c);
    if (factor == 1.0f && b.p[t] == b.o[t]) continue;
    const int64_t n = b.n2[t] >> 1;
    const char* p = static_cast<const char*>(b.p[t]);
    char* o = static_cast<char*>(b.o[t]);
    const int64_t at = (int64_t)(c - b.first[t]) * kChunkBytes;
    if (b.n2[t] & 1)
      chunk_scaled(reinterpret_cast<const bf16*>(p + at), reinterpret_cast<bf16*>(o + at),
                   (int)min(n - at / 2, (int64_t)(kChunkBytes / 2)), factor);
    else
      chunk_scaled(reinterpret_cast<const float*>(p + at), reinterpret_cast<float*>(o + at),
                   (int)min(n - at / 4, (int64_t)(kChunkBytes / 4)), factor);
  }
}

namespace {

// Adds tensor g to a launch's tensors; false: there is no room.  Empty tensors take none.
template <class B>
bool add_tensor(B* b, const GradTensor& g) {
  if (g.n == 0) return true;
  if (b->count == B::kMost) return false;
  const int i = b->count++;
  const int64_t per = kChunkBytes / (g.dtype == 1 ? 2 : 4);
  b->p[i] = g.grad;
  b->n2[i] = 2 * g.n + (g.dtype == 1 ? 1 : 0);
  b->first[i + 1] = b->first[i] + (int32_t)((g.n + per - 1) / per);
  return true;
}

}  // namespace

hipError_t launch_grad_norm(int64_t count, const GradTensor* g, double* partial, float* norm,
                            hipStream_t s) {
  int64_t sums = 0;
  for (int64_t i = 0; i < count;) {
    NormTensors b;
    b.count = 0;
    b.first[0] = 0;
    while (i < count && add_tensor(&b, g[i])) ++i;
    const int chunks = b.first[b.count];
    if (chunks == 0) continue;
    const int blocks = std::min(chunks, kNormBlocks);
    norm_kernel<<<blocks, kClipThreads, 0, s>>>(b, chunks, partial + sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sums += blocks;
  }
  norm_sum_kernel<<<1, 1024, 0, s>>>(partial, (int)sums, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(int64_t count, const GradTensor* g, float max_norm,
                            const float* norm, hipStream_t s) {
  for (int64_t i = 0; i < count;) {
    ClipTensors b;
    b.count = 0;
    b.first[0] = 0;
    while (i < count) {
      const int at = b.count;
      if (!add_tensor(&b, g[i])) break;
      if (b.count > at) b.o[at] = g[i].out;
      ++i;
    }
    const int chunks = b.first[b.count];
    if (chunks == 0) continue;
    clip_kernel<<<std::min(chunks, kClipBlocks), kClipThreads, 0, s>>>(b, chunks, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
