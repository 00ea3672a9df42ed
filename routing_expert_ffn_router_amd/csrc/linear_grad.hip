// The backward pass of an expert's linear layer up to its product:
//   dz[r, n] = dy[r, n] act'(z[r, n]),   db[e, n] = sum of dz[r, n] over the rows r of expert e.
//
// One pass over dy and z.  A block takes kGradRows rows of one expert and 512 (fp32: 256) columns,
// 16 bytes of a row for each lane of a wave, rows in turn over its waves; each lane keeps its
// columns' sums, the waves' are added through LDS, and a row of sums for each row tile goes to the
// workspace, added up by another launch in row order.  The sums are of the unrounded dz, in fp32,
// and repeat bit for bit.  Bound by HBM: 8191 rows of 14336 bf16 values, gelu, dz and db: 121 us for 705 MB,
// 5.8 TB/s, and 6 us for the sums of the row tiles.
#include <type_traits>

#include "act.h"
#include "kernels.h"

namespace moe {

// Row tiles need no table and no scan: expert e's tiles of B rows are numbered from
//   f(e) = offsets[e] / B + e
// on, which leaves room for them, since ceil(L / B) <= floor((r + L) / B) + 1 for 0 <= r.  The
// expert of slot s is the last one with f(e) <= s.
__device__ inline int slot_expert(const int32_t* __restrict__ offsets, int E, int R, int s) {
  if (!offsets) return 0;
  int below = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int e = e0 + lane_id();
    const bool in = e < E && min(max(offsets[e], 0), R) / kGradRows + e <= s;
    below += __builtin_popcountll(__ballot(in));
  }
  return max(below, 1) - 1;
}
struct Rows {
  int begin, end;
};
__device__ inline Rows expert_rows(const int32_t* __restrict__ offsets, int R, int e) {
  if (!offsets) return Rows{0, R};
  return Rows{min(max(offsets[e], 0), R), min(max(offsets[e + 1], 0), R)};
}

constexpr int kGradWaves = 4;

template <class T, int ACT>
__global__ void __launch_bounds__(kGradWaves* kWave)
linear_grad_kernel(const T* dy, const T* __restrict__ z, const int32_t* __restrict__ offsets,
                   T* dz, float* __restrict__ partial, int R, int E, int N, int strips) {
  constexpr int V = 16 / sizeof(T), BN = V * kWave;
  __shared__ float part[kGradWaves][BN];
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int slot = blockIdx.x / strips, strip = blockIdx.x - slot * strips;
  const int e = slot_expert(offsets, E, R, slot);
  const Rows rows = expert_rows(offsets, R, e);
  const int begin = rows.begin + (slot - (rows.begin / kGradRows + e)) * kGradRows;
  const int end = min(rows.end, begin + kGradRows);
  if (begin < rows.begin || begin >= end) return;
  const int col = strip * BN + lane * V;
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.f;
  if (col < N) {
    constexpr int U = 4;  // rows under way
    for (int r0 = begin + wave; r0 < end; r0 += U * kGradWaves) {
      u32x4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * kGradWaves;
        if (r < end) {
          a[u] = __builtin_nontemporal_load(
              reinterpret_cast<const u32x4*>(dy + (int64_t)r * N + col));
          if constexpr (ACT != kActNone)
            b[u] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4*>(z + (int64_t)r * N + col));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * kGradWaves;
        if (r >= end) break;
        typedef T tx __attribute__((ext_vector_type(16 / sizeof(T))));
        const tx g = __builtin_bit_cast(tx, a[u]);
        tx o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float v = Elt<T>::to_f32(g[j]);
          if constexpr (ACT != kActNone)
            v *= act_slope<ACT>(Elt<T>::to_f32(__builtin_bit_cast(tx, b[u])[j]));
          sum[j] += v;
          o[j] = Elt<T>::from_f32(v);
        }
        if (dz)
          *reinterpret_cast<u32x4*>(dz + (int64_t)r * N + col) = __builtin_bit_cast(u32x4, o);
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int j = 0; j < V; ++j) part[wave][lane * V + j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < BN; c += kGradWaves * kWave) {
    const int n = strip * BN + c;
    if (n >= N) break;
    float v = part[0][c];
#pragma unroll
    for (int w = 1; w < kGradWaves; ++w) v += part[w][c];
    partial[(int64_t)slot * N + n] = v;
  }
}

// db of 64 columns of one expert: the row tiles' sums in sixteen runs, and the runs, in order.
__global__ void __launch_bounds__(1024)
bias_sum_kernel(const float* __restrict__ partial, const int32_t* __restrict__ offsets,
                float* __restrict__ db, int R, int N) {
  __shared__ float part[16][kWave];
  const int wave = threadIdx.x / kWave, e = blockIdx.y, n = blockIdx.x * kWave + lane_id();
  const Rows rows = expert_rows(offsets, R, e);
  const int tiles = (max(rows.end - rows.begin, 0) + kGradRows - 1) / kGradRows;
  const int first = rows.begin / kGradRows + e, per = (tiles + 15) / 16;
  const int a = min(wave * per, tiles), b = min(a + per, tiles);
  float v = 0.f;
  for (int i = a; i < b; ++i) v += partial[(int64_t)(first + i) * N + n];
  part[wave][lane_id()] = v;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) v += part[w][lane_id()];
  db[(int64_t)e * N + n] = v;
}

template <class T>
static hipError_t run_linear_grad(int act, const T* dy, const T* z, const int32_t* offsets, T* dz,
                                  float* partial, int64_t R, int64_t E, int64_t N,
                                  hipStream_t s) {
  constexpr int BN = 16 / sizeof(T) * kWave;
  const int strips = (int)((N + BN - 1) / BN);
  const unsigned grid = (unsigned)(linear_grad_slots(R, E) * strips);
  return with_act(act, [&](auto tag) {
    linear_grad_kernel<T, decltype(tag)::value><<<grid, kGradWaves * kWave, 0, s>>>(
        dy, z, offsets, dz, partial, (int)R, (int)E, (int)N, strips);
    return hipGetLastError();
  });
}

hipError_t launch_linear_grad(int dtype, int act, const void* dy, const void* z,
                              const int32_t* offsets, void* dz, float* db, float* partial,
                              int64_t R, int64_t E, int64_t N, hipStream_t s) {
  hipError_t e = hipSuccess;
  float* sums = db ? partial : nullptr;
  if (R > 0 && (dz || db))
    e = dtype == 1 ? run_linear_grad<bf16>(act, (const bf16*)dy, (const bf16*)z, offsets, (bf16*)dz,
                                           sums, R, E, N, s)
                   : run_linear_grad<float>(act, (const float*)dy, (const float*)z, offsets,
                                            (float*)dz, sums, R, E, N, s);
  if (e != hipSuccess || !db) return e;
  bias_sum_kernel<<<dim3((unsigned)(N / kWave), (unsigned)E), 1024, 0, s>>>(partial, offsets, db,
                                                                          (int)R, (int)N);
  return hipGetLastError();
}

}  // namespace moe
