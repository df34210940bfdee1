// Tokens copied to the expert-sorted rows of their routes, and the gradient of
// that copy: with row(t, j) the row of route t*K + j,
//   rows[row(t, j), :] = x[t, :],      d x[t, :] = sum_j d rows[row(t, j), :].
// Both are bound by memory: a token's row is read once and written once for
// each of its routes (the gradient: the reverse), so the work goes by tokens and
// not by rows (4096 tokens of 14 KB to 8 rows each: 96 us by tokens, 127 by rows).
// One wave takes 1 KB of one token; lane j holds the row of slot j, which then reaches all lanes as a scalar.
#include "device.h"
#include "kernels.h"

namespace pmoe {

__device__ __forceinline__ int slot_rows(const int* row_of_route, long t, int K, int R, int lane) {
  const int r = lane < K ? row_of_route[t * K + lane] : -1;
  return r < R ? r : -1;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// kStream: more rows than the caches hold are stored past them (non-temporal): 96 us instead of 105.
template <bool kStream>
__global__ __launch_bounds__(256) void permute_kernel(const u32x4* __restrict__ x, const int* __restrict__ row_of_route,
                                                      long T, int K, int P, int chunks, u32x4* __restrict__ rows) {
  const int lane = threadIdx.x & 63;
  const long waves = (long)gridDim.x * 4;
  for (long w = (long)blockIdx.x * 4 + (threadIdx.x >> 6); w < T * chunks; w += waves) {
    const long t = w / chunks;
    const int p = (int)(w - t * chunks) * 64 + lane;
    const int mine = slot_rows(row_of_route, t, K, (int)(T * K), lane);
    if (__ballot(mine >= 0) == 0) continue;
    const u32x4 v = x[t * P + min(p, P - 1)];
    for (int j = 0; j < K; ++j) {
      const int r = __builtin_amdgcn_readlane(mine, j);
      if (r < 0 || p >= P) continue;
      if constexpr (kStream)
        __builtin_nontemporal_store(v, rows + (long)r * P + p);
      else
        rows[(long)r * P + p] = v;
    }
  }
}

// The sum is taken in FP32 in slot order from +0 and rounded once. 4095 tokens of 14 KB, 6 slots of
// which a quarter have rows: 26 us, 147 MB at 5.6 TB/s.
template <bool kF32>
__global__ __launch_bounds__(256) void permute_backward_kernel(const uint4* __restrict__ d_rows,
                                                               const int* __restrict__ row_of_route, long T, int K,
                                                               int R, int P, int chunks, uint4* __restrict__ dx) {
  constexpr int kE = kF32 ? 4 : 8;  // elements of a piece
  const int lane = threadIdx.x & 63;
  const long waves = (long)gridDim.x * 4;
  for (long w = (long)blockIdx.x * 4 + (threadIdx.x >> 6); w < T * chunks; w += waves) {
    const long t = w / chunks;
    const int p = (int)(w - t * chunks) * 64 + lane;
    const int mine = slot_rows(row_of_route, t, K, R, lane);
    float acc[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) acc[i] = 0.0f;
    for (int j = 0; j < K; ++j) {
      const int r = __builtin_amdgcn_readlane(mine, j);
      if (r < 0 || p >= P) continue;
      const uint4 u = d_rows[(long)r * P + p];
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kF32) {
          acc[i] += __uint_as_float(v[i]);
        } else {
          acc[2 * i] += __uint_as_float(v[i] << 16);
          acc[2 * i + 1] += __uint_as_float(v[i] & 0xFFFF0000u);
        }
      }
    }
    if (p >= P) continue;
    uint4 o;
    if constexpr (kF32)
      o = make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3]));
    else
      o = make_uint4(f32x2_to_bf16x2(acc[0], acc[1]), f32x2_to_bf16x2(acc[2], acc[3]),
                     f32x2_to_bf16x2(acc[4], acc[5]), f32x2_to_bf16x2(acc[6], acc[7]));
    dx[t * P + p] = o;
  }
}

static int wave_grid(long waves) {
  const long g = (waves + 3) / 4;
  return (int)(g < 1 << 20 ? g : 1 << 20);  // a launch has less than 2^32 threads
}

hipError_t launch_permute(const void* x, const int* row_of_route, int T, int K, long row_bytes, void* rows,
                          hipStream_t s) {
  const int P = (int)(row_bytes / 16), chunks = (P + 63) / 64;
  const int grid = wave_grid((long)T * chunks);
  const auto* xv = static_cast<const u32x4*>(x);
  auto* rv = static_cast<u32x4*>(rows);
  if ((long)T * K * row_bytes > 128L << 20)
    permute_kernel<true><<<grid, 256, 0, s>>>(xv, row_of_route, T, K, P, chunks, rv);
  else
    permute_kernel<false><<<grid, 256, 0, s>>>(xv, row_of_route, T, K, P, chunks, rv);
  return hipGetLastError();
}

hipError_t launch_permute_backward(const void* d_rows, bool f32, const int* row_of_route, int T, int K, int R, int H,
                                   void* dx, hipStream_t s) {
  const int P = f32 ? H / 4 : H / 8, chunks = (P + 63) / 64;
  const int grid = wave_grid((long)T * chunks);
  if (f32)
    permute_backward_kernel<true><<<grid, 256, 0, s>>>(static_cast<const uint4*>(d_rows), row_of_route, T, K, R, P,
                                                       chunks, static_cast<uint4*>(dx));
  else
    permute_backward_kernel<false><<<grid, 256, 0, s>>>(static_cast<const uint4*>(d_rows), row_of_route, T, K, R, P,
                                                        chunks, static_cast<uint4*>(dx));
  return hipGetLastError();
}

}  // namespace pmoe
