// Product of 8-bit integer matrices with scales per token and channel, on the CUDA cores: for rows
// that do not start on 16 bytes, which the tensor-core path's tile loads cannot read.
//
//   out[m, n] = (sum_k x[m, k] w[n, k]) sx[m] sw[n] + bias[n]
// with the sum in 32-bit integers (exact for K <= 131071, the host's limit).  A CTA of 256 threads forms
// a 64 x 64 tile from 64-deep slices in shared memory, four products per dp4a instruction: 8e13 op/s (75600 x 5120 x 5120
// 49.6 ms, a fortieth of the tensor cores' rate).  Rows padded to 16 bytes avoid it, and the quantisers write such rows.
#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

constexpr int kT = 64;    // tile rows and columns
constexpr int kK = 64;    // depth of a slice
constexpr int kPitch = kK / 4 + 1;   // words of a tile row in shared memory

template <typename T>
__global__ void __launch_bounds__(256) linear_i8_simt_kernel(const LinearArgs a) {
  __shared__ uint32_t sx[kT][kPitch], sw[kT][kPitch];
  const long long m0 = (long long)blockIdx.x * kT;
  const int n0 = blockIdx.y * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kK) {
    for (int i = threadIdx.x; i < kT * (kK / 4); i += 256) {
      const int r = i / (kK / 4), k = k0 + 4 * (i % (kK / 4));
      uint32_t vx = 0, vw = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k + e < a.K) {
          if (m0 + r < a.M) vx |= (uint32_t)(uint8_t)a.x[(m0 + r) * a.x_stride + k + e] << (8 * e);
          if (n0 + r < a.N) vw |= (uint32_t)(uint8_t)a.w[(n0 + r) * a.w_stride + k + e] << (8 * e);
        }
      }
      sx[r][i % (kK / 4)] = vx;
      sw[r][i % (kK / 4)] = vw;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK / 4; ++k) {
      int va[4], vb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        va[i] = (int)sx[ty + 16 * i][k];
        vb[i] = (int)sw[tx + 16 * i][k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(va[i], vb[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty + 16 * i;
    if (m >= a.M) continue;
    T* row = static_cast<T*>(a.out) + (m / a.tokens) * a.out_batch + (m % a.tokens) * a.out_token;
    const float s = a.x_scale[m];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= a.N) continue;
      const float v = fmaf((float)acc[i][j] * s, a.w_scale[n], a.bias ? a.bias[n] : 0.f);
      store_out(row + (n / a.d) * a.out_head + n % a.d, v);
    }
  }
}

}  // namespace

cudaError_t launch_linear_i8_simt(bool bf16, const LinearArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.M + kT - 1) / kT), (unsigned)((a.N + kT - 1) / kT));
  if (bf16) linear_i8_simt_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  else linear_i8_simt_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace da
