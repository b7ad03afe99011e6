// Product of 8-bit integer matrices with scales per token and channel, for a handful of rows of x.
//
//   out[m, n] = (sum_k x[m, k] w[n, k]) sx[m] sw[n] + bias[n]
// With up to kMaxRows rows the work is to read w once: 16 bytes of it meet 4 dp4a a row, which the CUDA cores do
// faster than HBM delivers.  A warp owns kCh channels and walks the depth in slices of 512 bytes, 16 a lane, several slices
// in flight; x comes from L1, once for the warp's channels.  Tiles, rings and tensor memory would only add latency here.
#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

constexpr int kMaxRows = 4;

__device__ __forceinline__ int dot16(const int4& a, const int4& b, int acc) {
  return __dp4a(a.w, b.w, __dp4a(a.z, b.z, __dp4a(a.y, b.y, __dp4a(a.x, b.x, acc))));
}

// The last K % 16 codes of a row, the rest zero: nothing behind the row is read.
__device__ __forceinline__ int4 tail16(const int8_t* p, int n) {
  int v[4] = {0, 0, 0, 0};
  for (int i = 0; i < n; ++i) v[i >> 2] |= (int)(uint8_t)p[i] << (8 * (i & 3));
  return make_int4(v[0], v[1], v[2], v[3]);
}

// w is read once and by nobody else: it need not stay in L1
__device__ __forceinline__ int4 load_once(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <typename T, int kRows, int kCh>
__global__ void __launch_bounds__(128) linear_i8_rows_kernel(const LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * kCh;
  if (n0 >= a.N) return;
  const int M = (int)a.M;
  const int8_t* w[kCh];
  const int8_t* x[kRows];
#pragma unroll
  for (int c = 0; c < kCh; ++c) w[c] = a.w + (long long)min(n0 + c, a.N - 1) * a.w_stride + lane * 16;
#pragma unroll
  for (int m = 0; m < kRows; ++m) x[m] = a.x + (long long)min(m, M - 1) * a.x_stride + lane * 16;
  int acc[kRows][kCh] = {};
  constexpr int kAhead = kCh >= 4 ? 2 : 4;   // slices in flight
  const int whole = a.K / 16 * 16;
  int k = 0;
  for (; k + (kAhead - 1) * 512 + lane * 16 < whole; k += kAhead * 512) {
    int4 wv[kAhead][kCh];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int c = 0; c < kCh; ++c) wv[s][c] = load_once(w[c] + k + s * 512);
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int m = 0; m < kRows; ++m) {
        const int4 xv = *reinterpret_cast<const int4*>(x[m] + k + s * 512);
#pragma unroll
        for (int c = 0; c < kCh; ++c) acc[m][c] = dot16(xv, wv[s][c], acc[m][c]);
      }
  }
  for (; k + lane * 16 < a.K; k += 512) {
    const int left = a.K - k - lane * 16;
    int4 wv[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) wv[c] = left >= 16 ? load_once(w[c] + k) : tail16(w[c] + k, left);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      const int4 xv = left >= 16 ? *reinterpret_cast<const int4*>(x[m] + k) : tail16(x[m] + k, left);
#pragma unroll
      for (int c = 0; c < kCh; ++c) acc[m][c] = dot16(xv, wv[c], acc[m][c]);
    }
  }
  int mine = 0;   // lane m * kCh + c keeps the sum of row m, channel c
#pragma unroll
  for (int m = 0; m < kRows; ++m)
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[m][c]);
      if (lane == m * kCh + c) mine = sum;
    }
  const int m = lane / kCh, n = n0 + lane % kCh;
  if (m < M && m < kRows && n < a.N) {
    const float v = fmaf((float)mine * a.x_scale[m], a.w_scale[n], a.bias ? a.bias[n] : 0.f);
    store_out(static_cast<T*>(a.out) + (m / a.tokens) * a.out_batch + (m % a.tokens) * a.out_token +
                  (long long)(n / a.d) * a.out_head + n % a.d, v);
  }
}

template <typename T, int kRows>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t s) {
  // four channels a warp share x, where that leaves every scheduler of the GPU a warp
  if (a.N >= 4 * 600) linear_i8_rows_kernel<T, kRows, 4><<<(a.N + 15) / 16, 128, 0, s>>>(a);
  else linear_i8_rows_kernel<T, kRows, 1><<<(a.N + 3) / 4, 128, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const LinearArgs& a, cudaStream_t s) {
  if (a.M == 1) return launch_rows<T, 1>(a, s);
  if (a.M == 2) return launch_rows<T, 2>(a, s);
  return launch_rows<T, 4>(a, s);
}

}  // namespace

bool linear_i8_rows_supported(const LinearArgs& a) { return a.M <= kMaxRows; }

cudaError_t launch_linear_i8_rows(bool bf16, const LinearArgs& a, cudaStream_t s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace da
