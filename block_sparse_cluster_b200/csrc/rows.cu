// Row operators of a layer's hidden states: root-mean-square norm with the residual's addition, its
// form with an output in 8-bit codes, and the quantiser of plain rows and of attention heads.
//
//   v = x + r                                   (fp32; the sum is rounded only where it is stored)
//   norm:      out = v / sqrt(mean v^2 + eps) * w
//   norm_i8:   t = v w,  m = max |t|,  q = rint(127 t / m) (ties to even),
//              scale = m / (127 sqrt(mean v^2 + eps));  the norm's own factor cancels in q
//   quantize:  t = x,  scale = m / 127
// A row of zeros has scale 0 and codes 0; a row with an infinity or a NaN has scale NaN and codes 0.
//
// Codes are the nearest ones of the exact quotient: 127 t / m is formed in fp32, whose error is
// below 2^-14 here (six roundings of 2^-24 relative, times 127), and only where it lies that close to
// a border k + 1/2 is the code taken again in fp64, from the inputs.  The row's maximum is likewise
// found in fp32 and then taken in fp64 over the few elements within 2^-21 of it.
//
// One group of threads owns a row and keeps it in registers between the reduction and the output,
// so every input is read once and every output written once: the kernels are bound by HBM.
#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

enum { kNorm = 0, kNormI8 = 1, kQuantI8 = 2 };

constexpr int kMaxWarps = 32;

// The low bytes of four words as one word.
__device__ __forceinline__ uint32_t low_bytes(const uint32_t* q) {
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// The larger of a and |b|; a NaN wins over every number.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// 1.5 * 2^23: adding it to |u| <= 2^22 rounds u to the nearest integer, ties to even, and leaves that integer in the sum's
// low bits, from where a code is taken as a byte without a conversion.
constexpr float kRound = 12582912.f;

template <int V>
struct Pack;   // V consecutive elements as one aligned load
template <>
struct Pack<1> {
  static __device__ __forceinline__ void load(const float* p, float* o) { o[0] = *p; }
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* o) { o[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) { *p = __float2bfloat16_rn(v[0]); }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) { *p = (int8_t)q[0]; }
};
template <>
struct Pack<4> {
  static __device__ __forceinline__ void load(const float* p, float* o) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) {
    *reinterpret_cast<uint32_t*>(p) = low_bytes(q);
  }
};
template <>
struct Pack<8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* o) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) {
    *reinterpret_cast<uint2*>(p) = make_uint2(low_bytes(q), low_bytes(q + 4));
  }
};

// Rows are walked as [tokens][heads][head_dim]; a plain matrix has one head.
struct RowArgs {
  const void* x;
  const void* residual;   // or null
  const void* weight;     // or null (1)
  void* sum_out;          // or null
  void* out;              // elements, or codes
  float* scale;           // codes only
  long long rows;
  int width, head_dim;
  int head_shift;         // log2 head_dim, or -1
  int tokens;             // rows of one batch entry (blockIdx.y)
  long long x_batch, x_head, x_token, r_stride, sum_stride, out_stride;
  float eps;
};

// A warp (WARP_ROW) or the whole block owns a row.
template <typename T, int V, int VPT, int MODE, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : 512)
row_kernel(const RowArgs a) {
  __shared__ float s_sum[kMaxWarps];
  __shared__ uint32_t s_max[kMaxWarps];
  __shared__ unsigned long long s_top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gt = WARP_ROW ? lane : threadIdx.x;
  const int gsize = WARP_ROW ? 32 : blockDim.x;
  const int token = WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  if (WARP_ROW && token >= a.tokens) return;
  const long long row = (long long)blockIdx.y * a.tokens + token;
  const T* x = static_cast<const T*>(a.x) + blockIdx.y * a.x_batch + token * a.x_token;
  const T* r = MODE != kQuantI8 && a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
  const T* w = MODE != kQuantI8 ? static_cast<const T*>(a.weight) : nullptr;
  auto x_at = [&](int c) -> const T* {
    if (MODE != kQuantI8) return x + c;
    const int h = a.head_shift >= 0 ? c >> a.head_shift : c / a.head_dim;
    return x + h * a.x_head + (c - h * a.head_dim);
  };

  float v[VPT][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * gsize + gt) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    if (c < a.width) {
      Pack<V>::load(x_at(c), v[i]);
      if (r) {
        float rv[V];
        Pack<V>::load(r + c, rv);
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] += rv[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(v[i][e], v[i][e], ss);
  }

  // t = v w; its sum of squares is v's
  float t[MODE == kNorm ? 1 : VPT][V];
  float mine = 0.f;
  if (MODE != kNorm) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * gsize + gt) * V;
      float wv[V];
#pragma unroll
      for (int e = 0; e < V; ++e) wv[e] = 1.f;
      if (w && c < a.width) Pack<V>::load(w + c, wv);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        t[i][e] = MODE == kNormI8 ? v[i][e] * wv[e] : v[i][e];
        mine = max_abs(mine, t[i][e]);
      }
    }
  }
  uint32_t top = __float_as_uint(mine);   // not negative: orders as an integer, a NaN above all

  // sums and maxima over the group, in a fixed order
  if (MODE != kQuantI8) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (MODE != kNorm) top = __reduce_max_sync(0xffffffffu, top);
  if (!WARP_ROW) {
    if (lane == 0) {
      s_sum[warp] = ss;
      s_max[warp] = top;
    }
    if (threadIdx.x == 0) s_top = 0;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    ss = lane < nw ? s_sum[lane] : 0.f;
    top = lane < nw ? s_max[lane] : 0u;
    if (MODE != kQuantI8) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (MODE != kNorm) top = __reduce_max_sync(0xffffffffu, top);
  }
  const float rms = MODE == kQuantI8 ? 1.f : rsqrtf(ss / (float)a.width + a.eps);

  if (MODE == kNorm) {
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
    T* sum = a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_stride : nullptr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * gsize + gt) * V;
      if (c < a.width) {
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = v[i][e] * rms;
        if (w) {
          float wv[V];
          Pack<V>::load(w + c, wv);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] *= wv[e];
        }
        if (sum) Pack<V>::store(sum + c, v[i]);
        Pack<V>::store(out + c, o);
      }
    }
    return;
  }

  const float m = __uint_as_float(top);
  // t of one element in fp64, from the inputs
  auto exact_t = [&](int c) -> double {
    double d = to_f32(*x_at(c));
    if (r) d += to_f32(r[c]);
    if (w) d *= to_f32(w[c]);
    return d;
  };
  double m64 = m;
  if (MODE == kNormI8) {
    unsigned long long best = 0;
    const float close = m * (1.f - 4.76837158e-7f);   // 1 - 2^-21
    if (mine >= close) {   // few threads; none where m is not finite, but infinity, whose row is answered below
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (fabsf(t[i][e]) >= close) {
            const int c = (i * gsize + gt) * V + e;
            if (c < a.width) best = max(best, (unsigned long long)__double_as_longlong(fabs(exact_t(c))));
          }
        }
      }
    }
    if (WARP_ROW) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    } else {
      if (best) atomicMax(&s_top, best);   // a maximum: the order does not matter
      __syncthreads();
      best = s_top;
    }
    m64 = __longlong_as_double((long long)best);
  }
  const bool finite = m < INFINITY;
  if (gt == 0) a.scale[row] = finite ? m * (1.f / 127.f) * (m > 0.f ? rms : 1.f) : __uint_as_float(0x7fffffffu);
  // below 1e-30 the fp32 quotient may lose more than its error bound (subnormal t, 127 / m infinite)
  const bool tiny = m < 1e-30f;
  const float inv = finite ? 127.f / m : 0.f;
  int8_t* q = static_cast<int8_t*>(a.out) + row * a.out_stride;
  T* sum = MODE == kNormI8 && a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_stride : nullptr;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * gsize + gt) * V;
    if (c < a.width) {
      uint32_t code[V];
      float far = 0.f;   // the largest distance of a quotient from its code
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = t[i][e] * inv, k = u + kRound;
        code[e] = __float_as_uint(k);
        far = fmaxf(far, fabsf(u - (k - kRound)));
      }
      if (tiny || far > 0.5f - 6.1035156e-5f) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          code[e] = m > 0.f ? (uint32_t)(int)rint(exact_t(c + e) * 127.0 / m64) : 0u;
      }
      if (!finite) {
#pragma unroll
        for (int e = 0; e < V; ++e) code[e] = 0u;
      }
      Pack<V>::store_codes(q + c, code);
      // the sum last: its buffer may be an input's, which the fp64 codes read again
      if (sum) Pack<V>::store(sum + c, v[i]);
    }
  }
}

// A row of up to 128 vectors is a warp's, so that it needs no barrier; longer ones take the block that holds them
// with VPT vectors a thread in at most 512 threads.
template <typename T, int V, int MODE>
cudaError_t launch_rows_v(const RowArgs& a, cudaStream_t s) {
  const int nvec = (a.width + V - 1) / V;
  const unsigned batch = (unsigned)(a.rows / a.tokens);
  if (nvec <= 128) {
    const dim3 grid((unsigned)((a.tokens + 3) / 4), batch);
    if (nvec <= 32) row_kernel<T, V, 1, MODE, true><<<grid, 128, 0, s>>>(a);
    else if (nvec <= 64) row_kernel<T, V, 2, MODE, true><<<grid, 128, 0, s>>>(a);
    else row_kernel<T, V, 4, MODE, true><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
  }
  const dim3 grid((unsigned)a.tokens, batch);
  auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  if (nvec <= 1024) row_kernel<T, V, 2, MODE, false><<<grid, threads(2), 0, s>>>(a);
  else if (nvec <= 2048) row_kernel<T, V, 4, MODE, false><<<grid, threads(4), 0, s>>>(a);
  else if (V < 8 && nvec <= 4096) row_kernel<T, V, V < 8 ? 8 : 4, MODE, false><<<grid, threads(8), 0, s>>>(a);
  else if (V < 4) row_kernel<T, V, V < 4 ? 32 : 4, MODE, false><<<grid, threads(32), 0, s>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

bool aligned_for(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The vector form needs every row of every tensor to start on the width of its vector.
template <typename T, int V, int MODE>
cudaError_t launch_rows_t(const RowArgs& a, cudaStream_t s) {
  const size_t in = sizeof(T) * V, out = MODE == kNorm ? in : (size_t)V;
  bool vec = a.width % V == 0 && a.head_dim % V == 0 && aligned_for(a.x, in) && a.x_batch % V == 0 &&
             a.x_head % V == 0 && a.x_token % V == 0 && aligned_for(a.out, out) && a.out_stride % V == 0;
  if (a.residual) vec = vec && aligned_for(a.residual, in) && a.r_stride % V == 0;
  if (a.sum_out) vec = vec && aligned_for(a.sum_out, in) && a.sum_stride % V == 0;
  if (a.weight) vec = vec && aligned_for(a.weight, in);
  return vec ? launch_rows_v<T, V, MODE>(a, s) : launch_rows_v<T, 1, MODE>(a, s);
}

template <int MODE>
cudaError_t launch_rows(bool bf16, const RowArgs& a, cudaStream_t s) {
  return bf16 ? launch_rows_t<__nv_bfloat16, 8, MODE>(a, s) : launch_rows_t<float, 4, MODE>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(bool bf16, long long rows, int width, const void* x, long long x_stride,
                            const void* residual, long long r_stride, const void* weight, float eps, void* sum_out,
                            long long sum_stride, void* out, long long out_stride, float* scale, cudaStream_t s) {
  const RowArgs a{x, residual, weight, sum_out, out, scale, rows, width, width, -1, (int)rows,
                  0, 0, x_stride, r_stride, sum_stride, out_stride, eps};
  return scale ? launch_rows<kNormI8>(bf16, a, s) : launch_rows<kNorm>(bf16, a, s);
}

cudaError_t launch_quantize_i8(bool bf16, int B, int H, int N, int d, const void* x, const da_head_strides& xs,
                               int8_t* q, long long q_stride, float* scale, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < d) ++shift;
  const RowArgs a{x, nullptr, nullptr, nullptr, q, scale, (long long)B * N, H * d, d, (1 << shift) == d ? shift : -1, N,
                  xs.batch, xs.head, xs.token, 0, 0, q_stride, 0.f};
  return launch_rows<kQuantI8>(bf16, a, s);
}

}  // namespace da
