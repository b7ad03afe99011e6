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
// Codes are the nearest ones of the exact quotient.  fp32 gives t * (127 / m) to within kNear of it; only where
// that lies so close to a border k + 1/2 is the side decided by comparing 127 |t| with (k + 1/2) m in fp64,
// from the inputs.  The row's maximum is likewise found in fp32 and, where such an element turns up, taken in
// fp64 over the few elements within 2^-21 of it.
//
// A warp or a block owns a row and keeps it in registers between the reduction and the output, so every
// input is read once and every output written once.  The bound is HBM, but instructions are close behind (a bf16 row
// of codes gives an SM 24 of them for each 32 elements at HBM's rate): arithmetic is done on packed pairs,
// codes are rounded by one addition, and a thread holds many elements so that a row's fixed work is spread.
#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

enum { kNorm = 0, kNormI8 = 1, kQuantI8 = 2 };

constexpr int kMaxWarps = 16;

// 1.5 * 2^23: adding it to |u| <= 2^22 rounds u to the nearest integer, ties to even, and leaves that integer in the sum's
// low bits, from where a code is taken as a byte without a conversion.
constexpr float kRound = 12582912.f;

// How far t * (127 / m) may be from the exact quotient, with u = 2^-24: the quantiser's t and m are exact and 127 / m
// rounds once, 127 u < 2^-16; the norm's t rounds twice (sum, product) and so does the m taken from it: 5 * 127 u < 2^-14.
template <int MODE>
constexpr float kNear = MODE == kQuantI8 ? 1.52587891e-5f : 6.10351562e-5f;

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest of a, |b| and |c|; a NaN wins over every number.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
// The low bytes of four words as one word.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// V consecutive elements of T as one load: raw words, floats and back.
template <typename T, int V>
struct Pack;
template <typename T>
struct Pack<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ Raw zero() { return T(0.f); }
  static __device__ __forceinline__ Raw load(const T* p) { return *p; }
  static __device__ __forceinline__ void unpack(Raw r, float* o) { o[0] = to_f32(r); }
  static __device__ __forceinline__ void store(T* p, const float* v) { store_out(p, v[0]); }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) { *p = (int8_t)q[0]; }
  // maximum of absolute values, as the bits of the elements (NaN above infinity)
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m, Raw r) { return max(m, __float_as_uint(fabsf(to_f32(r)))); }
  static __device__ __forceinline__ uint32_t max_float(uint32_t m) { return m; }
};
template <>
struct Pack<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const float4*>(p); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* o) {
    o[0] = r.x; o[1] = r.y; o[2] = r.z; o[3] = r.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) {
    *reinterpret_cast<uint32_t*>(p) = low_bytes(q[0], q[1], q[2], q[3]);
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m, const Raw& r) {
    m = max(max(m, __float_as_uint(fabsf(r.x))), __float_as_uint(fabsf(r.y)));
    return max(max(m, __float_as_uint(fabsf(r.z))), __float_as_uint(fabsf(r.w)));
  }
  static __device__ __forceinline__ uint32_t max_float(uint32_t m) { return m; }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* o) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
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
    *reinterpret_cast<uint2*>(p) = make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
  }
  // two maxima side by side, in the halves of a word
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m, const Raw& r) {
    m = __vmaxu2(__vmaxu2(m, r.x & 0x7fff7fffu), r.y & 0x7fff7fffu);
    return __vmaxu2(__vmaxu2(m, r.z & 0x7fff7fffu), r.w & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t max_float(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
};

// Rows are walked as [batch][tokens][heads][head_dim]; a plain matrix has one batch entry and one head.
struct RowArgs {
  const void* x;
  const void* residual;   // or null
  const void* weight;     // or null (1)
  void* sum_out;          // or null
  void* out;              // elements, or codes
  float* scale;           // codes only
  long long rows;
  int width, head_dim;
  int head_shift;         // log2 head_dim (30 with one head), or -1
  int tokens;             // rows of one batch entry (blockIdx.y)
  long long x_batch, x_head, x_token, r_stride, sum_stride, out_stride;
  float eps;
};

// A warp (WARP_ROW) or the whole block owns a row; each of its threads holds VPT vectors of V elements.
template <typename T, int V, int VPT, int MODE, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : 512)
row_kernel(const RowArgs a) {
  using P = Pack<T, V>;
  constexpr int E = VPT * V;   // elements of a thread, an even number
  static_assert(E % 2 == 0, "elements are worked on in pairs");
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
  auto column = [&](int i) { return (i * gsize + gt) * V; };

  // the row: the quantiser keeps it as it was loaded, the norms as fp32 sums in pairs
  typename P::Raw raw[VPT], res[MODE == kQuantI8 ? 1 : VPT];
  uint64_t v[MODE == kQuantI8 ? 1 : E / 2];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    raw[i] = P::zero();
    if (column(i) < a.width) raw[i] = P::load(x_at(column(i)));
  }
  if (MODE != kQuantI8) {
    if (r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        res[i] = P::zero();
        if (column(i) < a.width) res[i] = P::load(r + column(i));
      }
    }
    float f[E];
#pragma unroll
    for (int i = 0; i < VPT; ++i) P::unpack(raw[i], f + i * V);
#pragma unroll
    for (int p = 0; p < E / 2; ++p) v[p] = f2_pack(f[2 * p], f[2 * p + 1]);
    if (r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) P::unpack(res[i], f + i * V);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) v[p] = f2_add(v[p], f2_pack(f[2 * p], f[2 * p + 1]));
    }
  }
  // pairs of t = v w of the vectors that hold element pair p; weights come from L1 both times they are needed
  auto times_weight = [&](uint64_t (&t)[E / 2]) {
    if (MODE == kQuantI8) {
      float f[E];
#pragma unroll
      for (int i = 0; i < VPT; ++i) P::unpack(raw[i], f + i * V);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) t[p] = f2_pack(f[2 * p], f[2 * p + 1]);
    } else if (w) {
      float f[E];
#pragma unroll
      for (int i = 0; i < VPT; ++i) P::unpack(column(i) < a.width ? P::load(w + column(i)) : P::zero(), f + i * V);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) t[p] = f2_mul(v[p], f2_pack(f[2 * p], f[2 * p + 1]));
    } else {
#pragma unroll
      for (int p = 0; p < E / 2; ++p) t[p] = v[p];
    }
  };

  float ss = 0.f;
  uint32_t mine = 0;   // bits of the thread's max |t|: not negative, so it orders as an integer, a NaN above all
  if (MODE != kQuantI8) {
    uint64_t s2 = 0;
#pragma unroll
    for (int p = 0; p < E / 2; ++p) s2 = f2_fma(v[p], v[p], s2);
    float lo, hi;
    f2_unpack(s2, lo, hi);
    ss = lo + hi;
  }
  if (MODE == kQuantI8) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) mine = P::max_bits(mine, raw[i]);
    mine = P::max_float(mine);
  } else if (MODE == kNormI8) {
    uint64_t t[E / 2];
    times_weight(t);
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < E / 2; ++p) {
      float lo, hi;
      f2_unpack(t[p], lo, hi);
      top = max_abs(top, lo, hi);
    }
    mine = __float_as_uint(top);
  }

  // sums and maxima over the row's threads, in a fixed order
  uint32_t top = mine;
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
    if (MODE != kQuantI8) {
      ss = lane < nw ? s_sum[lane] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      ss = __shfl_sync(0xffffffffu, ss, 0);
    }
    if (MODE != kNorm) top = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
  }
  const float rms = MODE == kQuantI8 ? 1.f : rsqrtf(ss / (float)a.width + a.eps);
  T* sum = MODE != kQuantI8 && a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_stride : nullptr;
  auto store_sum = [&]() {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (column(i) < a.width) {
        float f[V < 2 ? 2 : V];
#pragma unroll
        for (int e = 0; e < V; e += 2) f2_unpack(v[(i * V + e) / 2], f[e], f[e + 1]);
        P::store(sum + column(i), V == 1 ? f + (i & 1) : f);
      }
  };

  if (MODE == kNorm) {
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
    if (sum) store_sum();
    uint64_t t[E / 2];
    times_weight(t);
    const uint64_t rms2 = f2_pack(rms, rms);
#pragma unroll
    for (int p = 0; p < E / 2; ++p) t[p] = f2_mul(t[p], rms2);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (column(i) < a.width) {
        float f[V < 2 ? 2 : V];
#pragma unroll
        for (int e = 0; e < V; e += 2) f2_unpack(t[(i * V + e) / 2], f[e], f[e + 1]);
        P::store(out + column(i), V == 1 ? f + (i & 1) : f);
      }
    return;
  }

  const float m = __uint_as_float(top);
  const bool finite = m < INFINITY;
  if (gt == 0) a.scale[row] = finite ? m * (1.f / 127.f) * (m > 0.f ? rms : 1.f) : __uint_as_float(0x7fffffffu);
  // below 1e-30 fp32 may lose more than kNear (subnormal t, 127 / m infinite): every code in fp64, by division
  const bool tiny = m > 0.f && m < 1e-30f;
  const float inv = finite && m >= 1e-30f ? 127.f / m : 0.f;
  int8_t* q = static_cast<int8_t*>(a.out) + row * a.out_stride;
  uint32_t open = 0;   // vectors of this thread with an element next to a border, or all of them
  uint64_t t[E / 2];
  times_weight(t);
  {
    const uint64_t inv2 = f2_pack(inv, inv), round2 = f2_pack(kRound, kRound), minus2 = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      uint32_t code[V < 2 ? 2 : V];
      float far = 0.f;   // the largest distance of a quotient from its code
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const uint64_t te = t[(i * V + e) / 2];
        const uint64_t k = f2_fma(te, inv2, round2);
        const uint64_t d = f2_fma(te, inv2, f2_fma(k, minus2, round2));
        float lo, hi;
        f2_unpack(k, lo, hi);
        code[e] = __float_as_uint(lo);
        code[e + 1] = __float_as_uint(hi);
        f2_unpack(d, lo, hi);
        if (V == 1) far = fabsf((i & 1) ? hi : lo);
        else far = fmax3(far, fabsf(lo), fabsf(hi));
      }
      if (!finite) {   // the same for the whole row; products of infinities and NaN are no codes
#pragma unroll
        for (int e = 0; e < (V < 2 ? 2 : V); ++e) code[e] = 0u;
        far = 0.f;
      }
      if (column(i) < a.width) {
        if (tiny || far > 0.5f - kNear<MODE>) open |= 1u << i;
        P::store_codes(q + column(i), V == 1 ? code + (i & 1) : code);
      }
    }
  }

  // t of one element in fp64, from the inputs
  auto exact_t = [&](int c) -> double {
    double d = to_f32(*x_at(c));
    if (r) d += to_f32(r[c]);
    if (w) d *= to_f32(w[c]);
    return d;
  };
  const bool any = MODE == kQuantI8 ? open != 0 : WARP_ROW ? __any_sync(0xffffffffu, open) : __syncthreads_or(open);
  if (any) {
    double m64 = m;
    if (MODE == kNormI8) {
      unsigned long long best = 0;
      const float close = tiny ? 0.f : m * (1.f - 4.76837158e-7f);   // 1 - 2^-21
      uint64_t near = 0;   // elements
      if (__uint_as_float(mine) >= close) {
#pragma unroll
        for (int p = 0; p < E / 2; ++p) {
          float lo, hi;
          f2_unpack(t[p], lo, hi);
          if (fabsf(lo) >= close) near |= 1ull << (2 * p);
          if (fabsf(hi) >= close) near |= 2ull << (2 * p);
        }
      }
      for (; near; near &= near - 1) {
        const int e = __ffsll((long long)near) - 1, c = column(e / V) + e % V;
        if (c < a.width) best = max(best, (unsigned long long)__double_as_longlong(fabs(exact_t(c))));
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
    uint64_t near = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (open >> i & 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float lo, hi;
          f2_unpack(t[(i * V + e) / 2], lo, hi);
          const float u = fabsf((i * V + e) & 1 ? hi : lo) * inv;
          if (tiny || fabsf(u - floorf(u) - 0.5f) < 2.f * kNear<MODE>) near |= 1ull << (i * V + e);
        }
      }
    }
    for (; near; near &= near - 1) {
      const int e = __ffsll((long long)near) - 1, c = column(e / V) + e % V;
      const double d = exact_t(c), size = 127.0 * fabs(d);
      double k;
      if (tiny) {
        k = rint(size / m64);
      } else {
        k = floorf(fabsf((float)d) * inv);   // below the border that t lies at
        const double border = (k + 0.5) * m64;
        if (size > border || (size == border && ((int)k & 1))) k += 1.0;
      }
      q[c] = (int8_t)(d < 0 ? -(int)k : (int)k);
    }
  }
  // the sum last: its buffer may be an input's, which the fp64 codes read again
  if (MODE == kNormI8 && sum) store_sum();
}

template <typename T, int V, int VPT, int MODE>
void launch_warp_rows(const RowArgs& a, unsigned batch, cudaStream_t s) {
  row_kernel<T, V, VPT, MODE, true><<<dim3((unsigned)((a.tokens + 3) / 4), batch), 128, 0, s>>>(a);
}
template <typename T, int V, int VPT, int MODE>
void launch_block_rows(const RowArgs& a, unsigned batch, int nvec, cudaStream_t s) {
  row_kernel<T, V, VPT, MODE, false><<<dim3((unsigned)a.tokens, batch), ((nvec + VPT - 1) / VPT + 31) / 32 * 32, 0, s>>>(a);
}

// A row of up to 256 vectors is a warp's, so that it needs no barrier; longer ones take the block that holds them with
// VPT vectors a thread in at most 512 threads.
template <typename T, int V, int MODE>
cudaError_t launch_rows_v(const RowArgs& a, cudaStream_t s) {
  const int nvec = (a.width + V - 1) / V;
  const unsigned batch = (unsigned)(a.rows / a.tokens);
  if constexpr (V > 1) {
    if (nvec <= 32) launch_warp_rows<T, V, 1, MODE>(a, batch, s);
    else if (nvec <= 64) launch_warp_rows<T, V, 2, MODE>(a, batch, s);
    else if (nvec <= 128) launch_warp_rows<T, V, 4, MODE>(a, batch, s);
    else if (nvec <= 192) launch_warp_rows<T, V, 6, MODE>(a, batch, s);
    else if (nvec <= 256) launch_warp_rows<T, V, 8, MODE>(a, batch, s);
    else if (nvec <= 2048) launch_block_rows<T, V, 4, MODE>(a, batch, nvec, s);
    else if (V < 8 && nvec <= 4096) launch_block_rows<T, V, V < 8 ? 8 : 4, MODE>(a, batch, nvec, s);
    else return cudaErrorInvalidValue;
  } else {
    if (nvec <= 128) launch_warp_rows<T, V, 4, MODE>(a, batch, s);
    else if (nvec <= 2048) launch_block_rows<T, V, 4, MODE>(a, batch, nvec, s);
    else if (nvec <= 4096) launch_block_rows<T, V, 8, MODE>(a, batch, nvec, s);
    else if (nvec <= 16384) launch_block_rows<T, V, 32, MODE>(a, batch, nvec, s);
    else return cudaErrorInvalidValue;
  }
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
  const RowArgs a{x, nullptr, nullptr, nullptr, q, scale, (long long)B * N, H * d, d, H == 1 ? 30 : (1 << shift) == d ? shift : -1, N,
                  xs.batch, xs.head, xs.token, 0, 0, q_stride, 0.f};
  return launch_rows<kQuantI8>(bf16, a, s);
}

}  // namespace da
