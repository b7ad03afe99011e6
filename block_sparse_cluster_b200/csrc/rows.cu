// Row operators of a layer's hidden states: root-mean-square norm with the residual's addition, its
// form with an output in 8-bit codes, and the quantiser of plain rows and of attention heads.
//
//   v = x + r                                   (fp32; the sum is rounded only where it is stored)
//   norm:      out = v / sqrt(mean v^2 + eps) * w
//   norm_i8:   t = v w,  m = max |t|,  q = rint(127 t / m) (ties to even),
//              scale = m / (127 sqrt(mean v^2 + eps));  the norm's own factor cancels in q
//   quantize:  t = x,  scale = m / 127
// A row of zeros has scale 0 and codes 0; a row with an infinity or a NaN has scale NaN and codes 0.
// Where mean v^2 + eps leaves [kLeastMean, fp32's largest number), squares or their sum are no fp32 numbers any more (from
// about 1e17 on in wide rows, and with eps = 0 from about 1e-15 down): such a row is squared again, times a power of two.
//
// Codes are the nearest ones of the exact quotient.  fp32 gives t * (127 / m) to within kNear of it; where that lies
// so close to a border k + 1/2, the codes of the vector are taken again from the inputs, comparing 127 |t| with
// (k + 1/2) m in fp64.  The row's maximum is likewise found in fp32 and, where such a vector turns up, taken in fp64
// over the few elements within 2^-21 of it.
//
// A warp or a block owns a row and keeps it in registers between the reduction and the output, so every
// input is read once and every output written once.  The bound is HBM, but instructions are close behind (at HBM's rate
// an SM has 16 for each 32 elements of a bf16 row of codes): arithmetic is done on packed pairs, codes are
// rounded by one addition, and a thread holds many elements so that a row's fixed work is spread.  Walking the rows
// with as many blocks as the GPU holds, each row's loads ahead of the row in front, was slower (75600 x 5120 codes:
// 338 us against 264 then; norm: 481 against 451): the registers of the loads ahead cost more warps than they hide.
//
// Measured, bf16: norm with residual 75600 x 5120 451 us (6.86 TB/s, 1.07 of the plain copy's rate); codes of the norm with
// residual 75600 x 1536 130-135 us (6.0 TB/s), x 5120 420-455 us (6.2 TB/s: two barriers a row, and a third for the 46 % of the
// rows that need a second look); codes of 40 heads of 75600 tokens 194 us (6.0 TB/s).  Rows that do not start on 16 bytes are
// walked in pairs (bf16, even) or element by element: norm with residual 75600 x 1001 187 us in bf16 (0.5 of the copy's
// rate) and 189 in fp32 (1.0), codes 263 and 258 (0.3 and 0.6).
#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

enum { kNorm = 0, kNormI8 = 1, kQuantI8 = 2 };

constexpr int kMaxWarps = 16;

// 1.5 * 2^23: adding it to |u| <= 2^22 rounds u to the nearest integer, ties to even, and leaves that integer in the sum's
// low bits, from where a code is taken as a byte without a conversion.
constexpr float kRound = 12582912.f;

// bf16 rows without a norm: t = T 2^a and m = M 2^b with 8-bit integers T and M, so 127 t / m is a border k + 1/2 or
// misses it by a 254 * 255th of itself: |254 T - (2k + 1) M 2^(b - a)| is a whole number.  fp32's u = t * (127 / m), off by
// 2^-24, is first rounded to 18 bits, as h = p - (p - u) with p = 65 u: that moves it by at most 2^-18 of itself, onto the
// border in the one case (a border has 8 bits) and not as far as the border in the other.  Rounding h to an integer
// then sends ties to even, and no element needs a second look.
constexpr float kSplit = 65.f;

// How far t * (127 / m) may be from the exact quotient, with u = 2^-24: the quantiser's t and m are exact and 127 / m
// rounds once, 127 u < 2^-16; the norm's t rounds twice (sum, product) and so does the m taken from it: 5 * 127 u < 2^-14.
template <int MODE>
constexpr float kNear = MODE == kQuantI8 ? 1.52587891e-5f : 6.10351562e-5f;

// 2^-100.  A square below fp32's normal numbers is off by up to 2^-150, and so is the mean of them: 2^-50 of this, not seen.
constexpr float kLeastMean = 0x1p-100f;

__device__ __forceinline__ float max3_nan(float a, float b, float c) {   // a NaN wins over every number
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
    m = __vimax3_u32(m, __float_as_uint(fabsf(r.x)), __float_as_uint(fabsf(r.y)));
    return __vimax3_u32(m, __float_as_uint(fabsf(r.z)), __float_as_uint(fabsf(r.w)));
  }
  static __device__ __forceinline__ uint32_t max_float(uint32_t m) { return m; }
};
template <>
struct Pack<__nv_bfloat16, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw zero() { return 0; }
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ void unpack(Raw r, float* o) {
    o[0] = __uint_as_float(r << 16);
    o[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
  }
  static __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t* q) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)__byte_perm(q[0], q[1], 0x0040);
  }
  // two maxima side by side, in the halves of a word
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m, Raw r) { return __vmaxu2(m, r & 0x7fff7fffu); }
  static __device__ __forceinline__ uint32_t max_float(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
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
    m = __vimax3_u16x2(m, r.x & 0x7fff7fffu, r.y & 0x7fff7fffu);
    return __vimax3_u16x2(m, r.z & 0x7fff7fffu, r.w & 0x7fff7fffu);
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
  int tokens;             // rows of one batch entry (blockIdx.y)
  long long x_batch, x_head, x_token, r_stride, sum_stride, out_stride;
  float eps, inv_width;
  long long x_step;       // from a thread's vector of x to its next one, or -1 where that is not the same for all
  uint32_t per_head;      // ceil(2^32 / head_dim): columns and head_dim are at most 2^14, so column * per_head >> 32 is the head
};

// Element c of a row of x.
__device__ __forceinline__ long long x_offset(const RowArgs& a, int c) {
  const int h = a.head_dim == 1 ? c : (int)__umulhi((uint32_t)c, a.per_head);
  return h * a.x_head + (c - h * a.head_dim);
}

// t = (x + r) w in fp64 of the V elements from column c on, of a norm.
template <typename T, int V>
__device__ __forceinline__ void exact_t(const T* x, const T* r, const T* w, int c, double* t) {
  using P = Pack<T, V>;
  float f[V];
  P::unpack(P::load(x + c), f);
#pragma unroll
  for (int e = 0; e < V; ++e) t[e] = f[e];
  if (r) {
    P::unpack(P::load(r + c), f);
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] += f[e];
  }
  if (w) {
    P::unpack(P::load(w + c), f);
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] *= f[e];
  }
}

// The power of two that brings the row into fp32's range once mean v^2 + eps has left [kLeastMean, infinity).  Above:
// some |v| >= 2^57 (2^14 columns), and 2^14 (2^(128 - 72))^2 is still a number.  Below: 2^-43 > |v|, whose shifted squares sum to
// less than 2^114, and the smallest subnormal becomes 2^-49.  A NaN stays one.
__device__ __forceinline__ float wide_shift(float mean) { return mean < kLeastMean ? 0x1p100f : 0x1p-72f; }

// 1 / sqrt(mean + eps) of the row divided by shift, from a thread's part of the sum of (v shift)^2; in a fixed order.
// part: the block's scratch, when it owns the row.
template <bool WARP_ROW>
__device__ __forceinline__ float wide_root(float squares, float shift, float inv_width, float eps, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, o);
  if (!WARP_ROW) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = squares;
    __syncthreads();
    squares = 0.f;
#pragma unroll 1
    for (int i = 0; i < (int)blockDim.x >> 5; ++i) squares += part[i];
  }
  return rsqrtf(squares * inv_width + eps * shift * shift);
}

// The norm's output of a wide row, from the inputs.  A thread reads a vector before it writes it, so that sum and out may be the
// inputs' buffers.
template <typename T, int V, bool WARP_ROW>
__device__ __noinline__ void wide_norm(const T* x, const T* r, const T* w, T* sum, T* out, int first, int width, int step,
                                       float inv_width, float eps, float mean, float* part) {
  using P = Pack<T, V>;
  const float shift = wide_shift(mean);
  float f[V], g[V], squares = 0.f;
  auto load_v = [&](int c) {
    P::unpack(P::load(x + c), f);
    if (r) {
      P::unpack(P::load(r + c), g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] += g[e];
    }
  };
#pragma unroll 1
  for (int c = first; c < width; c += step) {
    load_v(c);
#pragma unroll
    for (int e = 0; e < V; ++e) squares = fmaf(f[e] * shift, f[e] * shift, squares);
  }
  const float root = wide_root<WARP_ROW>(squares, shift, inv_width, eps, part);
#pragma unroll 1
  for (int c = first; c < width; c += step) {
    load_v(c);
    if (sum) P::store(sum + c, f);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = f[e] * shift * root;
    if (w) {
      P::unpack(P::load(w + c), g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] *= g[e];
    }
    P::store(out + c, f);
  }
}

// The norm's codes, scale and sum of a row of which fp32 loses the statistics or the t; as in wide_norm.  top: zero, the
// block's scratch, when it owns the row.  In place: a call costs the rows around it more (75600 x 2048: 211 us, 183 so).
template <typename T, int V, bool WARP_ROW>
__device__ __forceinline__ void wide_codes(const T* x, const T* r, const T* w, T* sum, int8_t* q, float* scale, int first, int width, int step,
                                           float inv_width, float eps, float shift, float* part, unsigned long long* top) {
  using P = Pack<T, V>;
  float squares = 0.f;
  unsigned long long best = 0;   // bits of max |t|, which order as integers
#pragma unroll 1
  for (int c = first; c < width; c += step) {
    double t[V];
    exact_t<T, V>(x, r, nullptr, c, t);
#pragma unroll
    for (int e = 0; e < V; ++e) squares = fmaf((float)t[e] * shift, (float)t[e] * shift, squares);
    exact_t<T, V>(x, r, w, c, t);
#pragma unroll
    for (int e = 0; e < V; ++e) best = max(best, (unsigned long long)__double_as_longlong(fabs(t[e])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (!WARP_ROW && (threadIdx.x & 31) == 0) atomicMax(top, best);
  const float root = wide_root<WARP_ROW>(squares, shift, inv_width, eps, part);   // the block's barrier is in it
  if (!WARP_ROW) best = *top;
  const double m = __longlong_as_double((long long)best);
  if (first == 0) *scale = m > 0.0 ? (float)(m * root * shift * (1.0 / 127.0)) : 0.f;
#pragma unroll 1
  for (int c = first; c < width; c += step) {
    double t[V];
    uint32_t code[V];
    exact_t<T, V>(x, r, w, c, t);
#pragma unroll
    for (int e = 0; e < V; ++e) code[e] = m > 0.0 ? (uint32_t)(int)rint(127.0 * t[e] / m) : 0;
    P::store_codes(q + c, code);
    if (sum) {
      float f[V];
      exact_t<T, V>(x, r, nullptr, c, t);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = (float)t[e];
      P::store(sum + c, f);
    }
  }
}

// The blocks of an SM that a form is compiled for (0: the compiler's choice): their registers bound the warps that hide the
// loads. The codes of the norm hold the most: rows of 1536 in warps, 129 us with 96 registers, 139 with the 110 of the free
// choice; rows of 5120 in blocks, 421 us with 64, 553 with 80. The short rows are not held to it (96 wide: 29 us, 34 held).
template <int V, int VPT, int MODE, int MAX_THREADS>
constexpr int kBlocks = MODE != kNormI8 || V <= 2 ? 0
                        : MAX_THREADS == 128 ? (VPT * V >= 48 ? 5 : 0)
                        : MAX_THREADS == 256 ? 4
                                             : 0;

// A warp (blocks of 128 threads) or the whole block owns a row; each of its threads holds VPT vectors of V elements.
template <typename T, int V, int VPT, int MODE, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, (kBlocks<V, VPT, MODE, MAX_THREADS>))
row_kernel(const RowArgs a) {
  constexpr bool WARP_ROW = MAX_THREADS == 128;
  using P = Pack<T, V>;
  constexpr int E = VPT * V;                  // elements of a thread
  constexpr int kChunk = V < 2 ? 2 : V;       // elements that are worked on together: a vector, or a pair of single ones
  static_assert(E % kChunk == 0 && VPT <= 32, "elements are worked on in pairs, and vectors noted in 32 bits");
  constexpr bool kCodes = MODE != kNorm, kScaled = MODE != kQuantI8;   // codes come out; the norm's factor is formed
  constexpr bool kSnaps = !kScaled && sizeof(T) == 2;
  __shared__ float s_sum[kMaxWarps];
  __shared__ uint32_t s_max[kMaxWarps];
  __shared__ unsigned long long s_top;
  __shared__ float s_wide[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gt = WARP_ROW ? lane : threadIdx.x;
  const int gsize = WARP_ROW ? 32 : blockDim.x;
  const int token = WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  if (WARP_ROW && token >= a.tokens) return;
  const long long row = (long long)blockIdx.y * a.tokens + token;
  const T* x = static_cast<const T*>(a.x) + blockIdx.y * a.x_batch + token * a.x_token;
  const T* r = kScaled && a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
  const T* w = kScaled ? static_cast<const T*>(a.weight) : nullptr;
  auto column = [&](int i) { return (i * gsize + gt) * V; };
  auto inside = [&](int i) { return min(column(i), a.width - V); };   // a vector of the row for every thread

  // the row: the quantiser keeps it as it was loaded, the norms as fp32 sums in pairs
  typename P::Raw raw[VPT], res[kScaled ? VPT : 1];
  uint64_t v[kScaled ? E / 2 : 1];
  if (kScaled) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      raw[i] = P::zero();
      if (column(i) < a.width) raw[i] = P::load(x + column(i));
    }
  } else if (a.x_step >= 0) {   // threads beyond the row repeat vectors of it, which change no maximum
    const T* x0 = x + x_offset(a, inside(0));
#pragma unroll
    for (int i = 0; i < VPT; ++i) raw[i] = P::load(column(i) < a.width ? x0 + i * a.x_step : x);
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) raw[i] = P::load(x + x_offset(a, inside(i)));
  }
  if (kScaled) {
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
  // t = v w of chunk k in pairs; weights come from L1 each time, so that they take no registers
  auto chunk_t = [&](bool weighted, int k, uint64_t (&t)[kChunk / 2]) {
    if (!kScaled || weighted) {
      float f[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; e += V) {
        const int i = (k * kChunk + e) / V;
        P::unpack(kScaled ? P::load(w + inside(i)) : raw[i], f + e);
      }
#pragma unroll
      for (int e = 0; e < kChunk; e += 2) t[e / 2] = f2_pack(f[e], f[e + 1]);
    }
    if (kScaled) {
#pragma unroll
      for (int e = 0; e < kChunk; e += 2) {
        const uint64_t ve = v[(k * kChunk + e) / 2];
        t[e / 2] = weighted ? f2_mul(ve, t[e / 2]) : ve;
      }
    }
  };
  // f(k, t) for every chunk; whether there is a weight is decided once, outside the loop
  auto for_chunks = [&](auto f) {
    if (kScaled && w) {
#pragma unroll
      for (int k = 0; k < E / kChunk; ++k) {
        uint64_t t[kChunk / 2];
        chunk_t(true, k, t);
        f(k, t);
      }
    } else {
#pragma unroll
      for (int k = 0; k < E / kChunk; ++k) {
        uint64_t t[kChunk / 2];
        chunk_t(false, k, t);
        f(k, t);
      }
    }
  };

  float ss = 0.f;
  uint32_t mine = 0;   // bits of the thread's max |t|: not negative, so it orders as an integer, a NaN above all
  if (kScaled) {
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
    float high = 0.f, low = 0.f;
    for_chunks([&](int, uint64_t (&t)[kChunk / 2]) {
#pragma unroll
      for (int e = 0; e < kChunk; e += 2) {
        float lo, hi;
        f2_unpack(t[e / 2], lo, hi);
        high = max3_nan(high, lo, hi);
        low = fmin3(low, lo, hi);
      }
    });
    mine = max(__float_as_uint(fabsf(high)), __float_as_uint(fabsf(low)));
  }

  // sums and maxima over the row's threads, in a fixed order
  uint32_t top = mine;
  if (kScaled) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (kCodes) top = __reduce_max_sync(0xffffffffu, top);
  if (!WARP_ROW) {
    if (lane == 0) {
      s_sum[warp] = ss;
      s_max[warp] = top;
    }
    if (MODE == kNormI8 && threadIdx.x == 0) s_top = 0;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    if (kScaled) {
      ss = lane < nw ? s_sum[lane] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      ss = __shfl_sync(0xffffffffu, ss, 0);
    }
    if (kCodes) top = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
  }
  const float mean = ss * a.inv_width + a.eps;
  float rms = kScaled ? rsqrtf(mean) : 1.f;
  // the mean is no number of [kLeastMean, infinity), as one comparison of its bits; the same for the whole row
  const bool wide = kScaled && __float_as_uint(mean) - __float_as_uint(kLeastMean) >= 0x7f800000u - __float_as_uint(kLeastMean);
  auto shifted_squares = [&](float shift) {
    const uint64_t shift2 = f2_pack(shift, shift);
    uint64_t s2 = 0;
#pragma unroll
    for (int p = 0; p < (kScaled ? E / 2 : 0); ++p) {
      const uint64_t u = f2_mul(v[p], shift2);
      s2 = f2_fma(u, u, s2);
    }
    float lo, hi;
    f2_unpack(s2, lo, hi);
    return lo + hi;
  };

  T* sum = kScaled && a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_stride : nullptr;
  auto store_chunk = [&](T* p, int k, const uint64_t* t) {
    float f[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; e += 2) f2_unpack(t[e / 2], f[e], f[e + 1]);
#pragma unroll
    for (int e = 0; e < kChunk; e += V) {
      const int c = column((k * kChunk + e) / V);
      if (c < a.width) P::store(p + c, f + e);
    }
  };
  auto store_sum = [&]() {
    if (kScaled && sum) {
#pragma unroll
      for (int k = 0; k < E / kChunk; ++k) store_chunk(sum, k, v + k * kChunk / 2);
    }
  };

  if (MODE == kNorm) {
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
    // rows that take many registers leave them to a call (fp32 37000 x 5120: 220 us, 235 in place), others do it in place (bf16
    // 37000 x 1002 with the residual: 52 us, 57 with the call)
    if constexpr (E >= 16) {
      if (wide) {
        wide_norm<T, V, WARP_ROW>(x, r, w, sum, out, gt * V, a.width, gsize * V, a.inv_width, a.eps, mean, s_wide);
        return;
      }
    }
    store_sum();
    if (E < 16 && wide) {
      const float shift = wide_shift(mean);
      rms = wide_root<WARP_ROW>(shifted_squares(shift), shift, a.inv_width, a.eps, s_wide);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) v[p] = f2_mul(v[p], f2_pack(shift, shift));
    }
    const uint64_t rms2 = f2_pack(rms, rms);
    for_chunks([&](int k, uint64_t (&t)[kChunk / 2]) {
#pragma unroll
      for (int p = 0; p < kChunk / 2; ++p) t[p] = f2_mul(t[p], rms2);
      store_chunk(out, k, t);
    });
    return;
  }

  const float m = __uint_as_float(top);
  int8_t* q = static_cast<int8_t*>(a.out) + row * a.out_stride;
  if (!(m < INFINITY)) {   // an infinity or a NaN: the same for the whole row
    if (gt == 0) a.scale[row] = __uint_as_float(0x7fffffffu);
    const uint32_t none[kChunk] = {};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (column(i) < a.width) P::store_codes(q + column(i), none);
    store_sum();
    return;
  }
  // below 1e-30 fp32 may lose more than kNear (subnormal t, 127 / m infinite): every code in fp64, by division
  const bool tiny = m > 0.f && m < 1e-30f;
  if (kScaled && (wide || tiny)) {
    wide_codes<T, V, WARP_ROW>(x, r, w, sum, q, a.scale + row, gt * V, a.width, gsize * V, a.inv_width, a.eps, wide ? wide_shift(mean) : 1.f,
                               s_wide, &s_top);
    return;
  }
  if (gt == 0) a.scale[row] = m * (1.f / 127.f) * (m > 0.f ? rms : 1.f);
  const float inv = m >= 1e-30f ? 127.f / m : 0.f;
  uint32_t open = 0;   // vectors of this thread with an element next to a border, or all of them
  const uint64_t inv2 = f2_pack(inv, inv), round2 = f2_pack(kRound, kRound), minus2 = f2_pack(-1.f, -1.f);
  const uint64_t split2 = f2_pack(kSplit * inv, kSplit * inv), back2 = f2_pack(-inv, -inv);
  for_chunks([&](int k, uint64_t (&t)[kChunk / 2]) {
    uint32_t code[kChunk];
    float far = 0.f;   // the largest distance of a quotient from its code
#pragma unroll
    for (int e = 0; e < kChunk; e += 2) {
      uint64_t n;
      if (kSnaps) {
        const uint64_t p = f2_mul(t[e / 2], split2);
        n = f2_add(f2_fma(f2_fma(t[e / 2], back2, p), minus2, p), round2);
      } else {
        n = f2_fma(t[e / 2], inv2, round2);
      }
      float lo, hi;
      f2_unpack(n, lo, hi);
      code[e] = __float_as_uint(lo);
      code[e + 1] = __float_as_uint(hi);
      if (!kSnaps) {
        f2_unpack(f2_fma(t[e / 2], inv2, f2_fma(n, minus2, round2)), lo, hi);
        far = fmax3(far, fabsf(lo), fabsf(hi));
      }
    }
    if (far > 0.5f - kNear<MODE>) open |= (kChunk > V ? 3u : 1u) << (k * kChunk / V);
#pragma unroll
    for (int e = 0; e < kChunk; e += V) {
      const int c = column((k * kChunk + e) / V);
      if (c < a.width) P::store_codes(q + c, code + e);
    }
  });
  if (!kScaled && tiny) open = ~0u >> (32 - VPT);

  const bool any = !kScaled ? open != 0 : WARP_ROW ? __any_sync(0xffffffffu, open != 0) : __syncthreads_or(open != 0);
  if (any) {
    double m64 = m;
    if (MODE == kNormI8) {
      unsigned long long best = 0;
      const float close = m * (1.f - 4.76837158e-7f);   // 1 - 2^-21
      if (__uint_as_float(mine) >= close) {
        uint32_t near = 0;   // vectors with an element this close to the maximum
        for_chunks([&](int k, uint64_t (&t)[kChunk / 2]) {
          float high = 0.f;
#pragma unroll
          for (int e = 0; e < kChunk; e += 2) {
            float lo, hi;
            f2_unpack(t[e / 2], lo, hi);
            high = fmax3(high, fabsf(lo), fabsf(hi));
          }
          if (high >= close) near |= (kChunk > V ? 3u : 1u) << (k * kChunk / V);
        });
#pragma unroll 1
        for (; near; near &= near - 1) {
          const int c = column(__ffs((int)near) - 1);
          if (c >= a.width) continue;
          double t[V];
          exact_t<T, V>(x, r, w, c, t);
#pragma unroll
          for (int e = 0; e < V; ++e) best = max(best, (unsigned long long)__double_as_longlong(fabs(t[e])));
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
#pragma unroll 1
    for (; open; open &= open - 1) {
      const int c = column(__ffs((int)open) - 1);
      if (c >= a.width) continue;
      uint32_t code[V];
      if (!kScaled && tiny) {
        float f[V];
        P::unpack(P::load(x + x_offset(a, c)), f);
#pragma unroll
        for (int e = 0; e < V; ++e) code[e] = (uint32_t)(int)rint(127.0 * (double)f[e] / m64);
      } else if (MODE == kQuantI8) {
        // t and m are exact, so fp32 tells the side: 254 |t| against (2k + 1) m, the product in two parts, both
        // scaled down so that neither overflows
        float f[V];
        P::unpack(P::load(x + x_offset(a, c)), f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float size = fabsf(f[e]), k = truncf(size * inv), odd = fmaf(2.f, k, 1.f), ms = m * 0x1p-10f;
          const float high = odd * ms, low = fmaf(odd, ms, -high), d = fmaf(254.f, size * 0x1p-10f, -high);
          const int n = (int)k, up = d > low || (d == low && (n & 1));
          code[e] = (uint32_t)(f[e] < 0.f ? -(n + up) : n + up);
        }
      } else {
        double t[V];
        exact_t<T, V>(x, r, w, c, t);
#pragma unroll
        for (int e = 0; e < V; ++e) {   // k or k + 1, by the side of the border between them; on it, the even one
          const double size = 127.0 * fabs(t[e]);
          const float k = truncf(fabsf((float)t[e]) * inv);
          const double border = (double)(k + 0.5f) * m64;
          const int n = (int)k, up = size > border || (size == border && (n & 1));
          code[e] = (uint32_t)(t[e] < 0 ? -(n + up) : n + up);
        }
      }
      P::store_codes(q + c, code);
    }
  }
  // the sum last: its buffer may be an input's, which the fp64 codes read again
  store_sum();
}

// How far apart a thread's vectors of x lie, if its next one, `columns` further, is in the same place of a later head.
long long vector_step(const RowArgs& a, int columns) {
  if (a.head_dim == a.width) return columns;
  return columns % a.head_dim == 0 ? columns / a.head_dim * a.x_head : -1;
}

template <typename T, int V, int VPT, int MODE>
void launch_warp_rows(RowArgs a, unsigned batch, cudaStream_t s) {
  a.x_step = vector_step(a, 32 * V);
  row_kernel<T, V, VPT, MODE, 128><<<dim3((unsigned)((a.tokens + 3) / 4), batch), 128, 0, s>>>(a);
}
template <typename T, int V, int VPT, int MODE>
void launch_block_rows(RowArgs a, unsigned batch, int nvec, cudaStream_t s) {
  const int threads = ((nvec + VPT - 1) / VPT + 31) / 32 * 32;
  a.x_step = vector_step(a, threads * V);
  const dim3 grid((unsigned)a.tokens, batch);
  if constexpr (VPT != 8 && VPT != 16) {   // rows that take 8 or 16 vectors a thread fill more than 256 threads
    if (threads <= 256) {
      row_kernel<T, V, VPT, MODE, 256><<<grid, threads, 0, s>>>(a);
      return;
    }
  }
  row_kernel<T, V, VPT, MODE, 512><<<grid, threads, 0, s>>>(a);
}

// A row of up to 256 vectors is a warp's, so that it needs no barrier; longer ones take the block that holds them with
// VPT vectors a thread in at most 512 threads.
template <typename T, int V, int MODE>
cudaError_t launch_rows_v(const RowArgs& a, cudaStream_t s) {
  const int nvec = (a.width + V - 1) / V;
  const unsigned batch = (unsigned)(a.rows / a.tokens);
  if constexpr (V > 2) {
    if (nvec <= 32) launch_warp_rows<T, V, 1, MODE>(a, batch, s);
    else if (nvec <= 64) launch_warp_rows<T, V, 2, MODE>(a, batch, s);
    else if (nvec <= 128) launch_warp_rows<T, V, 4, MODE>(a, batch, s);
    else if (nvec <= 192) launch_warp_rows<T, V, 6, MODE>(a, batch, s);
    else if (nvec <= 256) launch_warp_rows<T, V, 8, MODE>(a, batch, s);
    else if (nvec <= 2048) launch_block_rows<T, V, 4, MODE>(a, batch, nvec, s);
    else if (V < 8 && nvec <= 4096) launch_block_rows<T, V, V < 8 ? 8 : 4, MODE>(a, batch, nvec, s);
    else return cudaErrorInvalidValue;
  } else {
    constexpr int kLast = V == 2 ? 16 : 32;
    if (nvec <= 128) launch_warp_rows<T, V, 4, MODE>(a, batch, s);
    else if (nvec <= 2048) launch_block_rows<T, V, 4, MODE>(a, batch, nvec, s);
    else if (nvec <= 4096) launch_block_rows<T, V, 8, MODE>(a, batch, nvec, s);
    else if (nvec <= 512 * kLast) launch_block_rows<T, V, kLast, MODE>(a, batch, nvec, s);
    else return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

bool aligned_for(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Vectors of V elements need every row of every tensor to start on their width.
template <typename T, int V, int MODE>
bool rows_fit(const RowArgs& a) {
  const size_t in = sizeof(T) * V, out = MODE == kNorm ? in : (size_t)V;
  bool vec = a.width % V == 0 && a.head_dim % V == 0 && aligned_for(a.x, in) && a.x_batch % V == 0 &&
             a.x_head % V == 0 && a.x_token % V == 0 && aligned_for(a.out, out) && a.out_stride % V == 0;
  if (a.residual) vec = vec && aligned_for(a.residual, in) && a.r_stride % V == 0;
  if (a.sum_out) vec = vec && aligned_for(a.sum_out, in) && a.sum_stride % V == 0;
  if (a.weight) vec = vec && aligned_for(a.weight, in);
  return vec;
}

// The reciprocal that x_offset multiplies by; a head of one element needs none (2^32 does not fit).
uint32_t per_head(int d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); }

// 16 bytes of a row a load, or the elements one by one (4 bytes in fp32).  In bf16 pairs come between: 37000 rows of 1002,
// norm 37 us and 66 one by one, codes 76 and 142; of 9002, 383 and 1020, 668 and 1650.
template <int MODE>
cudaError_t launch_rows(bool bf16, const RowArgs& a, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (!bf16) return rows_fit<float, 4, MODE>(a) ? launch_rows_v<float, 4, MODE>(a, s) : launch_rows_v<float, 1, MODE>(a, s);
  if (rows_fit<B, 8, MODE>(a)) return launch_rows_v<B, 8, MODE>(a, s);
  return rows_fit<B, 2, MODE>(a) ? launch_rows_v<B, 2, MODE>(a, s) : launch_rows_v<B, 1, MODE>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(bool bf16, long long rows, int width, const void* x, long long x_stride,
                            const void* residual, long long r_stride, const void* weight, float eps, void* sum_out,
                            long long sum_stride, void* out, long long out_stride, float* scale, cudaStream_t s) {
  const RowArgs a{x, residual, weight, sum_out, out, scale, rows, width, width, (int)rows,
                  0, 0, x_stride, r_stride, sum_stride, out_stride, eps, 1.f / (float)width, 0, per_head(width)};
  return scale ? launch_rows<kNormI8>(bf16, a, s) : launch_rows<kNorm>(bf16, a, s);
}

cudaError_t launch_quantize_i8(bool bf16, int B, int H, int N, int d, const void* x, const da_head_strides& xs,
                               int8_t* q, long long q_stride, float* scale, cudaStream_t s) {
  const RowArgs a{x, nullptr, nullptr, nullptr, q, scale, (long long)B * N, H * d, d, N,
                  xs.batch, xs.head, xs.token, 0, 0, q_stride, 0.f, 1.f, 0, per_head(d)};
  return launch_rows<kQuantI8>(bf16, a, s);
}

}  // namespace da
