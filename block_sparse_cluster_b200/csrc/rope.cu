// Rotary positions over time, height and width, with the query/key norm in front of them.
//
// A head's d elements form d/2 pairs (a, b); pair p belongs to axis u (the first axis_dims[0] / 2
// pairs to time, and so on) and turns by angle = position_u * theta^(-2j / axis_dims[u]), j its
// index within the axis:  (a, b) -> (a cos - b sin, a sin + b cos).
// Positions come from the (time, height, width) grid of the token's index, or from the caller.
//
// Angles are formed in whole turns of 2^64: a frequency is a 64-bit fraction of a turn per position, and position times
// frequency modulo 2^64 is what is left of the angle after its whole turns, exactly, however far the position and whatever
// its sign.  Only the upper 32 bits, as half turns in [-1, 1), are rounded to fp32 for sincospif.
//
// A norm whose mean square (with eps) leaves [kLeastMean, fp32's largest number) is taken again of x times a power of two, as
// the row operators' norms are; behind the loop over the tokens, which only leaves out such heads' stores (a token's sums formed again
// in the loop cost 40 heads x 75600 tokens 10 us of 265).
//
// The kernel is bound by HBM: x is read once and out written once.  A thread's unit of work is two
// 16-byte vectors of a head, elements [j, j + V) and [j + d/2, j + d/2 + V): whole pairs in either pairing.
// A group of threads owns a token, all its heads (the norm over all heads needs them together); every unit of a
// thread has the same j, so its cosines and sines are loaded from shared memory once a token.  A group takes a run
// of tokens: the block forms the angles of all of them first, and each thread keeps the loads of the next kStages tokens
// in flight with cp.async, into shared memory that only it reads: loads ahead cost no registers and need no barrier.
//
// Measured, bf16, 40 heads of 128 and 75600 tokens (floor 241 us): 240 us without a norm, 246 with the head's, 256 with the
// norm over all heads, whose barrier a token is what is left; 12 heads, 32880 tokens (floor 31 us): 35, 39 and 44 us, where
// a token is 96 threads' work of 16 elements and its fixed instructions show.  fp32 runs at the copy's rate.
#include <math.h>

#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

constexpr int kMaxPairs = 64;   // d <= 128
constexpr int kMaxRun = 32;     // tokens of a block
constexpr int kStages = 3;      // tokens a thread holds in flight
constexpr int kMaxTurns = 16;   // tokens a group takes

enum { kNoNorm = 0, kHeadNorm = 1, kFullNorm = 2 };

struct RopeArgs {
  const void* x;
  void* out;
  const void* weight;
  const int* positions;        // [batch][N][3], or null: the grid
  long long pos_batch;
  int H, N;
  int heads_per_block;         // H, or less where a token's heads are spread over blocks
  int group;                   // threads of a token: a power of two up to 32, or the whole block
  int run;                     // tokens of a block
  long long xb, xh, xn, ob, oh, on;
  int grid[3];
  int norm, halves;
  float eps, inv_width;        // 1 / (H d)
  uint64_t freq[kMaxPairs];    // 2^-64 turns per position
  unsigned char axis[kMaxPairs];
};

// A unit's two raw vectors as V pairs: a[i] and b[i] hold the first and second elements of pairs 2i and 2i + 1, so that
// the rotation works on two pairs an instruction in either pairing.
template <typename T, bool HALVES>
struct Unit;

// (a, b) -> (a c - b s, a s + b c), two pairs at a time
template <int N>
__device__ __forceinline__ void rotate_pairs(uint64_t (&a)[N], uint64_t (&b)[N], const uint64_t (&c)[N], const uint64_t (&s)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const uint64_t t = a[e];
    a[e] = f2_fma(t, c[e], f2_mul(b[e], s[e] ^ 0x8000000080000000ull));
    b[e] = f2_fma(t, s[e], f2_mul(b[e], c[e]));
  }
}
template <bool HALVES>
struct Unit<__nv_bfloat16, HALVES> {
  static constexpr int n = 8;
  static __device__ __forceinline__ uint64_t low(uint32_t p, uint32_t q) {
    return f2_pack(__uint_as_float(p << 16), __uint_as_float(q << 16));
  }
  static __device__ __forceinline__ uint64_t high(uint32_t p, uint32_t q) {
    return f2_pack(__uint_as_float(p & 0xffff0000u), __uint_as_float(q & 0xffff0000u));
  }
  static __device__ __forceinline__ void unpack(const uint4 (&raw)[2], uint64_t (&a)[4], uint64_t (&b)[4]) {
    const uint32_t w[2][4] = {{raw[0].x, raw[0].y, raw[0].z, raw[0].w}, {raw[1].x, raw[1].y, raw[1].z, raw[1].w}};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (HALVES) {
        a[i] = f2_pack(__uint_as_float(w[0][i] << 16), __uint_as_float(w[0][i] & 0xffff0000u));
        b[i] = f2_pack(__uint_as_float(w[1][i] << 16), __uint_as_float(w[1][i] & 0xffff0000u));
      } else {
        a[i] = low(w[i / 2][2 * (i & 1)], w[i / 2][2 * (i & 1) + 1]);
        b[i] = high(w[i / 2][2 * (i & 1)], w[i / 2][2 * (i & 1) + 1]);
      }
    }
  }
  static __device__ __forceinline__ void rotate(uint64_t (&a)[4], uint64_t (&b)[4], const uint64_t (&c)[4], const uint64_t (&s)[4]) {
    rotate_pairs(a, b, c, s);
  }
  static __device__ __forceinline__ void pack(const uint64_t (&a)[4], const uint64_t (&b)[4], uint4 (&raw)[2]) {
    uint32_t w[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a0, a1, b0, b1;
      f2_unpack(a[i], a0, a1);
      f2_unpack(b[i], b0, b1);
      if (HALVES) {
        w[0][i] = pack_bf16x2(a0, a1);
        w[1][i] = pack_bf16x2(b0, b1);
      } else {
        w[i / 2][2 * (i & 1)] = pack_bf16x2(a0, b0);
        w[i / 2][2 * (i & 1) + 1] = pack_bf16x2(a1, b1);
      }
    }
    raw[0] = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
    raw[1] = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
  }
};
// fp32 vectors are taken as they lie: with adjacent pairs a[i] and b[i] are whole pairs of the first and second vector,
// and the rotation takes them apart (picking firsts and seconds together would cost moves; it was 10 % slower).
template <bool HALVES>
struct Unit<float, HALVES> {
  static constexpr int n = 4;
  static __device__ __forceinline__ uint64_t two(uint32_t p, uint32_t q) { return f2_pack(__uint_as_float(p), __uint_as_float(q)); }
  static __device__ __forceinline__ void unpack(const uint4 (&raw)[2], uint64_t (&a)[2], uint64_t (&b)[2]) {
    a[0] = two(raw[0].x, raw[0].y); a[1] = two(raw[0].z, raw[0].w);
    b[0] = two(raw[1].x, raw[1].y); b[1] = two(raw[1].z, raw[1].w);
  }
  static __device__ __forceinline__ uint64_t turn(uint64_t v, float c, float s) {
    float p, q;
    f2_unpack(v, p, q);
    return f2_pack(p * c - q * s, p * s + q * c);
  }
  static __device__ __forceinline__ void rotate(uint64_t (&a)[2], uint64_t (&b)[2], const uint64_t (&c)[2], const uint64_t (&s)[2]) {
    if (HALVES) {
      rotate_pairs(a, b, c, s);
    } else {
      float cs[4], sn[4];
      f2_unpack(c[0], cs[0], cs[1]); f2_unpack(c[1], cs[2], cs[3]);
      f2_unpack(s[0], sn[0], sn[1]); f2_unpack(s[1], sn[2], sn[3]);
      a[0] = turn(a[0], cs[0], sn[0]); a[1] = turn(a[1], cs[1], sn[1]);
      b[0] = turn(b[0], cs[2], sn[2]); b[1] = turn(b[1], cs[3], sn[3]);
    }
  }
  static __device__ __forceinline__ void pack(const uint64_t (&a)[2], const uint64_t (&b)[2], uint4 (&raw)[2]) {
    float v[8];
    f2_unpack(a[0], v[0], v[1]); f2_unpack(a[1], v[2], v[3]);
    f2_unpack(b[0], v[4], v[5]); f2_unpack(b[1], v[6], v[7]);
    raw[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    raw[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  }
};

// 2^-100: squares below fp32's normal numbers, each off by up to 2^-150, are not seen in such a mean.
constexpr float kLeastMean = 0x1p-100f;
__device__ __forceinline__ bool leaves_fp32(float mean) {   // as one comparison of the bits; a NaN does too
  return __float_as_uint(mean) - __float_as_uint(kLeastMean) >= 0x7f800000u - __float_as_uint(kLeastMean);
}
// The power of two that brings x into range.  Above: some |x| >= 2^57 (2^14 elements), and 2^14 (2^(128 - 72))^2 is still
// a number; elements that fall below 2^-126 by it are 2^110 below the rest.  Below: |x| < 2^-43, whose squares then sum to less
// than 2^114, and nothing is lost.
__device__ __forceinline__ float wide_shift(float mean) { return !leaves_fp32(mean) ? 1.f : mean < kLeastMean ? 0x1p100f : 0x1p-72f; }

// The heads or tokens of a run whose squares fp32 loses, which the loop over the tokens has not stored: x still holds them,
// whether or not out is x.  left: a bit a turn of the thread's group, and for the second of its units (a head's norm) kMaxTurns up.
// All threads that a sum joins call this together.
template <typename T, int D, int UPT, bool HALVES>
__device__ __noinline__ void rope_left(const RopeArgs& a, uint32_t left, int run, const float* s_cos, const int4* s_pos, float* s_wide) {
  using U = Unit<T, HALVES>;
  constexpr int V = U::n, kPerHead = D / 2 / V;
  const int groups = blockDim.x / a.group, g = threadIdx.x / a.group, gt = threadIdx.x - g * a.group;
  const int h0 = blockIdx.z * a.heads_per_block, units = min(a.heads_per_block, a.H - h0) * kPerHead;
  const int j = gt % kPerHead * V, head = h0 + gt / kPerHead, joined = a.norm == kHeadNorm ? kPerHead : a.group;
  const float* const s_sin = s_cos + a.run * (D / 2);
  auto total = [&](float v) {   // over the threads that a norm joins
    for (int o = min(joined, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (joined > 32) {
      if ((threadIdx.x & 31) == 0) s_wide[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0.f;
      for (int w = 0; w < blockDim.x >> 5; ++w) v += s_wide[w];
      __syncthreads();
    }
    return v;
  };
#pragma unroll 1
  for (int turn = 0; turn * groups < run; ++turn) {
#pragma unroll 1
    for (int i0 = 0; i0 < (a.norm == kHeadNorm ? min(UPT, 2) : 1); ++i0) {   // a head's norm: unit by unit; else all of them at once
      const bool mine = left >> (i0 * kMaxTurns + turn) & 1;
      if (!__any_sync(0xffffffffu, mine)) continue;
      const int k = turn * groups + g, n = blockIdx.x * a.run + k, end = a.norm == kHeadNorm ? i0 + 1 : UPT;
      uint64_t va[V / 2], vb[V / 2];
      auto load = [&](int i, float shift) {   // of a unit that is there
        const T* from = static_cast<const T*>(a.x) + blockIdx.y * a.xb + (long long)n * a.xn + (head + i * (a.group / kPerHead)) * a.xh + j;
        const uint4 raw[2] = {*reinterpret_cast<const uint4*>(from), *reinterpret_cast<const uint4*>(from + D / 2)};
        U::unpack(raw, va, vb);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          va[e] = f2_mul(va[e], f2_pack(shift, shift));
          vb[e] = f2_mul(vb[e], f2_pack(shift, shift));
        }
      };
      auto mean_of = [&](float shift) {
        float ss = 0.f;
#pragma unroll 1
        for (int i = i0; i < end; ++i) {
          if (!mine || gt + i * a.group >= units) continue;
          load(i, shift);
          uint64_t s2 = 0;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) s2 = f2_fma(va[e], va[e], f2_fma(vb[e], vb[e], s2));
          float lo, hi;
          f2_unpack(s2, lo, hi);
          ss += lo + hi;
        }
        return total(ss) * (a.norm == kHeadNorm ? 1.f / D : a.inv_width) + a.eps * shift * shift;
      };
      const float shift = wide_shift(mean_of(1.f)), root = rsqrtf(mean_of(shift));
#pragma unroll 1
      for (int i = i0; i < end; ++i) {
        if (!mine || gt + i * a.group >= units) continue;
        load(i, shift);
        const T* w = static_cast<const T*>(a.weight) + j + (a.norm == kFullNorm ? (gt + i * a.group) / kPerHead * D : 0);
        const uint4 wraw[2] = {*reinterpret_cast<const uint4*>(w), *reinterpret_cast<const uint4*>(w + D / 2)};
        uint64_t wa[V / 2], wb[V / 2], c[V / 2], s[V / 2];
        U::unpack(wraw, wa, wb);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          va[e] = f2_mul(f2_mul(va[e], f2_pack(root, root)), wa[e]);
          vb[e] = f2_mul(f2_mul(vb[e], f2_pack(root, root)), wb[e]);
        }
        if (s_pos[k].w != 0) {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const int at = k * (D / 2) + (HALVES ? j + 2 * e : j / 2 + e / (V / 4) * (D / 4) + e % (V / 4) * 2);
            c[e] = f2_pack(s_cos[at], s_cos[at + 1]);
            s[e] = f2_pack(s_sin[at], s_sin[at + 1]);
          }
          U::rotate(va, vb, c, s);
        }
        uint4 o2[2];
        U::pack(va, vb, o2);
        T* to = static_cast<T*>(a.out) + blockIdx.y * a.ob + (long long)n * a.on + (head + i * (a.group / kPerHead)) * a.oh + j;
        *reinterpret_cast<uint4*>(to) = o2[0];
        *reinterpret_cast<uint4*>(to + D / 2) = o2[1];
      }
    }
  }
}

// UPT: units a thread holds of a token.
template <typename T, int D, int UPT, bool HALVES, bool NORMED>
__global__ void __launch_bounds__(512) rope_kernel(const __grid_constant__ RopeArgs a) {
  using U = Unit<T, HALVES>;
  constexpr int V = U::n;
  constexpr int kPerHead = D / 2 / V;   // units of a head
  extern __shared__ __align__(16) uint4 s_ring[];   // [stage][unit][vector][thread]
  float* const s_cos = reinterpret_cast<float*>(s_ring + kStages * UPT * 2 * blockDim.x);   // [token of the run][pair]
  float* const s_sin = s_cos + a.run * (D / 2);
  __shared__ int4 s_pos[kMaxRun];   // time, height, width, whether the token turns at all
  __shared__ uint64_t s_freq[D / 2];
  __shared__ unsigned char s_axis[D / 2];
  __shared__ __align__(16) float s_part[2][16];
  __shared__ float s_wide[16];
  const int b = blockIdx.y, n0 = blockIdx.x * a.run, h0 = blockIdx.z * a.heads_per_block;
  const int run = min(a.run, a.N - n0);
  const int units = min(a.heads_per_block, a.H - h0) * kPerHead;
  const int groups = blockDim.x / a.group;
  const int g = threadIdx.x / a.group, gt = threadIdx.x - g * a.group;
  const int j = (gt % kPerHead) * V;    // the same for all units of a thread: group is a multiple of kPerHead
  const T* x = static_cast<const T*>(a.x) + b * a.xb + (h0 + gt / kPerHead) * a.xh + j;
  T* out = static_cast<T*>(a.out) + b * a.ob + (h0 + gt / kPerHead) * a.oh + j;

  // a thread's units lie the same number of heads apart in every token
  const long long x_step = a.group / kPerHead * a.xh, out_step = a.group / kPerHead * a.oh;
  auto has = [&](int i) { return gt + i * a.group < units; };
  // the stage that is read next, and filled again; the token that is fetched next
  uint4* const ring = s_ring + threadIdx.x;
  const int vec = blockDim.x, stage = UPT * 2 * vec;
  const T* next = x + (long long)(n0 + g) * a.xn;
  const long long x_turn = groups * a.xn;
  auto fetch = [&](int k, uint4* at) {   // token k of the run
    if (k < run) {
#pragma unroll
      for (int i = 0; i < UPT; ++i)
        if (has(i)) {
          cp_async16(at + (2 * i) * vec, next + i * x_step);
          cp_async16(at + (2 * i + 1) * vec, next + i * x_step + D / 2);
        }
    }
    next += x_turn;
    cp_async_commit();
  };
#pragma unroll
  for (int it = 0; it < kStages; ++it) fetch(g + it * groups, ring + it * stage);

  // weights of the thread's units, the same for every token
  uint4 wraw[NORMED ? UPT : 1][2];
  if (NORMED) {
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = gt + i * a.group;
      wraw[i][0] = wraw[i][1] = make_uint4(0, 0, 0, 0);
      if (u < units) {
        const T* w = static_cast<const T*>(a.weight) + j + (a.norm == kFullNorm ? u / kPerHead * D : 0);
        wraw[i][0] = *reinterpret_cast<const uint4*>(w);
        wraw[i][1] = *reinterpret_cast<const uint4*>(w + D / 2);
      }
    }
  }

  // positions of the run's tokens, and the frequencies out of the launch's constants (a warp reads those one at a time)
  for (int k = threadIdx.x; k < run; k += blockDim.x) {
    const unsigned n = (unsigned)(n0 + k);
    if (a.positions) {
      const int* pos = a.positions + b * a.pos_batch + (long long)n * 3;
      s_pos[k] = make_int4(pos[0], pos[1], pos[2], 1);
    } else {
      const unsigned line = n / (unsigned)a.grid[2], t = line / (unsigned)a.grid[1];
      s_pos[k] = make_int4((int)t, (int)(line - t * a.grid[1]), (int)(n - line * a.grid[2]), t < (unsigned)a.grid[0]);
    }
  }
  if (threadIdx.x < 32) (&s_part[0][0])[threadIdx.x] = 0.f;
  for (int p = threadIdx.x; p < D / 2; p += blockDim.x) {
    s_freq[p] = a.freq[p];
    s_axis[p] = a.axis[p];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < run * (D / 2); i += blockDim.x) {
    const int p = i % (D / 2);
    const int pos = reinterpret_cast<const int*>(&s_pos[i / (D / 2)])[s_axis[p]];
    const int turn = (int)(((uint64_t)(int64_t)pos * s_freq[p]) >> 32);   // 2^-31 half turns
    sincospif((float)turn * 0x1p-31f, &s_sin[i], &s_cos[i]);
  }
  __syncthreads();

  uint32_t left = 0;   // turns whose units are left to the end (rope_left)
  // every group takes the same number of turns, so that the barriers match
  uint4 raw[UPT][2];
#pragma unroll
  for (int i = 0; i < UPT; ++i) raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);   // stays so for units the thread lacks
  uint4* at = ring;
  T* o = out + (long long)(n0 + g) * a.on;
  const long long out_turn = groups * a.on;
  for (int k0 = 0, turn_no = 0; k0 < run; k0 += groups, ++turn_no, o += out_turn) {
    const int k = k0 + g, parity = turn_no & 1;
    auto bit = [&](int i) { return 1u << ((i & 1) * kMaxTurns + turn_no); };
    float ss = 0.f, factor[UPT];
    cp_async_wait<kStages - 1>();
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      if (has(i)) {   // behind the run's end, what an earlier turn left: worked on, not stored
        raw[i][0] = at[(2 * i) * vec];
        raw[i][1] = at[(2 * i + 1) * vec];
      }
      factor[i] = 1.f;
      if (NORMED) {
        uint64_t va[V / 2], vb[V / 2], s2 = 0;
        U::unpack(raw[i], va, vb);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) s2 = f2_fma(va[e], va[e], f2_fma(vb[e], vb[e], s2));
        float lo, hi;
        f2_unpack(s2, lo, hi);
        factor[i] = lo + hi;
        ss += factor[i];
      }
    }
    if (NORMED && a.norm == kHeadNorm) {
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
#pragma unroll
        for (int o = kPerHead / 2; o > 0; o >>= 1) factor[i] += __shfl_xor_sync(0xffffffffu, factor[i], o);
        const float mean = factor[i] * (1.f / D) + a.eps;
        factor[i] = rsqrtf(mean);
        if (k < run && has(i) && leaves_fp32(mean)) left |= bit(i);
      }
    } else if (NORMED) {
      for (int o = min(a.group, 32) / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (a.group > 32) {   // the block is the group: its warps' sums, in order; warps it lacks have left zeros
        if ((threadIdx.x & 31) == 0) s_part[parity][threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        for (int w = 0; w < blockDim.x >> 5; w += 4) {
          const float4 p = *reinterpret_cast<const float4*>(&s_part[parity][w]);
          ss += (p.x + p.y) + (p.z + p.w);
        }
      }
      const float mean = ss * a.inv_width + a.eps, f = rsqrtf(mean);
      if (k < run && leaves_fp32(mean)) left |= bit(0) | bit(1);
#pragma unroll
      for (int i = 0; i < UPT; ++i) factor[i] = f;
    }
    if (k < run) {
      const bool turn = s_pos[k].w != 0;
      // halves: pairs j .. j + V; adjacent: V / 2 pairs of each vector
      uint64_t c[V / 2], s[V / 2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = k * (D / 2) + (HALVES ? j + q * (V / 2) : j / 2 + q * (D / 4));
        if (V == 8) {
          const ulonglong2 cq = *reinterpret_cast<const ulonglong2*>(s_cos + at), sq = *reinterpret_cast<const ulonglong2*>(s_sin + at);
          c[2 * q] = cq.x; c[(2 * q + 1) % (V / 2)] = cq.y;
          s[2 * q] = sq.x; s[(2 * q + 1) % (V / 2)] = sq.y;
        } else {
          c[q] = *reinterpret_cast<const uint64_t*>(s_cos + at);
          s[q] = *reinterpret_cast<const uint64_t*>(s_sin + at);
        }
      }
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (!has(i) || (NORMED && left & bit(i))) continue;
        uint64_t va[V / 2], vb[V / 2];
        U::unpack(raw[i], va, vb);
        if (NORMED) {
          uint64_t wa[V / 2], wb[V / 2];
          U::unpack(wraw[i], wa, wb);
          const uint64_t f2 = f2_pack(factor[i], factor[i]);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            va[e] = f2_mul(va[e], f2_mul(wa[e], f2));
            vb[e] = f2_mul(vb[e], f2_mul(wb[e], f2));
          }
        }
        if (turn) U::rotate(va, vb, c, s);   // a token that does not turn is copied, whatever it holds
        uint4 o2[2];
        U::pack(va, vb, o2);
        T* e = o + i * out_step;
        *reinterpret_cast<uint4*>(e) = o2[0];
        *reinterpret_cast<uint4*>(e + D / 2) = o2[1];
      }
    }
    fetch(k + kStages * groups, at);   // into the stage that this turn has read
    at = at == ring + (kStages - 1) * stage ? ring : at + stage;
  }
  if (NORMED && __any_sync(0xffffffffu, left != 0)) rope_left<T, D, UPT, HALVES>(a, left, run, s_cos, s_pos, s_wide);
}

template <typename T, int D, int UPT>
cudaError_t launch_units(const RopeArgs& a, dim3 grid, int threads, cudaStream_t s) {
  auto kernel = a.halves ? rope_kernel<T, D, UPT, true, false> : rope_kernel<T, D, UPT, false, false>;
  // a norm comes with one or two units, and with four of the widest fp32 tokens
  if constexpr (UPT <= 2 || (UPT == 4 && sizeof(T) == 4))
    if (a.norm) kernel = a.halves ? rope_kernel<T, D, UPT, true, true> : rope_kernel<T, D, UPT, false, true>;
  const size_t smem = (size_t)kStages * UPT * 2 * threads * 16 + (size_t)a.run * D * 4;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_typed(RopeArgs& a, int B, cudaStream_t s) {
  constexpr int kPerHead = D / 2 * (int)sizeof(T) / 16;
  // without the norm over all heads a token's heads may go to several blocks
  a.heads_per_block = a.norm == kFullNorm ? a.H : (a.H < 1024 / kPerHead ? a.H : 1024 / kPerHead);
  const int units = a.heads_per_block * kPerHead;
  int threads, upt;
  // Few units: a warp, or less, a token, so that a sum stays in it; the norm's weights leave room for two units a thread.
  // More: a block a token, one unit a thread while that fills few warps, since registers are what bounds the warps of an
  // SM (bf16, 12 heads of 128, head norm: 37 us against 45 with three units in a warp; 16 heads: 79 against 158), two or
  // four where the barrier of the norm over all heads would join many warps (40 heads, runs of 8: 269 us against 296 with one).
  if (units <= (a.norm == kNoNorm ? 128 : 64)) {
    a.group = kPerHead;
    while (a.group < units && a.group < 32) a.group *= 2;
    upt = (units + 31) / 32;
    threads = 128;
  } else {
    upt = units <= (a.norm == kFullNorm ? 256 : 512) ? 1 : units <= 1024 ? 2 : 4;
    threads = a.group = ((units + upt - 1) / upt + 31) / 32 * 32;
  }
  const int groups = threads / a.group;
  // run: long enough to spread the angles over the threads and to keep loads ahead, short enough for the blocks to fill the
  // GPU several times over.  Blocks of many heads are few on an SM, so half as many fill it, and where the norm joins all
  // their warps longer runs pay (40 heads: 255 us with 16 tokens, 267 with 8, 268 with 32; without the norm 239 with 8, 242
  // with 16).
  const long long tokens = (long long)B * a.N, blocks = 148 * (upt >= 2 && threads > 128 ? 8 : 16);
  const int most = upt >= 2 && a.norm == kFullNorm ? kMaxTurns : 8;
  int per_group = 1;
  while (per_group < most && groups * per_group * 2 <= kMaxRun && tokens / (groups * per_group * 2) >= blocks) per_group *= 2;
  a.run = groups * per_group;
  const dim3 grid((unsigned)((a.N + a.run - 1) / a.run), (unsigned)B, (unsigned)((a.H + a.heads_per_block - 1) / a.heads_per_block));
  return upt == 1   ? launch_units<T, D, 1>(a, grid, threads, s)
         : upt == 2 ? launch_units<T, D, 2>(a, grid, threads, s)
         : upt == 3 ? launch_units<T, D, 3>(a, grid, threads, s)
                    : launch_units<T, D, 4>(a, grid, threads, s);
}

}  // namespace

cudaError_t launch_rope(bool bf16, const da_rope_plan& plan, int B, int H, int N, int d, const void* x,
                        const da_head_strides& xs, const int32_t* positions, long long pos_batch, const void* weight,
                        int weight_width, float eps, void* out, const da_head_strides& os, cudaStream_t s) {
  RopeArgs a{};
  a.x = x;
  a.out = out;
  a.weight = weight;
  a.positions = positions;
  a.pos_batch = pos_batch;
  a.H = H;
  a.N = N;
  a.xb = xs.batch; a.xh = xs.head; a.xn = xs.token;
  a.ob = os.batch; a.oh = os.head; a.on = os.token;
  for (int u = 0; u < 3; ++u) a.grid[u] = plan.grid[u];
  a.norm = !weight ? kNoNorm : weight_width == d ? kHeadNorm : kFullNorm;
  a.eps = eps;
  a.inv_width = 1.f / ((float)H * (float)d);
  a.halves = plan.pairing == DA_ROPE_HALVES;
  // theta^(-2j / D) / (2 pi) turns, in the 64-bit mantissa of long double; theta >= 1 keeps it below one.  Powers by
  // products of one ratio an axis: 63 roundings of 2^-64, and a microsecond less of the call than a power a pair.
  const long double log_theta = logl((long double)plan.theta);
  int p = 0;
  for (int u = 0; u < 3; ++u) {
    const int D = plan.axis_dims[u];
    if (D == 0) continue;
    const long double ratio = expl(log_theta * (-2.0L / D));
    long double f = 0.159154943091895335768883763372514362L;
    for (int j = 0; j < D / 2; ++j, ++p, f *= ratio) {
      a.freq[p] = (uint64_t)(f * 18446744073709551616.0L);
      a.axis[p] = (unsigned char)u;
    }
  }
  if (bf16) return d == 128 ? launch_typed<__nv_bfloat16, 128>(a, B, s) : launch_typed<__nv_bfloat16, 64>(a, B, s);
  return d == 128 ? launch_typed<float, 128>(a, B, s) : launch_typed<float, 64>(a, B, s);
}

}  // namespace da
