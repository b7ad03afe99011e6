// Rotary positions over time, height and width, with the query/key norm in front of them.
//
// A head's d elements form d/2 pairs (a, b); pair p belongs to axis u (the first axis_dims[0] / 2
// pairs to time, and so on) and turns by angle = position_u * theta^(-2j / axis_dims[u]), j its
// index within the axis:  (a, b) -> (a cos - b sin, a sin + b cos).
// Positions come from the (time, height, width) grid of the token's index, or from the caller.
//
// Angles are formed in fp64 in units of half turns, reduced to [-1, 1] there, and only then
// rounded for sincospif: position times frequency loses nothing however far the position.
// A token's d/2 angles are formed once and serve all its heads.
#include <math.h>

#include "da_common.cuh"
#include "da_internal.h"

namespace da {

namespace {

constexpr int kMaxPairs = 64;   // d <= 128

struct RopeArgs {
  const void* x;
  void* out;
  const void* weight;          // or null: no norm
  const int* positions;        // [batch][N][3], or null: the grid
  long long pos_batch;
  int H, N;
  long long rows;              // B * N
  long long xb, xh, xn, ob, oh, on;
  int grid[3];
  int full;                    // the norm runs over all heads
  float eps;
  double freq[kMaxPairs];      // frequency / pi: half turns per position
  unsigned char axis[kMaxPairs];
};

template <typename T, int D>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeArgs a, int halves) {
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  __shared__ float s_part[4];
  __shared__ int s_turn;
  const long long row = blockIdx.x;
  const int b = (int)(row / a.N), n = (int)(row % a.N);
  const int tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.x) + b * a.xb + n * a.xn;
  T* out = static_cast<T*>(a.out) + b * a.ob + n * a.on;
  if (tid < D / 2) {
    const int u = a.axis[tid];
    int pos;
    bool turn = true;
    if (a.positions) {
      pos = a.positions[b * a.pos_batch + (long long)n * 3 + u];
    } else {
      const int w = n % a.grid[2], h = n / a.grid[2] % a.grid[1], t = n / a.grid[2] / a.grid[1];
      pos = u == 0 ? t : u == 1 ? h : w;
      turn = t < a.grid[0];
    }
    double half_turns = (double)pos * a.freq[tid];
    half_turns -= 2.0 * rint(half_turns * 0.5);
    sincospif((float)half_turns, &s_sin[tid], &s_cos[tid]);
    if (tid == 0) s_turn = turn;
  }
  const int total = a.H * D;
  float full = 1.f;
  if (a.weight && a.full) {
    float ss = 0.f;
    for (int i = tid; i < total; i += blockDim.x) {
      const float v = to_f32(x[(i / D) * a.xh + i % D]);
      ss = fmaf(v, v, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) s_part[tid >> 5] = ss;
    __syncthreads();
    full = rsqrtf(((s_part[0] + s_part[1]) + (s_part[2] + s_part[3])) / (float)total + a.eps);
  }
  __syncthreads();
  const T* w = static_cast<const T*>(a.weight);
  // one warp per head: lane l holds pairs l, l + 32
  for (int h = tid >> 5; h < a.H; h += 4) {
    float va[D / 64], vb[D / 64];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int p = (tid & 31) + 32 * i;
      const int ia = halves ? p : 2 * p, ib = halves ? p + D / 2 : 2 * p + 1;
      va[i] = to_f32(x[h * a.xh + ia]);
      vb[i] = to_f32(x[h * a.xh + ib]);
      ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
    }
    float f = full;
    if (w && !a.full) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      f = rsqrtf(ss / (float)D + a.eps);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int p = (tid & 31) + 32 * i;
      const int ia = halves ? p : 2 * p, ib = halves ? p + D / 2 : 2 * p + 1;
      if (w) {
        va[i] *= f * to_f32(w[(a.full ? h * D : 0) + ia]);
        vb[i] *= f * to_f32(w[(a.full ? h * D : 0) + ib]);
      }
      const float c = s_cos[p], s = s_sin[p];
      // a token that does not turn is copied, whatever it holds
      store_out(out + h * a.oh + ia, s_turn ? va[i] * c - vb[i] * s : va[i]);
      store_out(out + h * a.oh + ib, s_turn ? va[i] * s + vb[i] * c : vb[i]);
    }
  }
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
  a.rows = (long long)B * N;
  a.xb = xs.batch; a.xh = xs.head; a.xn = xs.token;
  a.ob = os.batch; a.oh = os.head; a.on = os.token;
  for (int u = 0; u < 3; ++u) a.grid[u] = plan.grid[u];
  a.full = weight && weight_width == H * d && H > 1;
  a.eps = eps;
  int p = 0;
  for (int u = 0; u < 3; ++u)
    for (int j = 0; j < plan.axis_dims[u] / 2; ++j, ++p) {
      a.freq[p] = pow(plan.theta, -2.0 * j / plan.axis_dims[u]) / M_PI;
      a.axis[p] = (unsigned char)u;
    }
  const int halves = plan.pairing == DA_ROPE_HALVES;
  const unsigned grid = (unsigned)a.rows;
  if (bf16) {
    if (d == 128) rope_kernel<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(a, halves);
    else rope_kernel<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(a, halves);
  } else {
    if (d == 128) rope_kernel<float, 128><<<grid, 128, 0, s>>>(a, halves);
    else rope_kernel<float, 64><<<grid, 128, 0, s>>>(a, halves);
  }
  return cudaGetLastError();
}

}  // namespace da
