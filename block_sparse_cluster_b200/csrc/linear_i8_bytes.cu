// Product of 8-bit integer matrices with scales per token and channel, for rows that do not start on 16 bytes, which
// tile loads cannot read.
//
//   out[m, n] = (sum_k x[m, k] w[n, k]) sx[m] sw[n] + bias[n]
// The tensor cores form it all the same (kind::i8, 32-bit integer sums, exact for K <= 131071, the host's limit): the CTA's
// threads load the rows themselves, 8 bytes a thread.  A thread takes the two aligned 8 bytes that its own lie in, shifts them
// together and writes them where the 128-byte swizzle puts them.  A CTA forms 128 x n outputs (n = 128, or 64 or 32 where that
// fills the GPU) from slices of 128 deep in two buffers: a slice's words are loaded into registers while the one before is
// multiplied.  Two CTAs an SM.  The loads bound it, by their latency where there are few tiles and by their number where there
// are many.  Measured, bf16 out: 777 x 1537 x 1001 18 us, 2048 x 5120 x 5121 173-183 us, 8192 x 5120 x 5121 607-620 us (7e14 op/s, a
// quarter of the rate of rows on 16 bytes; one row of x, 1 x 5120 x 5121, still takes 46 us; four products an instruction on the CUDA cores reached 8e13).  Taking a thread's second
// word from its neighbour by shuffles halves the loads and was slower (950 us against 840 then); full
// tiles without a test a chunk are faster (722 -> 607).  The quantisers write rows that need none of it.
#include "da_common.cuh"
#include "da_internal.h"
#include "linear_i8.cuh"

namespace da {

namespace {

constexpr int kTileM = 128;
constexpr int kBlockK = 128;   // bytes of depth per slice
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 2 * kWarps;   // rows that the warps load together, one a half-warp
constexpr int kXChunks = kTileM / kChunk;
constexpr int kPitch = 33;           // of a staged row of 32 outputs
static_assert(2 * (kTileM + 32) * kBlockK >= kWarps * 32 * kPitch * 4, "the epilogue's staging fits the smallest buffers");

// The 8 aligned bytes at p; those outside [lo, hi) are not read (0).
__device__ __forceinline__ uint2 bytes_within(uintptr_t p, uintptr_t lo, uintptr_t hi) {
  if (p >= lo && p + 8 <= hi) return *reinterpret_cast<const uint2*>(p);
  uint64_t v = 0;
#pragma unroll 1
  for (int e = 0; e < 8; ++e)
    if (p + e >= lo && p + e < hi) v |= (uint64_t) * reinterpret_cast<const uint8_t*>(p + e) << (8 * e);
  return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
}

// Rows of x or w that a tile reads, as a thread sees them: it takes row `place` of each chunk of 16.  Those rows are
// 16 strides apart, so they all start at the same place within 8 bytes.
struct Rows {
  uintptr_t first, any;   // this thread's first row and a row that is always there, down to a multiple of 8
  uintptr_t lo, hi;       // where the matrix begins and ends
  long long step;
  int count, place, skew;   // rows of the tile; skew: bytes from `first` to the row

  __device__ __forceinline__ Rows(const int8_t* matrix, long long of, long long stride, long long row0, int count_, int place_, int K)
      : lo(reinterpret_cast<uintptr_t>(matrix)), hi(reinterpret_cast<uintptr_t>(matrix + (of - 1) * stride + K)), step(kChunk * stride),
        count(count_), place(place_) {
    const uintptr_t base = lo + (uintptr_t)(row0 * stride), mine = base + (uintptr_t)(place_ * stride);
    skew = (int)(mine & 7);
    first = mine - skew;
    any = base & ~(uintptr_t)7;
  }
};

// A thread's part of a slice: for its row of every chunk, the two aligned 8 bytes that bytes [k, k + 8) lie in.
template <int kChunks>
struct Words {
  uint2 lo[kChunks], hi[kChunks];

  // kInside: the words around the bytes lie in the row.  Otherwise a word is read where it holds bytes of the row, and where
  // it reaches out of the matrix byte by byte.  kFull: the tile has all its rows.
  template <bool kInside, bool kFull>
  __device__ __forceinline__ void load(const Rows& m, int k, int K) {
    uintptr_t row = m.first + k;
#pragma unroll
    for (int i = 0; i < kChunks; ++i, row += m.step) {
      if (!kFull && i * kChunk >= m.count) break;
      const uintptr_t at = kFull || i * kChunk + m.place < m.count ? row : m.any + k;
      if (kInside) {
        lo[i] = *reinterpret_cast<const uint2*>(at);
        hi[i] = *reinterpret_cast<const uint2*>(at + 8);
      } else {
        lo[i] = hi[i] = make_uint2(0, 0);
        if (k < K + m.skew) lo[i] = bytes_within(at, m.lo, m.hi);
        if (k + 8 < K + m.skew) hi[i] = bytes_within(at + 8, m.lo, m.hi);
      }
    }
  }
  __device__ __forceinline__ void load(const Rows& m, bool inside, int k, int K) {
    if (!inside) load<false, false>(m, k, K);
    else if (m.count == kChunks * kChunk) load<true, true>(m, k, K);
    else load<true, false>(m, k, K);
  }
  // To rows of 128 bytes in the 128-byte swizzle; mask keeps the bytes before the end of a row.
  template <bool kFull>
  __device__ __forceinline__ void store(uint8_t* to, const Rows& m, int l, uint2 mask) const {
    const bool far = m.skew & 4;
    const uint32_t shift = (m.skew & 3) * 8;
    uint8_t* at = to + m.place * kBlockK + (((l >> 1) ^ (m.place & 7)) << 4) + (l & 1) * 8;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (!kFull && i * kChunk >= m.count) break;
      const uint32_t a = far ? lo[i].y : lo[i].x, b = far ? hi[i].x : lo[i].y, c = far ? hi[i].y : hi[i].x;
      *reinterpret_cast<uint2*>(at + i * kChunk * kBlockK) =
          make_uint2(__funnelshift_r(a, b, shift) & mask.x, __funnelshift_r(b, c, shift) & mask.y);
    }
  }
  __device__ __forceinline__ void put(uint8_t* to, const Rows& m, int l, uint2 mask) const {
    if (m.count == kChunks * kChunk) store<true>(to, m, l, mask);
    else store<false>(to, m, l, mask);
  }
};

// The first n bytes of a word (none for n <= 0, all for n >= 4).
__device__ __forceinline__ uint32_t first_bytes(int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1; }

template <typename T, int n>   // n columns of a tile
__global__ void __launch_bounds__(kThreads, 2)
linear_i8_bytes_kernel(const LinearArgs a, int tiles_m, int tiles_n, int* status) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done[2], drain;   // the products of a buffer's slice have been formed
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int buffer = (kTileM + n) * kBlockK;
  volatile int* abort = &abort_flag;
  int tm, tn;
  tile_at(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * kTileM, n0 = tn * n;
  const int rows = (int)min((long long)kTileM, a.M - m0), cols = min(n, a.N - n0);

  if (threadIdx.x == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, n);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  const int place = threadIdx.x >> 4, l = threadIdx.x & 15;
  const Rows x(a.x, a.M, a.x_stride, m0, rows, place, a.K), w(a.w, a.N, a.w_stride, n0, cols, place, a.K);
  const int slices = (a.K + kBlockK - 1) / kBlockK;
  Words<kXChunks> xw;
  Words<n / kChunk> ww;
  auto load = [&](int kb) {
    const int k0 = kb * kBlockK, k = k0 + 8 * l;
    // between the first and the last slices the words around a thread's bytes lie in its row
    const bool inside = k0 > 0 && k0 + kBlockK + 8 <= a.K;
    xw.load(x, inside, k, a.K);
    ww.load(w, inside, k, a.K);
  };
  bool ok = true;
  load(0);
  for (int kb = 0; kb < slices; ++kb) {
    const int s = kb & 1;
    uint8_t* to = ring + s * buffer;
    if (kb >= 2) ok = mbar_wait(&done[s], ((kb >> 1) - 1) & 1, abort, status);
    if (ok) {
      const int left = a.K - kb * kBlockK - 8 * l;
      const uint2 mask = make_uint2(first_bytes(left), first_bytes(left - 4));
      xw.put(to, x, l, mask);
      ww.put(to + kTileM * kBlockK, w, l, mask);
    }
    if (kb + 1 < slices) load(kb + 1);
    fence_async_smem();
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (warp == 0) {
      tc_fence_after();
      if (elect_one()) {
        const uint64_t ad = sdesc_sw128(smem_u32(to), 16, 1024), bd = sdesc_sw128(smem_u32(to + kTileM * kBlockK), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < kBlockK / 32; ++ks)
          mma_i8<false>(tmem, ad + 2 * ks, bd + 2 * ks, idesc_i8(kTileM, n), kb || ks ? 1u : 0u);
        umma_commit(&done[s]);
      }
      __syncwarp();
    }
  }
  if (ok) ok = __syncthreads_and(mbar_wait(&done[(slices - 1) & 1], ((slices - 1) >> 1) & 1, abort, status));
  if (!ok && warp == 0) {   // products in flight end before the memory goes
    if (elect_one()) {
      umma_commit(&drain);
      mbar_wait_drain(&drain, 0);
    }
    __syncwarp();
  }
  if (ok) {
    tc_fence_after();
    // a warp's 32 rows, 32 columns at a time: through shared memory, so that a row's columns are stored together
    const int quarter = warp & 3;
    float* stage = reinterpret_cast<float*>(ring) + warp * 32 * kPitch;
    const int r = quarter * 32 + lane;
    const bool mine = r < rows;
    const float sx = mine ? a.x_scale[m0 + r] : 0.f;
    const int mb = (m0 + r) / a.tokens;
    const long long off = mb * a.out_batch + (m0 + r - mb * a.tokens) * a.out_token;
    const int valid = min(32, rows - quarter * 32);
    for (int c0 = 32 * (warp >> 2); c0 < cols; c0 += 64) {
      uint32_t acc[32];
      tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + c0, acc);
      tmem_wait_ld_into(acc);
#pragma unroll
      for (int i = 0; i < 32; ++i) stage[lane * kPitch + i] = (float)(int)acc[i] * sx;
      __syncwarp();
      const int c = n0 + c0 + lane;
      const bool in = c0 + lane < cols;
      const float sw = in ? a.w_scale[c] : 0.f, bias = in && a.bias ? a.bias[c] : 0.f;
      const int h = c / a.d;
      T* out = static_cast<T*>(a.out) + (h * a.out_head + (c - h * a.d));
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const long long ro = __shfl_sync(0xffffffffu, off, i);
        if (in && i < valid) store_out(out + ro, fmaf(stage[i * kPitch + lane], sw, bias));
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, n);
  }
}

template <typename T, int n>
cudaError_t launch_tile(const LinearArgs& a, long long tiles_m, int* status, cudaStream_t s) {
  constexpr size_t smem = 1024 + 2 * (size_t)(kTileM + n) * kBlockK;
  const cudaError_t e = cudaFuncSetAttribute(linear_i8_bytes_kernel<T, n>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long tiles_n = (a.N + n - 1) / n;
  if (tiles_m * tiles_n >= (1LL << 30)) return cudaErrorInvalidValue;
  linear_i8_bytes_kernel<T, n><<<(unsigned)(tiles_m * tiles_n), kThreads, smem, s>>>(a, (int)tiles_m, (int)tiles_n, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const LinearArgs& a, int* status, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long tiles_m = (a.M + kTileM - 1) / kTileM;
  if (tiles_m * ((a.N + 127) / 128) >= sms) return launch_tile<T, 128>(a, tiles_m, status, s);
  if (tiles_m * ((a.N + 63) / 64) >= sms) return launch_tile<T, 64>(a, tiles_m, status, s);
  return launch_tile<T, 32>(a, tiles_m, status, s);
}

}  // namespace

cudaError_t launch_linear_i8_bytes(bool bf16, const LinearArgs& a, int* status, cudaStream_t s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, status, s) : launch_typed<float>(a, status, s);
}

}  // namespace da
