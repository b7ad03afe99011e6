// Product of 8-bit integer matrices with scales per token and channel, on the tensor cores.
//
//   out[m, n] = (sum_k x[m, k] w[n, k]) sx[m] sw[n] + bias[n]
// tcgen05.mma kind::i8 sums in 32-bit integers in tensor memory, so the sum is exact; the epilogue
// converts it, applies both scales and the bias in fp32 and rounds once to the output's type.
//
// A persistent grid walks output tiles.  Roles of a CTA (384 threads):
//   warp 0     lane 0 loads 128-byte slices of the x and w rows by TMA into a ring of stages (128-byte
//              swizzle; rows and depth beyond the matrices read as zero);
//   warp 1     lane 0 issues the products of a stage (four k = 32 steps) into one of two accumulators;
//   warp 2     allocates tensor memory;
//   warps 4-11 epilogue: accumulator -> scaled rows -> shared memory -> the output (the matrix, or the attention's
//              heads), while the next tile's products fill the other accumulator.  Two groups of four warps take alternate
//              parts of 32 columns (one was the bound at shallow depths, a third gained nothing).  Boxes of 32 rows x 64 bytes
//              leave by TMA where the output's strides and widths are multiples of 16 bytes (16000 x 2048 x 512, fp32 out,
//              43.5 -> 35 us, and 32760 x 1536 x 1536, bf16, 62 -> 59 us against 16-byte stores by the warps); rows on 16
//              bytes that are no such boxes by 16-byte stores; others element by element, neighbouring lanes neighbouring
//              columns (16000 x 2049 x 512, fp32, 54 us; 90 with every row's address fetched from the lane that holds it).
//
// Two forms.  Pair (kPair): two CTAs of a cluster form a 256 x n tile (n 160 to 256) with cta_group::2; each loads its
// own 128 rows of x and half of the w rows, so every loaded byte serves 256 rows or n columns.  Single: one CTA forms 128 x n,
// n any multiple of 16 up to 256, so that the tiles of a small product can be cut to fill the GPU (choose_tile).
//
// A product of few rows is bound by the loads of w, and the waits of the ring would bound it first: then a stage
// holds up to four slices of depth, and only as many rows of x as there are.  The tensor core still reads 128 rows: the ones
// beyond are whatever lies behind in the block's shared memory, and their products are never stored.
//
// Measured, bf16 out: 75600 x 5120 x 5120 1.22 ms cold and 1.31-1.39 ms in a long run under the power cap (3.24e15 and
// 2.85-3.0e15 op/s; twice the bf16 library rate is 3.38e15 and 2.87e15), the tensor pipe 94 % busy; 2048 x 5120 x 5120
// 37 us, 512: 14 us, 128: 11 us.  32760 x 1536 x 1536 59-61 us (2.6e15): at shallow depths the epilogue is what bounds.
#include "da_common.cuh"
#include "da_internal.h"
#include "linear_i8.cuh"
#include "tma_host.h"

namespace da {

namespace {

constexpr int kBlockK = 128;                 // bytes (= elements) of depth per stage
constexpr int kTileM = 128;                  // rows of x per CTA
constexpr int kEpilogueGroups = 2;            // of four warps
constexpr int kEpilogueWarps = 4 * kEpilogueGroups;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kABytes = kTileM * kBlockK;    // 16 KB

constexpr int kMaxN = 256;                   // columns of a tile
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 6 * 32768;        // the pair's stages at n = 256; a single CTA's 128 + 256 rows fit four times
constexpr int kStagingBytes = kEpilogueWarps * 2048;   // 32 rows of 64 bytes a warp; behind the ring: a short tile of x is read up to 16 KB beyond it
constexpr size_t kSmem = 1024 + kRingBytes + kStagingBytes + 2 * 2 * kMaxN * 4 /*scales, bias*/;
static_assert(kStagingBytes >= kABytes, "a short tile of x is read as a whole one");
static_assert(kSmem + 1024 <= 232448, "shared memory of one CTA per SM");

struct Params {
  LinearArgs a;
  int tiles_m, tiles_n, k_blocks;
  int n;              // columns of a tile
  int a_rows, b_rows; // rows of x and w that a CTA loads for a tile
  int stages;         // of the ring
  int vec;            // rows of the output can be stored 16 bytes at a time
  int even;           // the 32 rows of a warp are out_token apart
  int boxes;          // and as boxes of 32 rows x 64 bytes, by TMA
  int* status;
};

struct __align__(8) Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// Place in the ring: stage and the parity of its turn.
struct Turn {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on a barrier of the other CTA (or this one).  What it orders is reads of tensor memory, which have completed and
// been fenced (tcgen05.fence::before_thread_sync): a release at cluster scope would wait for the epilogue's global stores.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// mbar_wait by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if (kPair)
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

// A box of shared memory into the output; out-of-range rows and columns are not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until this thread's stores have read their shared memory.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Arrive on `bar` (in both CTAs of a pair) when the products issued so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (kPair)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
  else
    umma_commit(bar);
}
template <bool kPair>
__device__ __forceinline__ void alloc_columns(uint32_t* dst, uint32_t n) {
  if (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(n) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, n);
    tmem_relinquish();
  }
}
template <bool kPair>
__device__ __forceinline__ void free_columns(uint32_t t, uint32_t n) {
  if (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(n) : "memory");
  else
    tmem_dealloc(t, n);
}

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpilogueWarps) : "memory"); }

template <typename T, bool kPair, int kSub>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* staging = ring + kRingBytes;
  float* s_cols = reinterpret_cast<float*>(staging + kStagingBytes);   // [2 tiles][scale, bias][kMaxN]

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // the same in all lanes, for the compiler too
  const uint32_t rank = kPair ? cluster_rank() : 0;
  const int first = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int step = kPair ? gridDim.x >> 1 : gridDim.x;
  const int tiles = p.tiles_m * p.tiles_n;
  constexpr int kRowsPerTile = kPair ? 2 * kTileM : kTileM;
  const int a_bytes = kPair ? kABytes : p.a_rows * kBlockK, slice_bytes = a_bytes + p.b_rows * kBlockK;
  const int stages = p.stages, stage_bytes = kSub * slice_bytes;
  volatile int* abort = &bars.abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], kPair ? 2 * kEpilogueWarps : kEpilogueWarps);   // one arrival per epilogue warp
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) alloc_columns<kPair>(&bars.tmem_base, 2 * kMaxN);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  // The issuing warps run their loops whole, and one lane issues: addresses and descriptors then stay in uniform registers.
  // With one lane running the loop a stage took 640 clocks to issue, whatever its products.
  if (warp == 0) {
    const bool leader = elect_one();
    if (leader) {
      tma_prefetch(&tm_x);
      tma_prefetch(&tm_w);
    }
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(&bars.full[0]);
    // a pair's copies all land on the leading CTA's barrier, which expects the bytes of both
    const uint32_t land0 = kPair ? map_to_rank(full0, 0) : full0;
    Turn turn;
    int it = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int row = tm * kRowsPerTile + (int)rank * kTileM;
      const int col = tn * p.n + (int)rank * p.b_rows;
      for (int kb = 0; kb < p.k_blocks; kb += kSub, ++it, turn.next(stages)) {
        ok = warp_wait(&bars.empty[turn.s], turn.ph ^ 1, abort, p.status);
        if (!ok) break;
        const uint32_t a = ring0 + turn.s * stage_bytes, bar = land0 + turn.s * 8;
        const int slices = kSub == 1 ? 1 : min(kSub, p.k_blocks - kb);
        if (leader) {
          if (rank == 0) expect_bytes(full0 + turn.s * 8, (uint32_t)(slices * slice_bytes) * (kPair ? 2u : 1u));
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            if (i < slices) {
              tma_load_2d<kPair>(a + i * slice_bytes, &tm_x, bar, (kb + i) * kBlockK, row);
              tma_load_2d<kPair>(a + i * slice_bytes + a_bytes, &tm_w, bar, (kb + i) * kBlockK, col);
            }
          }
        }
        __syncwarp();
      }
    }
    // given up: wait (within a limit) for the copies in flight before the block's memory goes
    if (!ok && rank == 0)
      for (int i = max(0, it - stages); i < it; ++i) mbar_wait_drain(&bars.full[i % stages], (i / stages) & 1);
  } else if (warp == 1 && rank == 0) {
    const bool leader = elect_one();
    const uint32_t idesc = idesc_i8(kRowsPerTile, p.n);
    const uint64_t desc0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    Turn turn;
    int n = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step, ++n) {
      const int b = n & 1;
      ok = warp_wait(&bars.acc_empty[b], ((n >> 1) & 1) ^ 1, abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + b * kMaxN;
      for (int kb = 0; kb < p.k_blocks; kb += kSub, turn.next(stages)) {
        ok = warp_wait(&bars.full[turn.s], turn.ph, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        // descriptors count addresses in 16 bytes
        const uint64_t ad = desc0 + (uint32_t)(turn.s * stage_bytes >> 4);
        const int slices = kSub == 1 ? 1 : min(kSub, p.k_blocks - kb);
        if (leader) {
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            if (i < slices) {
#pragma unroll
              for (int ks = 0; ks < kBlockK / 32; ++ks)
                mma_i8<kPair>(acc, ad + (uint32_t)(i * slice_bytes >> 4) + 2 * ks,
                              ad + (uint32_t)((i * slice_bytes + a_bytes) >> 4) + 2 * ks, idesc, i || ks ? 1u : kb != 0);
            }
          }
          mma_commit<kPair>(&bars.empty[turn.s]);
        }
        __syncwarp();
      }
      if (ok && leader) mma_commit<kPair>(&bars.acc_full[b]);
      __syncwarp();
    }
    if (*abort && leader) {   // products in flight end before the tensor memory is freed
      mma_commit<kPair>(&bars.drain);
      mbar_wait_drain(&bars.drain, 0);
    }
  } else if (warp >= 4) {
    const int ew = warp & 3, group = (warp - 4) >> 2;   // rows ew * 32 .. + 32; parts group, group + kEpilogueGroups, ...
    uint8_t* stage = staging + (warp - 4) * 2048;
    const LinearArgs& A = p.a;
    constexpr int kV = 16 / (int)sizeof(T);          // elements of a 16-byte store
    constexpr int kSeg = 64 / (int)sizeof(T);        // columns of a staged row
    const uint32_t empty0 = kPair ? map_to_rank(smem_u32(&bars.acc_empty[0]), 0) : 0;
    int n = 0;
    bool ok = true;   // after a wait that gave up the loop still runs, so that the warps' barriers match
    // scales and bias of a tile: thread i of the epilogue holds column i's, and its row's scale; loaded a tile ahead
    static_assert(32 * kEpilogueWarps >= kMaxN, "a thread a column");
    const int mine = threadIdx.x - 128;
    float col_scale = 0.f, col_bias = 0.f, row_scale = 0.f;
    auto load_scales = [&](int t) {
      if (t >= tiles) return;
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int c = tn * p.n + mine;
      const long long m = (long long)tm * kRowsPerTile + (int)rank * kTileM + ew * 32 + lane;
      const bool in = mine < p.n && c < A.N;
      col_scale = in ? A.w_scale[c] : 0.f;
      col_bias = in && A.bias ? A.bias[c] : 0.f;
      row_scale = m < A.M ? A.x_scale[m] : 0.f;
    };
    load_scales(first);
    for (int t = first; t < tiles; t += step, ++n) {
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int b = n & 1;
      const int n0 = tn * p.n, n1 = min(n0 + p.n, A.N);   // the tile's columns
      float* cs = s_cols + b * 2 * kMaxN;
      if (mine < kMaxN) {
        cs[mine] = col_scale;
        cs[kMaxN + mine] = col_bias;
      }
      const float sx = row_scale;
      load_scales(t + step);
      const long long m = (long long)tm * kRowsPerTile + (int)rank * kTileM + ew * 32 + lane;
      const int mb = (int)m / A.tokens;   // M stays below 2^31
      const long long off = mb * A.out_batch + ((int)m - mb * A.tokens) * A.out_token;
      const int valid = (int)min(32LL, max(0LL, A.M - (m - lane)));   // rows of this warp inside the matrix
      long long quad_off[4];   // of the rows whose segments this lane stores
#pragma unroll
      for (int i = 0; i < 4; ++i) quad_off[i] = __shfl_sync(0xffffffffu, off, i * 8 + (lane >> 2));
      epilogue_barrier();
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars.acc_full[b], (n >> 1) & 1, abort, p.status));
      if (!ok) continue;
      tc_fence_after();
      // a last part may reach beyond the tile: read, not stored; each part is read while the one before is stored, and
      // waited for in the turn that asked for it
      const uint32_t acc = tmem + ((uint32_t)(ew * 32) << 16) + b * kMaxN;
      uint32_t r[32];
      if (n0 + 32 * group < n1) {
        tmem_ld32(acc + 32 * group, r);
        tmem_wait_ld_into(r);
      }
#pragma unroll 1
      for (int c0 = 32 * group; n0 + c0 < n1; c0 += 32 * kEpilogueGroups) {
        const ulonglong2* sw2 = reinterpret_cast<const ulonglong2*>(cs + c0);
        const ulonglong2* bi2 = reinterpret_cast<const ulonglong2*>(cs + kMaxN + c0);
        const uint64_t sx2 = f2_pack(sx, sx);
        float v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 w = sw2[i], bi = bi2[i];
          const uint64_t lo = f2_pack((float)(int)r[4 * i], (float)(int)r[4 * i + 1]);
          const uint64_t hi = f2_pack((float)(int)r[4 * i + 2], (float)(int)r[4 * i + 3]);
          f2_unpack(f2_fma(f2_mul(lo, sx2), w.x, bi.x), v[4 * i], v[4 * i + 1]);
          f2_unpack(f2_fma(f2_mul(hi, sx2), w.y, bi.y), v[4 * i + 2], v[4 * i + 3]);
        }
        const bool more = n0 + c0 + 32 * kEpilogueGroups < n1;
        if (more) tmem_ld32(acc + c0 + 32 * kEpilogueGroups, r);
#pragma unroll
        for (int g = 0; g < 32 / kSeg; ++g) {   // a segment of 64 bytes a row
          if (p.boxes) {   // the store of the segment before has read the staging
            if (lane == 0) tma_store_read();
            __syncwarp();
          }
          // row `lane`, 16-byte chunk j at chunk j ^ (row / 2 & 3), the 64-byte swizzle: neither side of the transposition conflicts
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* e = v + g * kSeg + j * kV;
            uint4 o;
            if constexpr (sizeof(T) == 2)
              o = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
            else
              o = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = o;
          }
          const int s0 = n0 + c0 + g * kSeg;   // the segment's first column
          if (p.boxes) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && valid > 0 && s0 < n1) {
              const int h = s0 / A.d;
              tma_store_4d(&tm_out, smem_u32(stage), s0 - h * A.d, (int)m - mb * A.tokens, h, mb);
            }
            continue;
          }
          __syncwarp();
          if (p.vec) {
            // 4 lanes per row segment, 8 rows at a time
            const int c = s0 + (lane & 3) * kV, h = c / A.d;
            const long long head = h * A.out_head + (c - h * A.d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = i * 8 + (lane >> 2);
              const uint4 o = *reinterpret_cast<const uint4*>(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
              T* to = static_cast<T*>(A.out) + quad_off[i] + head;
              if (row < valid && c < n1) {
                if (c + kV <= n1) {
                  *reinterpret_cast<uint4*>(to) = o;
                } else {   // the last columns of the matrix: one head
                  const T* e = reinterpret_cast<const T*>(&o);
#pragma unroll
                  for (int k = 0; k < kV; ++k)
                    if (c + k < n1) to[k] = e[k];
                }
              }
            }
          } else {
            // rows of any alignment: kSeg lanes a row, neighbouring lanes neighbouring columns
            constexpr int kRows = 32 / kSeg;
            const int col = lane % kSeg, c = s0 + col, h = c / A.d, first = lane / kSeg;
            const int byte = col * (int)sizeof(T), below = c < n1 ? valid : 0;
            T* to = static_cast<T*>(A.out) + (h * A.out_head + (c - h * A.d));
            if (p.even) to += __shfl_sync(0xffffffffu, off, first);
#pragma unroll
            for (int i = 0; i < 32; i += kRows) {
              const int row = i + first;
              T* at = p.even ? to : to + __shfl_sync(0xffffffffu, off, row);
              // kRows divides 2, so that row / 2 is i / 2
              if (row < below) *at = *reinterpret_cast<const T*>(stage + row * 64 + (((byte >> 4) ^ ((i >> 1) & 3)) << 4) + (byte & 15));
              if (p.even) to += kRows * A.out_token;
            }
          }
          __syncwarp();
        }
        if (more) tmem_wait_ld_into(r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) arrive_at(empty0 + b * 8);
        else mbar_arrive(&bars.acc_empty[b]);
      }
    }
    if (p.boxes && lane == 0) tma_store_read();   // before the block's memory goes
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // neither CTA's barriers or tensor memory go while the other may still reach them
  if (warp == 2) {
    tc_fence_after();
    free_columns<kPair>(tmem, 2 * kMaxN);
  }
}

bool make_tmap_i8(CUtensorMap* m, const void* ptr, uint64_t K, uint64_t rows, uint64_t stride, uint32_t box_rows) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  cuuint64_t dims[2] = {K, rows};
  cuuint64_t strides[1] = {stride};
  cuuint32_t box[2] = {kBlockK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output as [B][H][tokens][d], stored in boxes of 32 tokens x 64 bytes.
template <typename T>
bool make_tmap_out(CUtensorMap* m, const LinearArgs& a) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const cuuint64_t B = a.M / a.tokens, H = a.N / a.d, esz = sizeof(T), row = ((cuuint64_t)a.d * esz + 15) / 16 * 16;
  // a dimension of one has a stride that nothing uses
  cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.tokens, H, B};
  cuuint64_t strides[3] = {a.tokens > 1 ? a.out_token * esz : row, H > 1 ? a.out_head * esz : row, B > 1 ? a.out_batch * esz : row};
  cuuint32_t box[4] = {64 / (cuuint32_t)esz, 32, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.out, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool kPair, int kSub>
cudaError_t launch_sub(const LinearArgs& a, Params& p, int sms, cudaStream_t s) {
  const int stage = kSub * (p.a_rows + p.b_rows) * kBlockK;
  p.stages = kRingBytes / stage < kMaxStages ? kRingBytes / stage : kMaxStages;
  // rows are at least their depth apart (the dispatch sees to it), one row may have any stride
  const uint64_t xs = a.M > 1 ? a.x_stride : (a.K + 15) / 16 * 16, ws = a.N > 1 ? a.w_stride : (a.K + 15) / 16 * 16;
  CUtensorMap tx, tw, to{};
  if (!make_tmap_i8(&tx, a.x, a.K, a.M, xs, p.a_rows)) return cudaErrorInvalidValue;
  if (!make_tmap_i8(&tw, a.w, a.K, a.N, ws, p.b_rows)) return cudaErrorInvalidValue;
  // a box has the tokens of one batch (even), its columns are one tile's and one head's, and a row's last 16 bytes are written whole
  constexpr int kSeg = 64 / (int)sizeof(T);
  p.even = a.tokens == a.M || a.tokens % 32 == 0;
  p.boxes = p.vec && a.d % (kSeg / 4) == 0 && p.even && (p.n % kSeg == 0 || p.tiles_n == 1) &&
            (a.d == a.N || a.d % kSeg == 0) && make_tmap_out<T>(&to, a);
  auto kernel = linear_i8_tc_kernel<T, kPair, kSub>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)p.tiles_m * p.tiles_n;
  if (tiles >= (1LL << 30)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  const int slots = kPair ? sms / 2 : sms;
  cfg.gridDim = dim3((unsigned)(tiles < slots ? tiles : slots) * (kPair ? 2 : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair ? 2 : 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tx, tw, to, p);
}

template <typename T, bool kPair>
cudaError_t launch_tile(const LinearArgs& a, int n, int sms, int* status, cudaStream_t s) {
  Params p;
  p.a = a;
  p.status = status;
  p.n = n;
  p.tiles_m = (int)((a.M + (kPair ? 255 : 127)) / (kPair ? 256 : 128));
  p.tiles_n = (a.N + n - 1) / n;
  p.k_blocks = (a.K + kBlockK - 1) / kBlockK;
  p.a_rows = a.M >= kTileM || kPair ? kTileM : ((int)a.M + 7) / 8 * 8;
  p.b_rows = kPair ? n / 2 : n;
  const int esz = (int)sizeof(T), v = 16 / esz;
  p.vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_batch % v == 0 && a.out_token % v == 0 &&
          (a.d == a.N || (a.d % v == 0 && a.out_head % v == 0));
  if constexpr (kPair) {
    return launch_sub<T, kPair, 1>(a, p, sms, s);
  } else {
    const int sub = kRingBytes / 4 / ((p.a_rows + p.b_rows) * kBlockK);   // slices of a stage, with four stages at least
    return sub >= 4   ? launch_sub<T, kPair, 4>(a, p, sms, s)
           : sub >= 2 ? launch_sub<T, kPair, 2>(a, p, sms, s)
                      : launch_sub<T, kPair, 1>(a, p, sms, s);
  }
}

struct Tile {
  bool pair;
  int n;
};

// The tile, by an estimate of the clocks of the longest CTA.  A wave of tiles takes, for each 32 of depth, what its
// products take (n / 2 clocks for 128 x n on one SM and for 256 x n on two) or, for a single CTA, what reading their operands
// from shared memory takes (4 KB + 32 n bytes at 128 a clock); and 2000 clocks for filling the ring and the last epilogue.
// The single tile pays a quarter more for its double traffic from L2.  Measured against every other n, the estimate's choice
// was the fastest or within 3 % of it for 14 of 15 sizes from 16 x 5120 x 5120 to 20000 x 1000 x 512 (8 % there).
Tile choose_tile(const LinearArgs& a, int sms) {
  const long long k = (a.K + 31) / 32;
  Tile best{true, kMaxN};
  long long least = 0;
  for (int n = kMaxN; n >= 160; n -= 32) {
    const long long tiles = (a.M + 255) / 256 * ((a.N + n - 1) / n);
    const long long clocks = (tiles + sms / 2 - 1) / (sms / 2) * (n / 2 * k + 2000);
    if (n == kMaxN || clocks < least) {
      least = clocks;
      best.n = n;
    }
  }
  for (int n = 16; n <= kMaxN; n += 16) {
    const long long tiles = (a.M + kTileM - 1) / kTileM * ((a.N + n - 1) / n);
    const int mma = n / 2, smem = 32 + n / 4;
    const long long clocks = (tiles + sms - 1) / sms * ((mma > smem ? mma : smem) * k * 5 / 4 + 2000);
    if (clocks < least || (clocks == least && !best.pair)) {
      least = clocks;
      best = Tile{false, n};
    }
  }
  return best;
}

template <typename T>
cudaError_t launch_typed(const LinearArgs& a, int* status, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const Tile t = choose_tile(a, sms);
  return t.pair ? launch_tile<T, true>(a, t.n, sms, status, s) : launch_tile<T, false>(a, t.n, sms, status, s);
}

}  // namespace

bool linear_i8_tc_supported(const LinearArgs& a) {
  auto rows_ok = [&](const void* p, long long rows, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || (stride % 16 == 0 && stride >= a.K && stride < (1LL << 40)));
  };
  return rows_ok(a.x, a.M, a.x_stride) && rows_ok(a.w, a.N, a.w_stride);
}

cudaError_t launch_linear_i8_tc(bool bf16, const LinearArgs& a, int* status, cudaStream_t s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, status, s) : launch_typed<float>(a, status, s);
}

}  // namespace da
