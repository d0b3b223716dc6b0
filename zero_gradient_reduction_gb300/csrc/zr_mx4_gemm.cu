// Products of microscaled 4-bit matrices on the tensor cores: out = A B^T with both matrices in
// MX4 tiles, and the few-token form that takes its tokens in 16 or 32 bits.
//
// Rows are the contraction's tiles as zr_mx4_quantize lays them out, so a stage is a handful of
// contiguous copies: 128 rows x 256 columns of codes already in the swizzle that the tensor cores
// read, and their scales already in the order that one copy takes to tensor memory. Products
// accumulate in fp32.
//
// Measured: pairs of blocks 8192^3 to bf16 in 146 us (7.5 PFLOP/s; the products' own rate, issued
// without a pause, is 9.9 in steps of K = 64, the ones used here), 8192 x 50304 x 2048 in 253 us (6.7).
// Both are bursts; back to back for seconds the power limit lowers the clock, to 1.67 GHz for the
// latter, which takes 281 us then. There the tensor pipe is active 72 % of the cycles, and counters say
// that shared memory is not what the rest waits for: of a stage's 707 cycles the tensor cores' reads
// take 280 (16 KB of A, 16 KB of B, of which a pair's block holds half, and 3 KB of scales), and the
// banks are at 24 % of their rate for reads and at 24 % for writes. What it is has not been settled; the
// scales' copies, to columns that the stage before still reads, cannot overlap its products. Blocks
// alone 2304 x 768 x 777 to fp32 in 5.1 us, of which 1.1 us until the first stage has landed and 1.5 us
// for the results. Few tokens: 1 x 2048 by 8192 x 2048 in 5.2 us, 8 x 2048 by 50304 x 2048 in 12.7 us,
// 4.3 TB/s. (K = 2048 with A's rows kept in shared memory for a run of tiles read half as much and
// was no faster, 294 us: its ring of 4 stages no longer covered a copy's latency.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <exception>
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_mx4.cuh"
#include "zr_nvtx.h"
#include "zr_tensor.cuh"

using zr::fail;

namespace {

// Counts the blocks, ever, whose wait ran out of time. It is never set back: what one stream has heard of
// another may still have to.
__device__ unsigned long long g_gave_up;
// The count that each stream (by device and id) has heard of by zr_mx4_status.
std::mutex g_heard_mu;
std::map<std::pair<int, unsigned long long>, unsigned long long> g_heard;
// Test hook (zr_mx4_stall_waits): bytes that every stage expects beyond those copied.
std::atomic<int> g_stall{0};

// ------------------------------------------------------------------ the general product
// Persistent blocks of six warps: a producer fills a ring of stages (256 columns of K each), one
// thread issues the products, four warps bring the accumulators out, 32 lanes each, while the next
// tile's products run. Two forms, PAIR or not:
//   a block alone takes 128 x 128 of the output;
//   a pair of blocks (a cluster of two on neighbouring multiprocessors) takes 256 x 256 as one
//   product of M = 256: each holds 128 rows of A and 128 of the tile's rows of B, so that 32 KB of
//   codes come in for 128 x 256 of output where a block alone would need 48 KB.
constexpr int kOutWarps = 4, kGemmThreads = 64 + 32 * kOutWarps;
constexpr int kSwizzle = 1024;  // the operands' swizzle repeats every 1024 bytes

template <bool PAIR>
struct Gemm {
  static constexpr int kTiles = PAIR ? 2 : 1;                       // MX4 tiles along M and along N
  static constexpr int kRows = 128 * kTiles, kCols = 128 * kTiles;  // output tile
  // a stage: A codes and scales, this block's B codes, the scales of all of the tile's B rows
  static constexpr int kBCodes = zr::kMxTileBytes, kBScales = kBCodes + zr::kMxCodeBytes;
  static constexpr int kStageBytes = kBScales + kTiles * zr::kMxScaleBytes;
  static constexpr int kStages = PAIR ? 6 : 5;
  // Tensor memory: two accumulators of kCols columns, 8 columns of A's scales, 8 for each tile of B's.
  // The pair's accumulators share 24 columns, or the scales would find no room in the 512: those are
  // read first, and the next tile's products wait for them alone.
  static constexpr int kD1 = PAIR ? 232 : 128, kScaleA = PAIR ? 488 : 256, kScaleB = kScaleA + 8;
  static constexpr int kLag = PAIR ? 1 : 2;   // an accumulator waits for the one so many turns before it
  // an epilogue warp's rows on their way out, 4 KB a time: a block alone has the room for three times,
  // so that it need not wait for each copy (a third of a short product); between a pair's tiles there is time
  static constexpr int kOutBuffers = PAIR ? 1 : 3, kOutBytes = 32 * 128;
  static constexpr int kSmem = kStages * kStageBytes + kOutWarps * kOutBuffers * kOutBytes + 256;
};

struct GemmArgs {
  const uint8_t* a;
  const uint8_t* b;
  void* out;
  int64_t M, N, ldo;
  int kt;          // tiles of 256 along K
  int mt, nt;      // output tiles
  int whole;       // tiles up to here are taken whole; the others, of a pair's last round, in two halves of 128 columns
  int split;       // blocks, a cluster of them, that share a tile's K (of the form with single blocks)
  uint32_t stall;  // test hook: bytes expected that never come
  int vec;         // rows of out begin on 16-byte boundaries, and a map can address it
};

// How a pair's copies see the two matrices: rows of 128 bytes, 136 to an MX4 tile (128 of codes, 8 of
// scales), and how many rows a copy takes. A copy through a map may report to the other block's
// barrier; the tile's bytes are in their place already, so the maps say nothing of swizzles.
constexpr int kTileLines = zr::kMxTileBytes / 128;
struct PairMaps {
  CUtensorMap out, a_tile, b_codes, b_half, b_scales;
};
// The output as a box of 32 rows of 128 bytes takes it, swizzled (unused where vec is 0).
struct OutMap {
  CUtensorMap out;
};

// Output tile of a number: groups of up to 32 tiles of rows, and within a group the rows first, so
// that the blocks at work at one time share few tiles of B and a band of A. `half`: 0 or 1 for one of
// a tile's halves, -1 for all of it.
struct Tile {
  int m, n, half;
};
__device__ __forceinline__ Tile tile_of(const GemmArgs& g, int id) {
  constexpr int kBand = 32;
  Tile t;
  t.half = -1;
  if (id >= g.whole) {
    t.half = (id - g.whole) & 1;
    id = g.whole + ((id - g.whole) >> 1);
  }
  const int per = kBand * g.nt, band = id / per, at = id - band * per;
  const int rows = min(kBand, g.mt - band * kBand);
  t.n = at / rows;
  t.m = band * kBand + (at - t.n * rows);
  return t;
}
__device__ __forceinline__ int tile_count(const GemmArgs& g) { return 2 * g.mt * g.nt - g.whole; }

// The values of 128 bytes of 32 rows, a row in each lane's registers, to memory. They go through this
// warp's staging rows in the order of the 128-byte swizzle (16-byte word j of a row at j ^ (row % 8),
// so that no two lanes write to a bank), from where one copy takes them; where the rows of out do not
// begin on 16-byte boundaries, a row at a time by the lanes.
template <int DT, int BUFFERS>
__device__ __forceinline__ void rows_out(const GemmArgs& g, const CUtensorMap* map, char* stage, const uint32_t* v,
                                         int64_t row0, int64_t col) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2, kCols = 128 / es;
  const int lane = threadIdx.x & 31;
  if (g.vec) {  // the copy that used these staging rows last has read them
    if (lane == 0) zr::stores_read<BUFFERS - 1>();
    __syncwarp();
  }
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (DT == zr::DT_F32) {
      mine[j ^ (lane & 7)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * j + i]);
      mine[j ^ (lane & 7)] = zr::pack8<DT == zr::DT_F32 ? zr::DT_BF16 : DT>(f);
    }
  }
  if (g.vec && (col + kCols <= g.N || g.N * es % 16 == 0)) {  // (copies write whole 16-byte words)
    zr::proxy_fence();
    __syncwarp();
    if (lane == 0) zr::box_store(map, (int)col, (int)row0, zr::smem_u32(stage));
    return;
  }
  __syncwarp();
  using T = typename std::conditional<DT == zr::DT_F32, uint32_t, uint16_t>::type;
  constexpr int kEach = kCols / 32;  // values of a row in a lane, 32 apart
  T* out = static_cast<T*>(g.out) + row0 * g.ldo + col + lane;
  const int rows = (int)(g.M - row0 < 32 ? g.M - row0 : 32);
  const int left = (int)(g.N - col < kCols ? g.N - col : kCols) - lane;
#pragma unroll 8
  for (int r = 0; r < 32; ++r, out += g.ldo) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (r < rows && 32 * i < left)
        out[32 * i] = *reinterpret_cast<const T*>(stage + r * 128 + (((lane + 32 * i) * es) ^ ((r & 7) << 4)));
  }
  if (g.vec && lane == 0) zr::no_store();  // the staging rows' turns are counted in stores
  __syncwarp();
}

// A tile of which each block of a cluster has the products of a part of K, in its shared memory: the
// blocks take its rows in equal shares, add the parts in the order of the blocks and store them. 64 x
// 2048 x 8192 to bf16 in 6.4 us by fours, 9.5 by blocks alone; two waits of the cluster and 64 KB through
// its network cost 1 to 3 us.
constexpr int kPartPitch = 132;  // floats: rows four banks apart
template <int S, int DT>
__device__ __forceinline__ void join_parts(const GemmArgs& g, const float* part, int rank, const Tile& t) {
  using T = typename std::conditional<DT == zr::DT_F32, uint32_t, uint16_t>::type;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)t.m * 128, col = (int64_t)t.n * 128 + lane * 4;
  const int rows = (int)(g.M - row0 < 128 ? g.M - row0 : 128), share = (rows + S - 1) / S;
  const int end = min(rows, (rank + 1) * share);
  auto put = [&](int64_t row, const float v[4]) {
    T u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == zr::DT_F32)
        u[i] = __float_as_uint(v[i]);
      else
        u[i] = zr::from_f32<DT>(v[i]);
    }
    T* out = static_cast<T*>(g.out) + row * g.ldo + col;
    if (g.vec && col + 4 <= g.N) {
      if constexpr (DT == zr::DT_F32)
        *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
      else
        *reinterpret_cast<uint2*>(out) = make_uint2(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < g.N) out[i] = u[i];
    }
  };
  constexpr int kWarps = kGemmThreads / 32, kOnce = S == 2 ? 8 : 2;  // a warp's rows on their way together
  float4 p[kOnce][S];
  for (int r0 = rank * share + warp; r0 < end; r0 += kOnce * kWarps) {
#pragma unroll
    for (int i = 0; i < kOnce; ++i) {
      const int r = r0 + i * kWarps;
      const uint32_t at = zr::smem_u32(part + r * kPartPitch + lane * 4);
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (r < end) p[i][q] = zr::cluster_load4(zr::cluster_addr(at, q));
    }
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
      if (r0 + i * kWarps < end) {
        float v[4] = {p[i][0].x, p[i][0].y, p[i][0].z, p[i][0].w};
#pragma unroll
        for (int q = 1; q < S; ++q) {
          v[0] += p[i][q].x;
          v[1] += p[i][q].y;
          v[2] += p[i][q].z;
          v[3] += p[i][q].w;
        }
        put(row0 + r0 + i * kWarps, v);
      }
  }
}

template <bool PAIR>
using Maps = typename std::conditional<PAIR, PairMaps, OutMap>::type;

template <bool PAIR, int DT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs g, const __grid_constant__ Maps<PAIR> maps) {
  using G = Gemm<PAIR>;
  extern __shared__ __align__(kSwizzle) char smem[];
  const uint32_t stages = zr::smem_u32(smem);
  char* staging = smem + G::kStages * G::kStageBytes;  // (a multiple of the swizzle, too)
  char* tail = staging + kOutWarps * G::kOutBuffers * G::kOutBytes;
  // full: a stage's copies have landed (a pair's, in both blocks: the first block's barrier counts them
  // all); empty: its products are done; done: an accumulator is complete; freed: the turn kLag later
  // may begin
  const uint32_t full = zr::smem_u32(tail), empty = full + 8 * G::kStages, done = empty + 8 * G::kStages,
                 freed = done + 16, drained = freed + 16;
  volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 224);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(tail + 232);
  const int warp = threadIdx.x >> 5;
  const bool split = !PAIR && g.split > 1;  // a tile to a cluster: each block has a part of K
  const int rank = PAIR || split ? (int)zr::cluster_rank() : 0;
  const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x / g.split, step = PAIR ? gridDim.x >> 1 : gridDim.x / g.split;
  const int k0 = split ? (int)((int64_t)g.kt * rank / g.split) : 0;
  const int k1 = split ? (int)((int64_t)g.kt * (rank + 1) / g.split) : g.kt;

  if (warp == 0) {
    zr::tmem_alloc<PAIR>(zr::smem_u32(tmem_at), 512);
  } else if (threadIdx.x == 32) {
    for (int s = 0; s < G::kStages; ++s) {
      zr::bar_init(full + 8 * s, 1);
      zr::bar_init(empty + 8 * s, 1);
    }
    for (int d = 0; d < 2; ++d) {
      zr::bar_init(done + 8 * d, 1);
      zr::bar_init(freed + 8 * d, G::kTiles * kOutWarps);
    }
    zr::bar_init(drained, 1);
    zr::bar_init_fence();
    *gave_up = 0;
  }
  __syncwarp();
  zr::tmem_fence_before();
  if (PAIR)
    zr::cluster_sync();
  else
    __syncthreads();
  zr::tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  const int tiles = tile_count(g);
  zr::let_next_begin();  // it waits for this one's end before it reads or writes
  const int64_t row_bytes = (int64_t)g.kt * zr::kMxTileBytes;  // a row of MX4 tiles

  if (warp == 0) {
    if (zr::elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      zr::wait_for_previous();
      for (int id = first; id < tiles && ok; id += step) {
        const Tile t = tile_of(g, id);
        const bool halved = PAIR && t.half >= 0;
        // a pair's tile may reach past the rows of A or B by an MX4 tile, which is not read then:
        // what the products make of the bytes in its place is not stored
        const int64_t am = PAIR ? 2 * (int64_t)t.m + rank : t.m;
        const int64_t bn = PAIR ? 2 * (int64_t)t.n + (halved ? t.half : 0) : t.n;
        const bool has_a = !PAIR || am * 128 < g.M, second = PAIR && !halved && (bn + 1) * 128 < g.N;
        const uint8_t *a = g.a + am * row_bytes, *b = g.b + bn * row_bytes;
        const int a_line = (int)(am * g.kt) * kTileLines, b_line = (int)(bn * g.kt) * kTileLines;
        // the first block expects the pair's bytes
        const bool peer_a = PAIR && (am + 1) * 128 < g.M;
        const uint32_t pair_bytes =
            zr::kMxTileBytes * (peer_a ? 2 : 1) + (zr::kMxCodeBytes + 2 * zr::kMxScaleBytes) * (second ? 2 : 1);
        const uint32_t bytes = g.stall + (PAIR ? pair_bytes : 2 * zr::kMxTileBytes);
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % G::kStages;
          if (it >= G::kStages && !(ok = zr::bar_wait(empty + 8 * s, (it / G::kStages - 1) & 1, gave_up))) break;
          const uint32_t at = stages + s * G::kStageBytes;
          if constexpr (PAIR) {
            const uint32_t bar = zr::cluster_addr(full + 8 * s, 0);
            const int line = k * kTileLines;
            if (rank == 0) zr::bar_expect(full + 8 * s, bytes);
            if (has_a) zr::pair_copy(at, &maps.a_tile, 0, a_line + line, bar);
            const int next = g.kt * kTileLines;  // the tile's second rows of B
            if (halved)  // 64 rows of it in each block
              zr::pair_copy(at + G::kBCodes, &maps.b_half, 0, b_line + line + rank * 64, bar);
            else if (rank == 0 || second)
              zr::pair_copy(at + G::kBCodes, &maps.b_codes, 0, b_line + line + rank * next, bar);
            zr::pair_copy(at + G::kBScales, &maps.b_scales, 0, b_line + line + 128, bar);
            if (second)
              zr::pair_copy(at + G::kBScales + zr::kMxScaleBytes, &maps.b_scales, 0, b_line + next + line + 128, bar);
          } else {
            const int64_t ko = (int64_t)k * zr::kMxTileBytes;
            zr::bar_expect(full + 8 * s, bytes);
            zr::bulk_copy(at, a + ko, zr::kMxTileBytes, full + 8 * s);
            zr::bulk_copy(at + G::kBCodes, b + ko, zr::kMxTileBytes, full + 8 * s);
          }
        }
      }
      // the block may end once its copies have landed and its stages' products are done
      const uint32_t from = it < G::kStages ? 0 : it - G::kStages;
      for (uint32_t i = from; i < it && ok; ++i)
        ok = zr::bar_wait(empty + 8 * (i % G::kStages), (i / G::kStages) & 1, gave_up);
      if (!ok && (!PAIR || rank == 0)) {  // (the first block waits for the pair's copies; the other ends after it)
        int never = 0;
        for (uint32_t i = from; i < it; ++i) zr::bar_wait(full + 8 * (i % G::kStages), (i / G::kStages) & 1, &never);
      }
    }
  } else if (warp == 1) {
    if ((!PAIR || rank == 0) && zr::elect_one()) {  // a pair's products are issued by its first block
      uint32_t it = 0, turn = 0;
      bool ok = true;
      zr::wait_for_previous();  // nothing is copied before that, and its time is not this product's
      auto release = [&](uint32_t bar) {
        if (PAIR)
          zr::pair_commit(bar, 3);
        else
          zr::mma_commit(bar);
      };
      for (int id = first; id < tiles && ok; id += step, ++turn) {
        const uint32_t d = tmem + (turn & 1) * G::kD1, past = turn - G::kLag;
        const bool halved = PAIR && id >= g.whole;
        if (turn >= G::kLag && !(ok = zr::bar_wait(freed + 8 * (past & 1), (past >> 1) & 1, gave_up))) break;
        zr::tmem_fence_after();
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % G::kStages;
          if (!(ok = zr::bar_wait(full + 8 * s, (it / G::kStages) & 1, gave_up))) break;
          zr::tmem_fence_after();
          const uint32_t at = stages + s * G::kStageBytes;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            zr::copy_scales<PAIR>(tmem + G::kScaleA + 4 * h, zr::scale_rows(at + zr::kMxCodeBytes + 512 * h));
#pragma unroll
            for (int t = 0; t < G::kTiles; ++t)
              if (t == 0 || !halved)
                zr::copy_scales<PAIR>(tmem + G::kScaleB + 4 * (G::kTiles * h + t),
                                      zr::scale_rows(at + G::kBScales + t * zr::kMxScaleBytes + 512 * h));
          }
          const uint64_t da = zr::swizzled_operand(at), db = zr::swizzled_operand(at + G::kBCodes);
#pragma unroll
          for (int q = 0; q < 4; ++q)  // 64 columns, 32 bytes of each row, at a time
            zr::mx_mma<PAIR>(d, da + 2 * q, db + 2 * q, zr::mx_product(G::kRows, halved ? 128 : G::kCols, q & 1),
                             tmem + G::kScaleA + 4 * (q >> 1), tmem + G::kScaleB + 4 * G::kTiles * (q >> 1),
                             k > k0 || q > 0);
          release(empty + 8 * s);
        }
        if (ok) release(done + 8 * (turn & 1));
      }
      if (!ok) {  // no product may be in flight when the tensor memory is given back
        int never = 0;
        if (PAIR)
          zr::pair_commit(drained, 1);
        else
          zr::mma_commit(drained);
        zr::bar_wait(drained, 0, &never);
      }
    }
  } else {
    const int lanes = (warp & 3) * 32;  // the lanes of tensor memory that this warp may read
    char* stage = staging + (warp & 3) * G::kOutBuffers * G::kOutBytes;
    int buffer = 0;
    constexpr int kOnce = DT == zr::DT_F32 ? 32 : 64, kChunks = G::kCols / kOnce;
    auto tell = [&](uint32_t bar) {  // the thread that issues the products
      zr::tmem_fence_before();
      __syncwarp();
      if (zr::elect_one()) {
        if (PAIR)
          zr::cluster_arrive(zr::cluster_addr(bar, 0));
        else
          zr::bar_arrive(bar);
      }
    };
    uint32_t turn = 0;
    zr::wait_for_previous();
    for (int id = first; id < tiles; id += step, ++turn) {
      const Tile t = tile_of(g, id);
      if (!__all_sync(0xFFFFFFFFu, zr::bar_wait(done + 8 * (turn & 1), (turn >> 1) & 1, gave_up))) break;
      zr::tmem_fence_after();
      const uint32_t d = tmem + (turn & 1) * G::kD1 + ((uint32_t)lanes << 16);
      const int64_t row0 = (int64_t)t.m * G::kRows + (PAIR ? rank * 128 : 0) + lanes;
      const int64_t col0 = (int64_t)t.n * G::kCols + (t.half == 1 ? 128 : 0);
      const int chunks = PAIR && t.half >= 0 ? kChunks / 2 : kChunks;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        // the first accumulator's last columns are the second's first
        const int at = (turn & 1) ? c : chunks - 1 - c;
        const int64_t col = col0 + at * kOnce;
        uint32_t v[kOnce];
        if constexpr (kOnce == 32)
          zr::tmem_load32(d + at * kOnce, v);
        else
          zr::tmem_load64(d + at * kOnce, v);
        if (c == (PAIR ? 0 : kChunks - 1)) tell(freed + 8 * (turn & 1));
        if (split) {  // over the stages, which are used up
          float* part = reinterpret_cast<float*>(smem) + (lanes + (threadIdx.x & 31)) * kPartPitch + at * kOnce;
#pragma unroll
          for (int i = 0; i < kOnce; i += 4) *reinterpret_cast<uint4*>(part + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else if (row0 < g.M && col < g.N) {
          rows_out<DT, G::kOutBuffers>(g, &maps.out, stage + buffer * G::kOutBytes, v, row0, col);
          buffer = buffer + 1 < G::kOutBuffers ? buffer + 1 : 0;
        }
      }
    }
    if ((threadIdx.x & 31) == 0) zr::stores_done();  // out of this block's shared memory
  }
  __syncwarp();
  if (split) {
    zr::cluster_sync();
    const Tile t = tile_of(g, first);
    const float* part = reinterpret_cast<const float*>(smem);
    if (g.split == 2)
      join_parts<2, DT>(g, part, rank, t);
    else if (g.split == 4)
      join_parts<4, DT>(g, part, rank, t);
    else
      join_parts<8, DT>(g, part, rank, t);
    __syncwarp();
  }
  zr::tmem_fence_before();
  if (PAIR || split)
    zr::cluster_sync();  // neither block's shared or tensor memory goes before the other is done with it
  else
    __syncthreads();
  zr::tmem_fence_after();
  if (threadIdx.x == 0 && *gave_up) atomicAdd(&g_gave_up, 1ull);
  if (warp == 0) zr::tmem_free<PAIR>(tmem, 512);
}

// ------------------------------------------------------------------ the few-token form
// The weights are the operand with 128 rows, the tokens the one with 16 columns. A block takes
// 128 outputs and, in a cluster of S blocks, 1/S of K: it starts its weight copies, quantises its
// part of the tokens into shared memory meanwhile (or copies them, quantised once by a launch
// before it whose end only this part awaits), and multiplies as the stages arrive. The cluster's
// partial results are added in the order of its blocks.
constexpr int kFewTokens = ZR_MX4_FEW, kFewThreads = 256, kFewStages = 5;  // at most
// A 256-column piece of 16 tokens: 2048 bytes of codes and, behind the codes of all pieces, twice 256
// of scales (what a copy of 512 brings of the next piece's stands for tokens past the 16th).
constexpr int kXCodes = 2048, kXScales = 512;
constexpr int kFewTail = 256;

struct FewArgs {
  const void* x;
  const uint8_t* xq;  // the tokens as an MX4 matrix, or null: quantised here from x
  const uint8_t* w;
  void* out;
  int64_t M, K, N, ldx, ldo;
  int kt, xdt, odt;
  int stages;  // of a block's ring
  uint32_t stall;  // test hook: bytes expected that never come
};

__host__ __device__ constexpr int few_smem(int k_tiles, int stages) {
  return stages * zr::kMxTileBytes + k_tiles * (kXCodes + kXScales) + 256 + kFewTail;
}

// Eight values of a row from element e on, as they are (the upper eight bytes pair only in fp32);
// zeros past the `left` that the row still has.
struct Eight {
  uint4 lo, hi;
};
__device__ __forceinline__ Eight load_eight(const void* x, int dt, int64_t e, int64_t left) {
  const int es = dt == zr::DT_F32 ? 4 : 2;
  const char* p = static_cast<const char*>(x) + e * es;
  Eight r{};
  if (left >= 8) {
    r.lo = zr::load16(p);
    if (dt == zr::DT_F32) r.hi = zr::load16(p + 16);
  } else {
    uint32_t w[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if (dt == zr::DT_F32)
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else
          w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      }
    r.lo = make_uint4(w[0], w[1], w[2], w[3]);
    r.hi = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}
__device__ __forceinline__ void open_eight(const Eight& u, int dt, float v[8]) {
  if (dt == zr::DT_F32) {
    const uint32_t w[8] = {u.lo.x, u.lo.y, u.lo.z, u.lo.w, u.hi.x, u.hi.y, u.hi.z, u.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else if (dt == zr::DT_BF16) {
    zr::unpack8<zr::DT_BF16>(u.lo, v);
  } else {
    zr::unpack8<zr::DT_F16>(u.lo, v);
  }
}

__device__ __forceinline__ void store_as(void* out, int dt, int64_t i, float v) {
  if (dt == zr::DT_F32)
    static_cast<float*>(out)[i] = v;
  else
    static_cast<uint16_t*>(out)[i] = dt == zr::DT_BF16 ? zr::from_f32<zr::DT_BF16>(v) : zr::from_f32<zr::DT_F16>(v);
}

template <int S>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ FewArgs g) {
  extern __shared__ __align__(kSwizzle) char smem[];
  const int n = blockIdx.x / S, rank = S > 1 ? (int)zr::cluster_rank() : 0;
  const int k0 = (int)((int64_t)g.kt * rank / S), nk = (int)((int64_t)g.kt * (rank + 1) / S) - k0;
  const int k_most = (g.kt + S - 1) / S;
  char* xq = smem + g.stages * zr::kMxTileBytes;
  char* xscale = xq + k_most * kXCodes;
  char* tail = xscale + k_most * kXScales + 256;
  const uint32_t stages = zr::smem_u32(smem);
  const uint32_t full = zr::smem_u32(tail), empty = full + 8 * kFewStages, done = empty + 8 * kFewStages,
                 tokens = done + 8;
  volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 192);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(tail + 200);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* w = g.w + ((int64_t)n * g.kt + k0) * zr::kMxTileBytes;

  if (warp == 0) {
    zr::tmem_alloc(zr::smem_u32(tmem_at), 32);
  } else if (warp == 5 && lane == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      zr::bar_init(full + 8 * s, 1);
      zr::bar_init(empty + 8 * s, 1);
    }
    zr::bar_init(done, 1);
    zr::bar_init(tokens, 1);
    zr::bar_init_fence();
    zr::proxy_fence();
    *gave_up = 0;
    for (int k = 0; k < nk && k < g.stages; ++k) {
      zr::bar_expect(full + 8 * k, zr::kMxTileBytes + g.stall);
      zr::bulk_copy(stages + k * zr::kMxTileBytes, w + (int64_t)k * zr::kMxTileBytes, zr::kMxTileBytes, full + 8 * k);
    }
  }
  __syncwarp();
  if (g.xq) {
    if (warp == 5 && lane == 0) {  // the first 16 rows of each tile and of its scales
      zr::wait_for_previous();
      zr::bar_expect(tokens, nk * (kXCodes + kXScales));
      for (int k = 0; k < nk; ++k) {
        const uint8_t* tile = g.xq + (int64_t)(k0 + k) * zr::kMxTileBytes;
        zr::bulk_copy(zr::smem_u32(xq + k * kXCodes), tile, kXCodes, tokens);
        for (int h = 0; h < 2; ++h)
          zr::bulk_copy(zr::smem_u32(xscale + k * kXScales + h * 256), tile + zr::kMxCodeBytes + h * 512, 256, tokens);
      }
    }
  } else {
    // four lanes to a block of 32 values, a warp to 256 of a row, several rows' loads in flight. What
    // lies in the place of tokens beyond M is left as it is: what it gives is not stored.
    constexpr int kBatch = 4, kWarps = kFewThreads / 32;
    const int j = lane >> 2;
    for (int t0 = warp; t0 < nk * (int)g.M; t0 += kBatch * kWarps) {
      Eight u[kBatch];
      int row[kBatch], piece[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i * kWarps;
        row[i] = t / nk;
        piece[i] = t - row[i] * nk;
        const int64_t c = (int64_t)(k0 + piece[i]) * 256 + lane * 8;
        u[i] = row[i] < g.M && c < g.K ? load_eight(g.x, g.xdt, row[i] * g.ldx + c, g.K - c) : Eight{};
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = row[i], k = piece[i];
        if (r >= g.M) break;
        float v[8];
        open_eight(u[i], g.xdt, v);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int byte = zr::mx_scale_byte<false>(m);
        const float inv = byte == 255 ? 0.0f : zr::mx_inverse(byte);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], inv);
        const uint32_t codes = byte == 255 ? 0u : zr::mx_codes8(v);
        *reinterpret_cast<uint32_t*>(xq + k * kXCodes + r * 128 + ((j ^ (r & 7)) << 4) + (lane & 3) * 4) = codes;
        if ((lane & 3) == 0) xscale[k * kXScales + (j >> 2) * 256 + r * 16 + (j & 3)] = (char)byte;
      }
    }
  }
  __syncwarp();
  zr::proxy_fence();
  zr::tmem_fence_before();
  __syncthreads();
  zr::tmem_fence_after();
  const uint32_t tmem = *tmem_at, scale_a = tmem + 16, scale_b = tmem + 24;

  if (warp == 4) {
    if (zr::elect_one()) {
      int k = g.xq && !zr::bar_wait(tokens, 0, gave_up) ? nk : 0;
      for (; k < nk; ++k) {
        const int s = k % g.stages;
        if (!zr::bar_wait(full + 8 * s, (k / g.stages) & 1, gave_up)) break;
        zr::tmem_fence_after();
        const uint32_t at = stages + s * zr::kMxTileBytes, xt = zr::smem_u32(xq + k * kXCodes);
        const uint32_t xsc = zr::smem_u32(xscale + k * kXScales);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          zr::copy_scales(scale_a + 4 * h, zr::scale_rows(at + zr::kMxCodeBytes + 512 * h));
          zr::copy_scales(scale_b + 4 * h, zr::scale_rows(xsc + 256 * h));
        }
        const uint64_t da = zr::swizzled_operand(at), db = zr::swizzled_operand(xt);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          zr::mx_mma(tmem, da + 2 * q, db + 2 * q, zr::mx_product(128, 16, q & 1), scale_a + 4 * (q >> 1),
                     scale_b + 4 * (q >> 1), (k | q) != 0);
        if (k + g.stages < nk) zr::mma_commit(empty + 8 * s);
      }
      if (k < nk || *gave_up) {  // no copy may be in flight at the end
        int never = 0;
        if (g.xq) zr::bar_wait(tokens, 0, &never);
        for (int i = 0; i < nk && nk <= g.stages; ++i) zr::bar_wait(full + 8 * i, 0, &never);
      }
      zr::mma_commit(done);  // after a wait that gave up too: nothing may be in flight at the end
    }
  } else if (warp == 5 && nk > g.stages) {
    if (zr::elect_one()) {
      int k = g.stages;
      for (; k < nk; ++k) {
        const int s = k % g.stages;
        if (!zr::bar_wait(empty + 8 * s, (k / g.stages - 1) & 1, gave_up)) break;
        zr::bar_expect(full + 8 * s, zr::kMxTileBytes + g.stall);
        zr::bulk_copy(stages + s * zr::kMxTileBytes, w + (int64_t)k * zr::kMxTileBytes, zr::kMxTileBytes, full + 8 * s);
      }
      int never = 0;
      for (int i = k - g.stages; i < k; ++i) zr::bar_wait(full + 8 * (i % g.stages), (i / g.stages) & 1, &never);
    }
  }
  __syncwarp();

  float* part = reinterpret_cast<float*>(smem);  // [token][128], over the stages once they are used up
  if (warp < 4) {
    uint32_t v[16];
    const bool ok = __all_sync(0xFFFFFFFFu, zr::bar_wait(done, 0, gave_up));
    zr::tmem_fence_after();
    if (ok) {
      zr::tmem_load16(tmem + ((uint32_t)(warp * 32) << 16), v);
      const int64_t col = (int64_t)n * 128 + warp * 32 + lane;
#pragma unroll
      for (int t = 0; t < kFewTokens; ++t)
        if (t < g.M) {
          if (S > 1)
            part[t * 128 + warp * 32 + lane] = __uint_as_float(v[t]);
          else if (col < g.N)
            store_as(g.out, g.odt, t * g.ldo + col, __uint_as_float(v[t]));
        }
    }
    zr::tmem_fence_before();
  }
  __syncwarp();
  if (S > 1) {
    zr::cluster_sync();
    constexpr int kShare = 128 / S;
    for (int e = threadIdx.x; e < (int)g.M * kShare; e += kFewThreads) {
      const int t = e / kShare, c = rank * kShare + e % kShare;
      const uint32_t at = zr::smem_u32(part + t * 128 + c);
      float sum = 0.0f;
#pragma unroll
      for (int r = 0; r < S; ++r) {
        const float p = zr::cluster_load(zr::cluster_addr(at, r));
        sum = r ? sum + p : p;
      }
      const int64_t col = (int64_t)n * 128 + c;
      if (col < g.N) store_as(g.out, g.odt, t * g.ldo + col, sum);
    }
    __syncwarp();
    zr::cluster_sync();  // a block's shared memory stays until the others have read it
  } else {
    __syncthreads();
  }
  zr::tmem_fence_after();
  if (threadIdx.x == 0 && *gave_up) atomicAdd(&g_gave_up, 1ull);
  if (warp == 0) zr::tmem_free(tmem, 32);
}

// The driver's encoder of tensor maps, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    return (PFN_cuTensorMapEncodeTiled_v12000)(e == cudaSuccess && found == cudaDriverEntryPointSuccess ? p : nullptr);
  }();
  return fn;
}

// A map of an MX4 matrix's `tiles` tiles as lines of 128 bytes, copied `lines` at a time.
bool encode_lines(CUtensorMap* map, const void* q, int64_t tiles, int lines) {
  const cuuint64_t size[2] = {128, (cuuint64_t)(tiles * kTileLines)}, stride[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)lines}, step[2] = {1, 1};
  return map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), size, stride, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of the output.
bool encode_out(CUtensorMap* map, const GemmArgs& g, int dt) {
  const int es = dt == zr::DT_F32 ? 4 : 2;
  const CUtensorMapDataType type = dt == zr::DT_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dt == zr::DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t size[2] = {(cuuint64_t)g.N, (cuuint64_t)g.M}, stride[1] = {(cuuint64_t)g.ldo * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32}, step[2] = {1, 1};
  return map_encoder()(map, type, 2, g.out, size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, int DT>
zr_status launch_gemm(const GemmArgs& g, int blocks, cudaStream_t s) {
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_mx4_matmul", (const void*)gemm_kernel<PAIR, DT>, Gemm<PAIR>::kSmem)) return st;
  Maps<PAIR> maps;
  if (!map_encoder() || (g.vec && !encode_out(&maps.out, g, DT)))
    return fail(ZR_ERR_CUDA, "zr_mx4_matmul: the driver gave no tensor map");
  if constexpr (PAIR) {
    const int64_t a_tiles = zr::mx_tiles(g.M, zr::kMxRows) * g.kt, b_tiles = zr::mx_tiles(g.N, zr::kMxRows) * g.kt;
    if (!encode_lines(&maps.a_tile, g.a, a_tiles, kTileLines) ||
        !encode_lines(&maps.b_codes, g.b, b_tiles, zr::kMxRows) ||
        (g.whole < g.mt * g.nt && !encode_lines(&maps.b_half, g.b, b_tiles, zr::kMxRows / 2)) ||
        !encode_lines(&maps.b_scales, g.b, b_tiles, zr::kMxScaleBytes / 128))
      return fail(ZR_ERR_CUDA, "zr_mx4_matmul: the driver gave no tensor map");
  }
  cudaError_t e = zr::launch(gemm_kernel<PAIR, DT>, blocks, kGemmThreads, Gemm<PAIR>::kSmem, PAIR ? 2 : g.split, true, s, g,
                             maps);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_mx4_matmul: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}

// Tiles of 256 x 256 that pairs take in rounds. A last round that fewer than half of the pairs would be
// busy with is taken in halves (2048 x 8192 x 8192: 48.2 us in 4 rounds, 45.6 in 3.5); not where the last
// column of tiles has no second half, and not for want of a first round (256 x 8192 x 8192 in halves
// 20.5 us, where as many whole tiles take 14.3).
bool halves_last(int64_t M, int64_t N, int sms) {
  const int64_t nt = zr::mx_tiles(N, 256), tiles = zr::mx_tiles(M, 256) * nt, pairs = sms / 2, last = tiles % pairs;
  return tiles > pairs && last > 0 && 2 * last <= pairs && nt * 256 - N < 128;
}

// Whether pairs with their larger tiles are faster than single blocks. A pair's round costs about 1.3
// times a block's and does twice the work, but its start and its last output take longer, so that few
// rounds, or few of K, favour blocks. The times, in 10 ns: a start, then for each round 256 columns of K
// at a time and what of the output does not overlap (measured; blocks and pairs at 2048 x 2048 x 2048 7.0
// and 7.7 us, 2048 x 2048 x 8192 16.7 and 14.3, 2135 x 2109 x 8192 18.1 and 22.2, 2048 x 6144 x 512 to
// fp32 11.2 and 14.5).
bool pairs_faster(int64_t M, int64_t N, int64_t kt, zr_dtype dt, int sms) {
  const int64_t m1 = zr::mx_tiles(M, 128), n1 = zr::mx_tiles(N, 128), m2 = zr::mx_tiles(M, 256), n2 = zr::mx_tiles(N, 256);
  const int64_t most = 0x7FFFFFFF / kTileLines;
  if (m1 > most / kt || n1 > most / kt) return false;  // 32 bits hold a matrix's lines
  const int64_t pairs = sms / 2;
  const int64_t rounds = (m1 * n1 + sms - 1) / sms, twice = 2 * ((m2 * n2 + pairs - 1) / pairs) - halves_last(M, N, sms);
  const bool wide = dt == ZR_F32;
  const int64_t single = 22 * kt + (wide ? 80 : 30), paired = 29 * kt + (wide ? 210 : kt < 6 ? 200 - 29 * kt : 40);
  return 470 + twice * paired / 2 < 290 + rounds * single;
}

// How many blocks share a tile's K, where there are more of them than tiles: what it saves at 0.22 us for
// 256 columns against what it costs, which grows with the rows (measured for 17, 64 and 128). The blocks
// of a cluster lie on neighbouring SMs, so that not all SMs find a place in one of four, and only half in
// one of eight (128 of those took two rounds).
int shares_of_k(int64_t M, int64_t tiles, int64_t kt, int sms) {
  const int64_t rows = M < 128 ? M : 128;
  int best = 1;
  int64_t gain = 20;
  for (int s = 2; s <= 8 && s <= kt && tiles * s <= (s == 2 ? sms : s == 4 ? sms * 6 / 7 : sms / 2); s *= 2) {
    const int64_t g = (kt < 1000 ? 22 * kt : 22000) * (s - 1) / s - 85 - rows * (100 + 8 * s) / 100;
    if (g > gain) gain = g, best = s;
  }
  return best;
}

zr_status matmul(const char* what, const void* a, int64_t M, const void* b, int64_t N, int64_t K, void* out,
                 zr_dtype dt, int64_t ldo, cudaStream_t s) {
  const int es = dt == ZR_F32 ? 4 : 2;
  if (K == 0) {  // a sum of nothing
    cudaError_t e = cudaMemset2DAsync(out, (size_t)ldo * es, 0, (size_t)N * es, (size_t)M, s);
    return e == cudaSuccess ? ZR_OK : fail(ZR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  const int sms = zr::sm_count(what);
  if (sms == 0) return ZR_ERR_CUDA;
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.b = static_cast<const uint8_t*>(b);
  g.out = out;
  g.M = M; g.N = N; g.ldo = ldo;
  g.stall = g_stall.load(std::memory_order_relaxed) ? 16 : 0;
  const int64_t kt = zr::mx_tiles(K, zr::kMxCols);
  const bool pair = pairs_faster(M, N, kt, dt, sms);
  const int64_t mt = zr::mx_tiles(M, pair ? 256 : 128), nt = zr::mx_tiles(N, pair ? 256 : 128);
  if (kt > 0x7FFFFFFF || nt > (1 << 25) || mt > 0x3FFFFFFF / nt)
    return fail(ZR_ERR_UNSUPPORTED, "%s: the product has too many tiles", what);
  g.kt = (int)kt; g.mt = (int)mt; g.nt = (int)nt;
  g.vec = ldo * es % 16 == 0 && ldo < (int64_t)1 << 36 && M <= 0x7FFFFFFF && N <= 0x7FFFFFFF;
  g.whole = g.mt * g.nt;
  g.split = 1;
  if (pair) {
    const int pairs = sms / 2, last = g.whole % pairs, blocks = 2 * (g.whole < pairs ? g.whole : pairs);
    if (halves_last(M, N, sms)) g.whole -= last;
    if (dt == ZR_F16) return launch_gemm<true, zr::DT_F16>(g, blocks, s);
    if (dt == ZR_BF16) return launch_gemm<true, zr::DT_BF16>(g, blocks, s);
    return launch_gemm<true, zr::DT_F32>(g, blocks, s);
  }
  g.split = shares_of_k(M, mt * nt, kt, sms);
  const int blocks = g.split > 1 ? (int)(mt * nt) * g.split : (int)(mt * nt < sms ? mt * nt : sms);
  if (dt == ZR_F16) return launch_gemm<false, zr::DT_F16>(g, blocks, s);
  if (dt == ZR_BF16) return launch_gemm<false, zr::DT_BF16>(g, blocks, s);
  return launch_gemm<false, zr::DT_F32>(g, blocks, s);
}

template <int S>
zr_status launch_few(const FewArgs& g, int blocks, int smem, cudaStream_t s) {
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_mx4_linear", (const void*)few_kernel<S>, zr::kSmemMost)) return st;
  cudaError_t e = zr::launch(few_kernel<S>, blocks, kFewThreads, smem, S, g.xq != nullptr, s, g);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_mx4_linear: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}

}  // namespace

extern "C" zr_status zr_mx4_matmul(const void* a, int64_t M, const void* b, int64_t N, int64_t K, void* out,
                                   zr_dtype dt, int64_t ldo, void* stream) {
  zr::clear_error();
  zr::Range range("zr_mx4_matmul");
  if (!zr::dtype_ok(dt)) return fail(ZR_ERR_INVALID, "zr_mx4_matmul: bad dtype %d", (int)dt);
  if (M < 0 || N < 0 || K < 0) return fail(ZR_ERR_INVALID, "zr_mx4_matmul: negative size");
  if (ldo < N) return fail(ZR_ERR_INVALID, "zr_mx4_matmul: the row stride of out is under N");
  if (M == 0 || N == 0) return ZR_OK;
  if (!out || (K > 0 && (!a || !b))) return fail(ZR_ERR_INVALID, "zr_mx4_matmul: null pointer");
  if (!zr::aligned16(a) || !zr::aligned16(b) || !zr::aligned16(out))
    return fail(ZR_ERR_INVALID, "zr_mx4_matmul: a pointer is not 16-byte aligned");
  return matmul("zr_mx4_matmul", a, M, b, N, K, out, dt, ldo, static_cast<cudaStream_t>(stream));
}

extern "C" zr_status zr_mx4_linear(const void* x, zr_dtype xdt, int64_t M, int64_t ldx, const void* w, int64_t N,
                                   int64_t K, void* out, zr_dtype dt, int64_t ldo, void* xq, void* stream) {
  zr::clear_error();
  zr::Range range("zr_mx4_linear");
  if (!zr::dtype_ok(xdt) || !zr::dtype_ok(dt)) return fail(ZR_ERR_INVALID, "zr_mx4_linear: bad dtype");
  if (M < 0 || N < 0 || K < 0) return fail(ZR_ERR_INVALID, "zr_mx4_linear: negative size");
  if (ldx < K || ldo < N) return fail(ZR_ERR_INVALID, "zr_mx4_linear: a row stride is under the row");
  if (M == 0 || N == 0) return ZR_OK;
  if (!out || (K > 0 && (!x || !w))) return fail(ZR_ERR_INVALID, "zr_mx4_linear: null pointer");
  if (!zr::aligned16(x) || !zr::aligned16(w) || !zr::aligned16(out) || !zr::aligned16(xq))
    return fail(ZR_ERR_INVALID, "zr_mx4_linear: a pointer is not 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t kt = zr::mx_tiles(K, zr::kMxCols), nt = zr::mx_tiles(N, 128);
  // blocks of a cluster share K where the outputs alone would leave multiprocessors idle: two blocks
  // fit on one, so up to twice their number
  const int sms = zr::sm_count("zr_mx4_linear");
  if (sms == 0) return ZR_ERR_CUDA;
  int split = 1;
  while (split < 8 && nt * split * 2 <= 2 * sms && split * 2 <= kt) split *= 2;
  auto pieces = [&](int by) { return (int)(zr::mx_tiles(kt, by) < 4096 ? zr::mx_tiles(kt, by) : 4096); };
  while (split < 8 && split * 2 <= kt && few_smem(pieces(split), 1) > zr::kSmemMost) split *= 2;
  const int most = pieces(split);
  if (M <= kFewTokens && K > 0 && few_smem(most, 1) <= zr::kSmemMost && nt * split <= 0x7FFFFFFF) {
    FewArgs g{};
    g.x = x; g.w = static_cast<const uint8_t*>(w); g.out = out;
    g.M = M; g.K = K; g.N = N; g.ldx = ldx; g.ldo = ldo;
    g.kt = (int)kt; g.xdt = (int)xdt; g.odt = (int)dt;
    g.stall = g_stall.load(std::memory_order_relaxed) ? 16 : 0;
    const int blocks = (int)(nt * split);
    // as many stages as fit where every block that there is, up to three to a multiprocessor, is resident
    // at once: one more wave costs more than a shorter ring
    const int resident = blocks <= sms ? 1 : blocks <= 2 * sms ? 2 : 3;
    g.stages = kFewStages < most ? kFewStages : most;
    while (g.stages > 2 && few_smem(most, g.stages) > (zr::kSmemMost + 1024) / resident - 1024) --g.stages;
    while (g.stages > 1 && few_smem(most, g.stages) > zr::kSmemMost) --g.stages;
    const int smem = few_smem(most, g.stages);
    // Every block quantises its part of the tokens anew, in a time that its warps' pieces of 256 values
    // decide; past four each (8 tokens of 2048:
    // 15.3 us for 50304 outputs, against 12.7) a launch that does it once is faster.
    if (xq && M * most > 4 * (kFewThreads / 32)) {
      if (zr_status st = zr_mx4_quantize(x, xdt, M, K, ldx, nullptr, 0, xq, nullptr, stream)) return st;
      g.xq = static_cast<const uint8_t*>(xq);
    }
    if (split == 8) return launch_few<8>(g, blocks, smem, s);
    if (split == 4) return launch_few<4>(g, blocks, smem, s);
    if (split == 2) return launch_few<2>(g, blocks, smem, s);
    return launch_few<1>(g, blocks, smem, s);
  }
  if (K > 0) {
    if (!xq) return fail(ZR_ERR_INVALID, "zr_mx4_linear: more than %d tokens (or a very long K) need xq", kFewTokens);
    if (zr_status st = zr_mx4_quantize(x, xdt, M, K, ldx, nullptr, 0, xq, nullptr, stream)) return st;
  }
  return matmul("zr_mx4_linear", xq, M, w, N, K, out, dt, ldo, s);
}

extern "C" zr_status zr_mx4_status(void* stream) {
  zr::clear_error();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int device = 0;
  unsigned long long id = 0, count = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaStreamGetId(s, &id);  // (a handle may come again for another stream)
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&count, g_gave_up, sizeof count, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_mx4_status: %s", cudaGetErrorString(e));
  bool more = false;
  try {
    std::lock_guard<std::mutex> lock(g_heard_mu);
    unsigned long long& heard = g_heard[{device, id}];
    more = count > heard;
    if (more) heard = count;
  } catch (const std::exception&) {
    return fail(ZR_ERR_OOM, "zr_mx4_status: no memory for the stream's record");
  }
  if (more)
    return fail(ZR_ERR_TIMEOUT, "zr_mx4_status: a product gave up a wait; outputs since this stream's last check are void");
  return ZR_OK;
}

extern "C" zr_status zr_mx4_stall_waits(int on) {
  zr::clear_error();
  g_stall.store(on ? 1 : 0, std::memory_order_relaxed);
  return ZR_OK;
}
