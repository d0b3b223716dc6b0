// Quantisation of a matrix to the microscaled 4-bit format (by its rows, by its columns, or
// both from one read) and back to the values that the codes stand for.
//
// Quantising reads a value once and writes 17/32 byte of it for each direction; a block brings a
// patch to shared memory by asynchronous copies and lets each thread take whole blocks of 32 from
// there, along the rows and then along the columns, so that no scale needs a reduction between
// threads. To nearest it is bound by memory: fp32 50304 x 2048 both ways in 80 us, 6.5 TB/s of the
// 6.7 that a copy reaches. By chance, with a random byte more per value, the rounding's whole-number
// steps bind it: bf16 8192 x 8192 both ways in 64 us, 4.3 TB/s with the integer pipe at 75 %.
// Dequantising bf16 50304 x 2048 takes 39 us, 6.7 TB/s; with rows of odd length 4099 x 2049 in
// 7.0 us, 3.0 TB/s, where 4096 x 2048 takes 3.9.
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_mx4.cuh"
#include "zr_nvtx.h"
#include "zr_tensor.cuh"

using zr::fail;

namespace {

// A block quantises 64 x 128 values: half a tile's rows by half its columns in q, half a tile's rows by
// a quarter of its columns in qt. Blocks of twice the rows and threads left a longer last wave (4099 x
// 2049 in bf16 by chance both ways 21.1 us, then; 16.9 now).
constexpr int kThreads = 128, kRows = 64, kCols = 128;
constexpr int kDequantThreads = 256;

struct QuantArgs {
  const void* x;
  const uint8_t* rand;  // 8 random bits per value, or null (to nearest)
  uint8_t* q;           // rows x cols, or null
  uint8_t* qt;          // cols x rows, or null
  int64_t rows, cols, ldx, ldr;
  int64_t q_tiles, qt_tiles;  // tiles along the columns of q, of qt
  int64_t col_patches;        // patches along the columns of x
  int x_step, rand_step;      // bytes that the beginnings of their rows are multiples of: 16, 8, 4, or less
  int q_row_patches, qt_col_patches;  // patches that q has along its rows, qt along x's columns
};

template <int DT>
struct Shape {
  static constexpr int es = DT == zr::DT_F32 ? 4 : 2;
  static constexpr int pitch = kCols * es + 16;
  // Rows 16 bytes apart in their banks, the two blocks of 32 rows another 64 bytes: so the 8 rows' or
  // the 2 row blocks' worth of lanes that one access serves fall on different banks.
  __host__ __device__ static constexpr int at(int r) { return r * pitch + (r >> 5) * 64; }
  static constexpr int bytes = kRows * pitch + 64;
};
constexpr int kRandPitch = kCols + 16;
__host__ __device__ constexpr int rand_at(int r) { return r * kRandPitch + (r >> 5) * 32; }
constexpr int kRandBytes = kRows * kRandPitch + 32;

// The largest magnitude so far and those of a word of the patch (one fp32 value, or two of 16 bits
// apart). NaN, if there is one.
template <int DT>
__device__ __forceinline__ uint32_t amax_word(uint32_t m, uint32_t w) {
  uint32_t r;
  if (DT == zr::DT_F32)
    asm("{\n .reg .f32 a;\n abs.f32 a, %2;\n max.NaN.f32 %0, %1, a;\n}\n"
        : "=f"(*reinterpret_cast<float*>(&r))
        : "f"(__uint_as_float(m)), "f"(__uint_as_float(w)));
  else if (DT == zr::DT_BF16)
    asm("{\n .reg .b32 a;\n abs.bf16x2 a, %2;\n max.NaN.bf16x2 %0, %1, a;\n}\n" : "=r"(r) : "r"(m), "r"(w));
  else
    asm("{\n .reg .b32 a;\n abs.f16x2 a, %2;\n max.NaN.f16x2 %0, %1, a;\n}\n" : "=r"(r) : "r"(m), "r"(w));
  return r;
}

// The fp32 bits of a magnitude's 16-bit pattern.
template <int DT>
__device__ __forceinline__ uint32_t bits_of_half(uint32_t h) {
  return __float_as_uint(zr::to_f32<DT>((uint16_t)h));
}

// Eight values to codes; `dither` only by chance.
template <bool CHANCE>
__device__ __forceinline__ uint32_t codes_of(const float x[8], float inv, const uint32_t dither[8]) {
  if constexpr (CHANCE) {
    return zr::mx_codes8_by_chance(x, __fmul_rn(inv, 0.25f), dither);
  } else {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __fmul_rn(x[j], inv);
    return zr::mx_codes8(t);
  }
}

// Combines the scale bytes of N lanes (lane % N = byte) into a word.
template <int N>
__device__ __forceinline__ uint32_t lane_bytes(int byte) {
  uint32_t w = (uint32_t)byte << (8 * (threadIdx.x & (N - 1)));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 1);
  if (N == 4) w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2);
  return w;
}

// The memory words that hold a patch's rows, WORDS + 1 for each (the first may begin before the row),
// to its places in shared memory; zeros for what lies past `bytes` of a row and past `rows`. A copy of
// no bytes still names an address, which has to be one that is there: `any`, the matrix's first.
template <int WORDS>
__device__ __forceinline__ void fetch(int (*at)(int), char* to, const void* any, const char* from, int64_t pitch,
                                      int rows, int bytes) {
  constexpr int kEach = WORDS + 1, kDown = kThreads / kEach, kOver = kThreads % kEach;
  int r = threadIdx.x / kEach, j = threadIdx.x % kEach;
  const char* row = from + r * pitch;
#pragma unroll 3
  for (; r < kRows;) {
    const int before = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    const int left = r < rows && bytes > 0 ? bytes + before - 16 * j : 0;
    const void* word = left > 0 ? row - before + 16 * j : any;
    zr::copy16_of(zr::smem_u32(to + at(r) + 16 * j), word, left < 16 ? (left > 0 ? left : 0) : 16);
    const int down = j + kOver >= kEach ? kDown + 1 : kDown;
    j += j + kOver >= kEach ? kOver - kEach : kOver;
    r += down;
    row += down * pitch;
  }
}
// The same of rows that begin on boundaries of STEP bytes: STEP at a time they are in their places at
// once: 20000 x 1028 bf16 in 12.0 us, 15.5 by words of 16 bytes that are moved then. Values 4 bytes at a time
// were no faster than those (20000 x 1025 fp32 25.3 and 24.4 us); random bytes, a quarter as many, were.
template <int WORDS, int STEP>
__device__ __forceinline__ void fetch_by(int (*at)(int), char* to, const void* any, const char* from, int64_t pitch,
                                         int rows, int bytes) {
  constexpr int kEach = WORDS * 16 / STEP, kDown = kThreads / kEach;  // copies to a row, rows between a thread's
  const int first = threadIdx.x / kEach, j = threadIdx.x % kEach;
  const int left = min(max(bytes - j * STEP, 0), STEP);
  const char* p = from + first * pitch + j * STEP;
#pragma unroll 8
  for (int r = first; r < kRows; r += kDown, p += kDown * pitch) {
    const int n = r < rows ? left : 0;
    zr::copy_of<STEP>(zr::smem_u32(to + at(r) + STEP * j), n > 0 ? p : any, n);
  }
}
// Moves each of those rows to the beginning of its place.
template <int WORDS>
__device__ __forceinline__ void align(int (*at)(int), char* rows, const char* from, int64_t pitch) {
  constexpr int kAtOnce = 32 / WORDS;  // rows of a warp
  const int lane = threadIdx.x & 31, j = lane % WORDS;
#pragma unroll 4
  for (int r = (threadIdx.x >> 5) * kAtOnce + lane / WORDS; r < kRows; r += kThreads / WORDS) {
    uint4* row = reinterpret_cast<uint4*>(rows + at(r));
    const uint32_t before = (uint32_t)(reinterpret_cast<uintptr_t>(from + r * pitch) & 15);
    const uint4 v = zr::shift16(row[j], row[j + 1], before);
    __syncwarp();
    if (before) row[j] = v;
  }
}

template <int DT, bool CHANCE>
__global__ void __launch_bounds__(kThreads, DT == zr::DT_F32 ? (CHANCE ? 5 : 6) : 8)
    quant_kernel(const __grid_constant__ QuantArgs a) {
  using S = Shape<DT>;
  extern __shared__ __align__(16) char smem[];
  uint8_t* srand = reinterpret_cast<uint8_t*>(smem + S::bytes);
  const int tid = threadIdx.x;
  const int64_t pr = blockIdx.x / a.col_patches, pc = blockIdx.x - pr * a.col_patches;
  const int64_t r0 = pr * kRows, c0 = pc * kCols;
  zr::let_next_begin();  // a product of what this writes (it waits for that before it reads)

  // ---- the patch to shared memory as it is, zeros outside the matrix
  constexpr int kWords = kCols * S::es / 16, kRandWords = kCols / 16;  // 16-byte words of a row
  const char* x = static_cast<const char*>(a.x) + (r0 * a.ldx + c0) * S::es;
  const char* rnd0 = reinterpret_cast<const char*>(a.rand) + r0 * a.ldr + c0;
  const int64_t down = a.rows - r0, right = a.cols - c0;
  const int rows = (int)(down < kRows ? (down > 0 ? down : 0) : kRows);
  const int cols = (int)(right < kCols ? (right > 0 ? right : 0) : kCols);
  const bool inside = rows == kRows && cols == kCols;
  if (a.x_step == 16 && inside) {
    constexpr int kStep = kThreads / kWords;  // rows between a thread's words
    const char* from = x + (tid / kWords) * a.ldx * S::es + (tid % kWords) * 16;
    const uint32_t to = zr::smem_u32(smem) + (tid / kWords) * S::pitch + (tid % kWords) * 16;
#pragma unroll
    for (int i = 0; i < kRows / kStep; ++i) zr::copy16(to + S::at(i * kStep), from + i * kStep * a.ldx * S::es);
  } else if (a.x_step == 16) {
    fetch_by<kWords, 16>(S::at, smem, a.x, x, a.ldx * S::es, rows, cols * S::es);
  } else if (a.x_step == 8) {
    fetch_by<kWords, 8>(S::at, smem, a.x, x, a.ldx * S::es, rows, cols * S::es);
  } else {
    fetch<kWords>(S::at, smem, a.x, x, a.ldx * S::es, rows, cols * S::es);
  }
  if (CHANCE) {
    if (a.rand_step == 16 && inside) {
      constexpr int kStep = kThreads / kRandWords;
      const char* from = rnd0 + (tid / kRandWords) * a.ldr + (tid % kRandWords) * 16;
      const uint32_t to = zr::smem_u32(srand) + (tid / kRandWords) * kRandPitch + (tid % kRandWords) * 16;
#pragma unroll
      for (int i = 0; i < kRows / kStep; ++i) zr::copy16(to + rand_at(i * kStep), from + i * kStep * a.ldr);
    } else if (a.rand_step == 16) {
      fetch_by<kRandWords, 16>(rand_at, reinterpret_cast<char*>(srand), a.rand, rnd0, a.ldr, rows, cols);
    } else if (a.rand_step == 8) {
      fetch_by<kRandWords, 8>(rand_at, reinterpret_cast<char*>(srand), a.rand, rnd0, a.ldr, rows, cols);
    } else if (a.rand_step == 4) {
      fetch_by<kRandWords, 4>(rand_at, reinterpret_cast<char*>(srand), a.rand, rnd0, a.ldr, rows, cols);
    } else {
      fetch<kRandWords>(rand_at, reinterpret_cast<char*>(srand), a.rand, rnd0, a.ldr, rows, cols);
    }
  }
  zr::copies_done();
  __syncthreads();
  if (a.x_step < 8 || (CHANCE && a.rand_step < 4)) {
    if (a.x_step < 8) align<kWords>(S::at, smem, x, a.ldx * S::es);
    if (CHANCE && a.rand_step < 4) align<kRandWords>(rand_at, reinterpret_cast<char*>(srand), rnd0, a.ldr);
    __syncthreads();
  }

  // ---- by rows: a thread takes 32 neighbours of a row, a quad of lanes a row's four blocks
  if (a.q && pr < a.q_row_patches) {
    uint8_t* tile = a.q + ((pr >> 1) * a.q_tiles + (pc >> 1)) * zr::kMxTileBytes;
    const int tr = (int)(pr & 1) * kRows;  // the patch's first row in its tile
#pragma unroll 1
    for (int it = 0; it < 2; ++it) {
      const int task = tid + it * kThreads, r = task >> 2, b = task & 3;
      // the four 8-value words of the block in an order that differs between the lanes of a
      // quad, so that they read different banks: word (i + rot) % 4 comes i-th
      const int rot = DT == zr::DT_F32 ? b : (b & 2);
      const char* row = smem + S::at(r) + b * 32 * S::es;
      uint4 raw[4][S::es / 2];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int w = (i + rot) & 3;
#pragma unroll
        for (int h = 0; h < S::es / 2; ++h) {
          const uint4 u = *reinterpret_cast<const uint4*>(row + w * 8 * S::es + h * 16);
          raw[i][h] = u;
          m = amax_word<DT>(amax_word<DT>(amax_word<DT>(amax_word<DT>(m, u.x), u.y), u.z), u.w);
        }
      }
      // (of two 16-bit patterns the larger as whole numbers, with NaN on top)
      if (DT != zr::DT_F32) m = bits_of_half<DT>((m >> 16) > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu);
      const int byte = zr::mx_scale_byte<CHANCE>(m);
      uint32_t o[4];
      if (byte == 255) {
        o[0] = o[1] = o[2] = o[3] = 0;
      } else {
        const float inv = zr::mx_inverse(byte);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
          if (DT == zr::DT_F32) {
            const uint4 u = raw[i][0], w = raw[i][S::es / 2 - 1];
            const uint32_t f[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(f[j]);
          } else {
            zr::unpack8<DT>(raw[i][0], x);
          }
          uint32_t dither[8];
          if (CHANCE) {
            const uint2 r8 = *reinterpret_cast<const uint2*>(srand + rand_at(r) + b * 32 + ((i + rot) & 3) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) dither[j] = zr::mx_dither(j < 4 ? r8.x : r8.y, j & 3);
          }
          o[i] = codes_of<CHANCE>(x, inv, dither);
        }
      }
      if (rot & 1) {
        const uint32_t z = o[3];
        o[3] = o[2]; o[2] = o[1]; o[1] = o[0]; o[0] = z;
      }
      if (rot & 2) {
        uint32_t z = o[0];
        o[0] = o[2]; o[2] = z;
        z = o[1];
        o[1] = o[3]; o[3] = z;
      }
      const int j = (int)(pc & 1) * 4 + b;
      *reinterpret_cast<uint4*>(tile + zr::mx_chunk_at(tr + r, j)) = make_uint4(o[0], o[1], o[2], o[3]);
      const uint32_t bytes = lane_bytes<4>(byte);
      if (b == 0) *reinterpret_cast<uint32_t*>(tile + zr::mx_scale_at(tr + r, j)) = bytes;
    }
  }

  // ---- by columns: a thread takes 32 neighbours of one column (of two in 16 bits), a pair of
  // lanes a column's two blocks
  if (a.qt && pc < a.qt_col_patches) {
    uint8_t* tile = a.qt + (pc * a.qt_tiles + (pr >> 2)) * zr::kMxTileBytes;
    constexpr int kOwn = DT == zr::DT_F32 ? 1 : 2;
#pragma unroll 1
    for (int it = 0; it < 2 / kOwn; ++it) {
      const int task = tid + it * kThreads, c = (task >> 1) * kOwn, b = task & 1;
      const char* col = smem + S::at(b * 32) + c * S::es;
      uint32_t raw[32];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        raw[i] = *reinterpret_cast<const uint32_t*>(col + i * S::pitch);
        m = amax_word<DT>(m, raw[i]);
      }
      int byte[kOwn];
      float inv[kOwn];
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        byte[k] = zr::mx_scale_byte<CHANCE>(DT == zr::DT_F32 ? m : bits_of_half<DT>(k ? m >> 16 : m & 0xFFFFu));
        inv[k] = byte[k] == 255 ? 0.0f : zr::mx_inverse(byte[k]);
      }
      uint32_t o[kOwn][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t rnd[8];
        if (CHANCE) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // the random bytes of this thread's one or two columns
            const uint8_t* at = srand + rand_at(b * 32) + (i * 8 + j) * kRandPitch + c;
            rnd[j] = kOwn == 2 ? *reinterpret_cast<const uint16_t*>(at) : *at;
          }
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          float x[8];
          uint32_t dither[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t w = raw[i * 8 + j];
            x[j] = DT == zr::DT_F32    ? __uint_as_float(w)
                   : DT == zr::DT_BF16 ? __uint_as_float(k ? w & 0xFFFF0000u : w << 16)
                                       : zr::to_f32<DT>((uint16_t)(k ? w >> 16 : w));
            if (CHANCE) dither[j] = zr::mx_dither(rnd[j], k);
          }
          o[k][i] = codes_of<CHANCE>(x, inv[k], dither);
        }
      }
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int j = (int)(pr & 3) * 2 + b;
        const bool bad = byte[k] == 255;
        *reinterpret_cast<uint4*>(tile + zr::mx_chunk_at(c + k, j)) =
            bad ? make_uint4(0, 0, 0, 0) : make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        const uint32_t bytes = lane_bytes<2>(byte[k]);
        if (b == 0) *reinterpret_cast<uint16_t*>(tile + zr::mx_scale_at(c + k, j)) = (uint16_t)bytes;
      }
    }
  }
}

struct DequantArgs {
  const uint8_t* q;
  void* out;
  int64_t rows, cols, ld, tiles;  // tiles along the columns
};

constexpr int kDequantRows = 32, kRowsPerWarp = kDequantRows / (kDequantThreads / 32);

// A block takes 32 rows of a tile, a warp four of them at once (their loads in flight together), a
// lane eight values of a row. ALIGNED: the rows of out begin on 16-byte boundaries; others leave in
// whole aligned words, too, but for their ends: in 16 bits a lane's word from its own values and the
// next lane's; in 32, and at the matrix's last columns, by way of shared memory.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kDequantThreads) dequant_kernel(const __grid_constant__ DequantArgs a) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2, kRowBytes = zr::kMxCols * es;
  __shared__ __align__(16) char staging[ALIGNED ? 1 : kDequantThreads / 32][ALIGNED ? 16 : kRowBytes + 16];
  const int64_t t = blockIdx.x >> 2, rt = t / a.tiles, ct = t - rt * a.tiles;
  const uint8_t* tile = a.q + t * zr::kMxTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane >> 2;
  const int64_t c0 = ct * zr::kMxCols;
  const int n = (int)(a.cols - c0 < zr::kMxCols ? a.cols - c0 : zr::kMxCols);  // columns of this tile
  const int r0 = (int)(blockIdx.x & 3) * kDequantRows + warp;
  zr::wait_for_previous();
  zr::let_next_begin();
  uint32_t codes[kRowsPerWarp];
  int byte[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int r = r0 + i * (kDequantThreads / 32);
    codes[i] = *reinterpret_cast<const uint32_t*>(tile + zr::mx_chunk_at(r, j) + (lane & 3) * 4);
    byte[i] = tile[zr::mx_scale_at(r, j)];
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = rt * zr::kMxRows + r0 + i * (kDequantThreads / 32);
    if (row >= a.rows) return;
    float v[8];
    zr::mx_decode8(codes[i], v);
    const float s = zr::mx_scale_value(byte[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], s);
    uint4 w[es / 2];
    if constexpr (DT == zr::DT_F32) {
      w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      w[0] = zr::pack8<DT>(v);
    }
    char* out = static_cast<char*>(a.out) + (row * a.ld + c0) * es;
    if (ALIGNED) {
      if (lane * 8 + 8 <= n) {
#pragma unroll
        for (int k = 0; k < es / 2; ++k) zr::st_once(out + (lane * (es / 2) + k) * 16, w[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (lane * 8 + k < n) {
            if constexpr (DT == zr::DT_F32)
              reinterpret_cast<float*>(out)[lane * 8 + k] = v[k];
            else
              reinterpret_cast<uint16_t*>(out)[lane * 8 + k] = zr::from_f32<DT>(v[k]);
          }
      }
      continue;
    }
    const int lead = (int)(reinterpret_cast<uintptr_t>(out) & 15);
    if (DT != zr::DT_F32 && n == zr::kMxCols && lead != 0) {
      auto from_lane = [&](int l) {
        return make_uint4(__shfl_sync(0xFFFFFFFFu, w[0].x, l), __shfl_sync(0xFFFFFFFFu, w[0].y, l),
                          __shfl_sync(0xFFFFFFFFu, w[0].z, l), __shfl_sync(0xFFFFFFFFu, w[0].w, l));
      };
      const int skip = 16 - lead, head = skip / 2;  // what a lane leaves to the word of the one before it
      const uint4 next = from_lane((lane + 1) & 31);
      if (lane < 31) zr::st_once(out + skip + lane * 16, zr::shift16(w[0], next, (uint32_t)skip));
      // the row's first values up to a boundary and its last ones behind one, eight together: a lane each
      const uint4 end = from_lane(lane < head ? 0 : 31);
      const uint32_t pick = (lane & 4) ? ((lane & 2) ? end.w : end.z) : ((lane & 2) ? end.y : end.x);
      if (lane < 8)
        reinterpret_cast<uint16_t*>(out)[lane < head ? lane : zr::kMxCols - 8 + lane] =
            (uint16_t)(pick >> (16 * (lane & 1)));
      continue;
    }
    char* stage = staging[warp];
#pragma unroll
    for (int k = 0; k < es / 2; ++k) *reinterpret_cast<uint4*>(stage + (lane * (es / 2) + k) * 16) = w[k];
    __syncwarp();
    // the values before the first boundary, whole words from there, the values behind the last
    const int head = lead ? (16 - lead) / es < n ? (16 - lead) / es : n : 0;
    const int whole = (n - head) * es / 16, tail = n - head - whole * (16 / es);
    for (int k = lane; k < whole; k += 32) {
      const int from = head * es + k * 16;
      const uint4* at = reinterpret_cast<const uint4*>(stage + (from & ~15));
      zr::st_once(out + from, zr::shift16(at[0], at[1], (uint32_t)from & 15u));
    }
    const int one = lane < head ? lane : lane >= 16 && lane - 16 < tail ? n - tail + lane - 16 : -1;
    if (one >= 0) {
      if (es == 4)
        reinterpret_cast<uint32_t*>(out)[one] = reinterpret_cast<const uint32_t*>(stage)[one];
      else
        reinterpret_cast<uint16_t*>(out)[one] = reinterpret_cast<const uint16_t*>(stage)[one];
    }
    __syncwarp();
  }
}

template <int DT>
cudaError_t launch_dequant(const DequantArgs& a, int64_t blocks, bool aligned, cudaStream_t s) {
  return aligned ? zr::launch(dequant_kernel<DT, true>, blocks, kDequantThreads, 0, 1, true, s, a)
                 : zr::launch(dequant_kernel<DT, false>, blocks, kDequantThreads, 0, 1, true, s, a);
}

template <int DT, bool CHANCE>
zr_status launch_quant(const QuantArgs& a, int64_t patches, cudaStream_t s) {
  constexpr int smem = Shape<DT>::bytes + (CHANCE ? kRandBytes : 0);
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_mx4_quantize", (const void*)quant_kernel<DT, CHANCE>, smem)) return st;
  // Not early: its blocks would crowd onto the SMs that the launch before leaves room on (592 x 2789 x 1238 there
  // and back 26.2 us, 18.8 like this), and a product may read its weights before this one's end.
  cudaError_t e = zr::launch(quant_kernel<DT, CHANCE>, patches, kThreads, smem, 1, false, s, a);
  return e == cudaSuccess ? ZR_OK : fail(ZR_ERR_CUDA, "zr_mx4_quantize: launch failed: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" int64_t zr_mx4_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return -1;
  const int64_t down = zr::mx_tiles(rows, zr::kMxRows), over = zr::mx_tiles(cols, zr::kMxCols);
  if (over > 0 && down > INT64_MAX / zr::kMxTileBytes / over) return -1;
  return down * over * zr::kMxTileBytes;
}

extern "C" zr_status zr_mx4_quantize(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ldx,
                                     const uint8_t* rand, int64_t ldr, void* q, void* qt, void* stream) {
  zr::clear_error();
  zr::Range range("zr_mx4_quantize");
  if (!zr::dtype_ok(dt)) return fail(ZR_ERR_INVALID, "zr_mx4_quantize: bad dtype %d", (int)dt);
  if (rows < 0 || cols < 0) return fail(ZR_ERR_INVALID, "zr_mx4_quantize: negative size");
  if (ldx < cols || (rand && ldr < cols)) return fail(ZR_ERR_INVALID, "zr_mx4_quantize: a row stride is under cols");
  if (rows == 0 || cols == 0) return ZR_OK;
  if (!q && !qt) return fail(ZR_ERR_INVALID, "zr_mx4_quantize: neither q nor qt given");
  if (!x) return fail(ZR_ERR_INVALID, "zr_mx4_quantize: null x");
  if (!zr::aligned16(x) || !zr::aligned16(rand) || !zr::aligned16(q) || !zr::aligned16(qt))
    return fail(ZR_ERR_INVALID, "zr_mx4_quantize: a pointer is not 16-byte aligned");
  QuantArgs a{};
  a.x = x; a.rand = rand;
  a.q = static_cast<uint8_t*>(q); a.qt = static_cast<uint8_t*>(qt);
  a.rows = rows; a.cols = cols; a.ldx = ldx; a.ldr = ldr;
  auto step = [](int64_t stride) { return stride % 16 == 0 ? 16 : stride % 8 == 0 ? 8 : stride % 4 == 0 ? 4 : 1; };
  a.x_step = step(ldx * (dt == ZR_F32 ? 4 : 2));
  a.rand_step = step(ldr);
  a.q_tiles = zr::mx_tiles(cols, zr::kMxCols);
  a.qt_tiles = zr::mx_tiles(rows, zr::kMxCols);
  // patches to the end of both outputs' tiles: 128 rows by 256 columns of q, 128 columns by 256 rows for qt
  const int64_t row128 = 2 * zr::mx_tiles(rows, 128), col128 = zr::mx_tiles(cols, kCols);
  const int64_t row_patches = qt ? 4 * a.qt_tiles : row128;
  a.col_patches = q ? 2 * a.q_tiles : col128;
  if (row_patches > 0x7FFFFFFF / a.col_patches) return fail(ZR_ERR_UNSUPPORTED, "zr_mx4_quantize: matrix too large for one launch");
  const int64_t patches = row_patches * a.col_patches;
  a.q_row_patches = (int)row128;
  a.qt_col_patches = (int)col128;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rand) {
    if (dt == ZR_F16) return launch_quant<zr::DT_F16, true>(a, patches, s);
    if (dt == ZR_BF16) return launch_quant<zr::DT_BF16, true>(a, patches, s);
    return launch_quant<zr::DT_F32, true>(a, patches, s);
  }
  if (dt == ZR_F16) return launch_quant<zr::DT_F16, false>(a, patches, s);
  if (dt == ZR_BF16) return launch_quant<zr::DT_BF16, false>(a, patches, s);
  return launch_quant<zr::DT_F32, false>(a, patches, s);
}

extern "C" zr_status zr_mx4_dequantize(const void* q, int64_t rows, int64_t cols, void* out, zr_dtype dt, int64_t ld,
                                       void* stream) {
  zr::clear_error();
  zr::Range range("zr_mx4_dequantize");
  if (!zr::dtype_ok(dt)) return fail(ZR_ERR_INVALID, "zr_mx4_dequantize: bad dtype %d", (int)dt);
  if (rows < 0 || cols < 0) return fail(ZR_ERR_INVALID, "zr_mx4_dequantize: negative size");
  if (ld < cols) return fail(ZR_ERR_INVALID, "zr_mx4_dequantize: the row stride is under cols");
  if (rows == 0 || cols == 0) return ZR_OK;
  if (!q || !out) return fail(ZR_ERR_INVALID, "zr_mx4_dequantize: null pointer");
  if (!zr::aligned16(q) || !zr::aligned16(out))
    return fail(ZR_ERR_INVALID, "zr_mx4_dequantize: a pointer is not 16-byte aligned");
  DequantArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.out = out;
  a.rows = rows; a.cols = cols; a.ld = ld;
  a.tiles = zr::mx_tiles(cols, zr::kMxCols);
  const int64_t row_blocks = zr::mx_tiles(rows, zr::kMxRows) * (zr::kMxRows / kDequantRows);
  if (row_blocks > 0x7FFFFFFF / a.tiles)
    return fail(ZR_ERR_UNSUPPORTED, "zr_mx4_dequantize: matrix too large for one launch");
  const int64_t blocks = row_blocks * a.tiles;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool aligned = ld * (dt == ZR_F32 ? 4 : 2) % 16 == 0;
  const cudaError_t e = dt == ZR_F16    ? launch_dequant<zr::DT_F16>(a, blocks, aligned, s)
                        : dt == ZR_BF16 ? launch_dequant<zr::DT_BF16>(a, blocks, aligned, s)
                                        : launch_dequant<zr::DT_F32>(a, blocks, aligned, s);
  return e == cudaSuccess ? ZR_OK : fail(ZR_ERR_CUDA, "zr_mx4_dequantize: launch failed: %s", cudaGetErrorString(e));
}
