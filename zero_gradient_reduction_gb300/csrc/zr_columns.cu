// Sums of a matrix's columns: a bias's gradient, the sum over tokens of its layer's output gradient.
//
// Each value is read once and the sums are small, so the matrix's read bounds it. A block takes a strip of
// columns and, in a cluster of C blocks, 1/C of the rows; a thread adds 16 bytes of each of its rows, and the
// parts are joined by the lanes of each warp, in shared memory, then between the cluster's blocks, in an order that
// the sizes decide. Eight rows are added in fp32, their sums in two words, the second what rounding has taken from the
// first, so that a sum is right to a few half units of fp32 whatever the number of rows: 8192 of bf16 in an rms of 2.5e-8, as if
// rounded once, of fp32 in 5.4e-8. The six additions, shared by two columns and eight rows, are hidden by the loads.
// 8192 x 8192 bf16 in 24.4 us from memory (5.5 TB/s; with one word 25.2), 8192 x 2048 in 8.2 (6.3 from L2); rows off
// 16-byte boundaries, a value a thread, 8192 x 2049 in 12.9.
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_device.cuh"
#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_nvtx.h"
#include "zr_rows.cuh"
#include "zr_tensor.cuh"

using zr::fail;

namespace {

constexpr int kThreads = 256;

struct SumArgs {
  const void* x;
  float* out;
  int64_t M, N, ld;
};

// Of one column, or of two with an instruction for both.
__device__ __forceinline__ float sum_of(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float less(float a, float b) { return __fsub_rn(a, b); }
__device__ __forceinline__ zr::Two sum_of(zr::Two a, zr::Two b) { return zr::add2(a, b); }
__device__ __forceinline__ zr::Two less(zr::Two a, zr::Two b) { return zr::fma2(b, zr::Two(-1.0f, -1.0f), a); }

template <class T>
__device__ __forceinline__ T nothing() {
  if constexpr (sizeof(T) == sizeof(float)) return 0.0f;
  else return T(0.0f, 0.0f);
}

// Sums in two words.
template <class T>
struct Sums {
  T value = nothing<T>(), rest = nothing<T>();
  __device__ void add(T b) {
    const T s = sum_of(value, b), t = less(s, value);
    rest = sum_of(rest, sum_of(less(value, less(s, t)), less(b, t)));
    value = s;
  }
  // Eight rows' values, added in three steps: the rows' number costs no accuracy.
  template <class Of>
  __device__ void add_eight(Of of) {
    add(sum_of(sum_of(sum_of(of(0), of(1)), sum_of(of(2), of(3))), sum_of(sum_of(of(4), of(5)), sum_of(of(6), of(7)))));
  }
};
// Columns 2 j and 2 j + 1 of a word.
template <int DT>
__device__ __forceinline__ zr::Two two_of(uint4 u, int j) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (DT == zr::DT_F32) return zr::Two(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  if constexpr (DT == zr::DT_BF16) return zr::Two(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  return zr::Two(zr::to_f32<zr::DT_F16>((uint16_t)w[j]), zr::to_f32<zr::DT_F16>((uint16_t)(w[j] >> 16)));
}

// A sum of another block of the cluster.
__device__ __forceinline__ zr::Pair cluster_pair(uint32_t addr) {
  zr::Pair p;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(p.value), "=f"(p.rest) : "r"(addr) : "memory");
  return p;
}

// LANES threads side by side take PER columns each.
template <int DT, int LANES, int PER, int C>
__global__ void __launch_bounds__(kThreads, PER == 4 ? 4 : 2) column_kernel(const __grid_constant__ SumArgs a) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2, kCols = LANES * PER, kRows = kThreads / LANES, kOnce = 8;
  // 16-bit values have their next rows on the way while these are added (70,001 x 512 bf16 in 24.7 us, 31 without), in 128
  // registers; fp32 has twice the blocks on an SM instead (8192 x 8192 in 44.3 us, 48 to 49 with rows ahead).
  constexpr bool kAhead = PER == 8;
  __shared__ __align__(16) zr::Pair parts[kThreads / 32][kCols], sums[kCols];
  const int lane = threadIdx.x % LANES, r0 = threadIdx.x / LANES;
  zr::let_next_begin();
  zr::wait_for_previous();
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  const int64_t col0 = (int64_t)(blockIdx.x / C) * kCols, col = col0 + lane * PER;
  const int64_t share = (a.M + C - 1) / C, first = share * rank, end = first + share < a.M ? first + share : a.M;
  const int left = (int)(a.N - col < PER ? (a.N > col ? a.N - col : 0) : PER);
  const char* x = static_cast<const char*>(a.x) + col * es;
  const int64_t step = a.ld * es * kRows;
  const char* from = x + (first + r0) * a.ld * es;
  int64_t r = first + r0;
  zr::Pair s[PER];
  if constexpr (PER > 1) {
    Sums<zr::Two> sum[PER / 2];
    if (left == PER) {
      // (not by the read-only path: the launch before may have written x since this one began)
      uint4 u[kAhead ? 2 : 1][kOnce];
      auto ask = [&](uint4 (&to)[kOnce]) {
#pragma unroll
        for (int i = 0; i < kOnce; ++i) to[i] = zr::ld_row(from + i * step);
        from += kOnce * step;
      };
      auto take = [&](const uint4 (&v)[kOnce]) {
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) sum[j].add_eight([&](int i) { return two_of<DT>(v[i], j); });
      };
      const int64_t rows = end - r, groups = rows > (kOnce - 1) * kRows ? (rows - (kOnce - 1) * kRows - 1) / (kOnce * kRows) + 1 : 0;
      r += groups * kOnce * kRows;
      if constexpr (kAhead) {
        if (groups > 0) ask(u[0]);
        for (int64_t g = groups; g > 0; g -= 2) {
          if (g > 1) ask(u[1]);
          take(u[0]);
          if (g > 2) ask(u[0]);
          if (g > 1) take(u[1]);
        }
      } else {
        for (int64_t g = groups; g > 0; --g) {
          ask(u[0]);
          take(u[0]);
        }
      }
      for (; r < end; r += kRows, from += step) {
        const uint4 v = zr::ld_row(from);
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) sum[j].add(two_of<DT>(v, j));
      }
    } else {
      auto two = [&](int i, int j) {
        return zr::Two(2 * j < left ? zr::load1<DT>(from + i * step, 2 * j) : 0.0f,
                       2 * j + 1 < left ? zr::load1<DT>(from + i * step, 2 * j + 1) : 0.0f);
      };
      for (; r + (kOnce - 1) * kRows < end; r += kOnce * kRows, from += kOnce * step)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) sum[j].add_eight([&](int i) { return two(i, j); });
      for (; r < end; r += kRows, from += step)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) sum[j].add(two(0, j));
    }
#pragma unroll
    for (int j = 0; j < PER / 2; ++j) {
      s[2 * j] = zr::Pair{sum[j].value.lo(), sum[j].rest.lo()};
      s[2 * j + 1] = zr::Pair{sum[j].value.hi(), sum[j].rest.hi()};
    }
  } else {
    Sums<float> sum;
    if (left > 0) {
      for (; r + (kOnce - 1) * kRows < end; r += kOnce * kRows, from += kOnce * step) {
        float v[kOnce];
#pragma unroll
        for (int i = 0; i < kOnce; ++i) v[i] = zr::load1<DT>(from + i * step, 0);
        sum.add_eight([&](int i) { return v[i]; });
      }
      for (; r < end; r += kRows, from += step) sum.add(zr::load1<DT>(from, 0));
    }
    s[0] = zr::Pair{sum.value, sum.rest};
  }
  // The lanes of a warp that have the same columns: each gives away one half of those that it has left and takes in
  // the other lane's part of the half that it keeps.
  int cols = PER, at = lane * PER;
#pragma unroll
  for (int bit = LANES; bit < 32; bit *= 2) {
    auto other = [&](zr::Pair p) {
      return zr::Pair{__shfl_xor_sync(0xFFFFFFFFu, p.value, bit), __shfl_xor_sync(0xFFFFFFFFu, p.rest, bit)};
    };
    const bool up = threadIdx.x & bit;
    if (cols == 1) {
      s[0] = zr::plus(s[0], other(s[0]));
    } else {
      cols /= 2;
#pragma unroll
      for (int k = 0; k < PER / 2; ++k)
        if (k < cols) s[k] = zr::plus(up ? s[k + cols] : s[k], other(up ? s[k] : s[k + cols]));
      at += up ? cols : 0;
    }
  }
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (k < cols) parts[threadIdx.x / 32][at + k] = s[k];
  __syncthreads();
  if (threadIdx.x < kCols) {
    zr::Pair w[kThreads / 32];
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) w[i] = parts[i][threadIdx.x];
#pragma unroll
    for (int n = kThreads / 64; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) w[i] = zr::plus(w[i], w[i + n]);
    sums[threadIdx.x] = w[0];
  }
  __syncwarp();
  if (C > 1) zr::cluster_sync();
  if (rank == 0 && threadIdx.x < kCols && col0 + threadIdx.x < a.N) {
    zr::Pair all = sums[threadIdx.x];
    zr::Pair p[C];
#pragma unroll
    for (int q = 1; q < C; ++q) p[q] = cluster_pair(zr::cluster_addr(zr::smem_u32(&sums[threadIdx.x]), q));
#pragma unroll
    for (int q = 1; q < C; ++q) all = zr::plus(all, p[q]);
    // (where the first word is infinite or no number the second says nothing)
    a.out[col0 + threadIdx.x] = all.value - all.value == 0.0f ? __fadd_rn(all.value, all.rest) : all.value;
  }
  __syncwarp();
  if (C > 1) zr::cluster_sync();  // a block's shared memory stays until the first has read it
}

template <int DT, int LANES, int PER>
cudaError_t launch(const SumArgs& a, int sms, cudaStream_t s) {
  const int64_t strips = (a.N - 1) / (LANES * PER) + 1;
  // as many blocks to a strip as keep all SMs busy and 64 rows each
  if (strips * 4 <= sms * 2 && a.M >= 8 * 64) return zr::launch(column_kernel<DT, LANES, PER, 8>, strips * 8, kThreads, 0, 8, true, s, a);
  if (strips <= sms * 2 && a.M >= 4 * 64) return zr::launch(column_kernel<DT, LANES, PER, 4>, strips * 4, kThreads, 0, 4, true, s, a);
  return zr::launch(column_kernel<DT, LANES, PER, 1>, strips, kThreads, 0, 1, true, s, a);
}

template <int DT>
cudaError_t launch(const SumArgs& a, bool whole, int sms, cudaStream_t s) {
  constexpr int per = DT == zr::DT_F32 ? 4 : 8;
  if (!whole) return launch<DT, 32, 1>(a, sms, s);
  // strips of 128 bytes of a row, or of 32 where those would be fewer than a cluster each to a third of the SMs
  return a.N > sms / 24 * 8 * per ? launch<DT, 8, per>(a, sms, s) : launch<DT, 2, per>(a, sms, s);
}

}  // namespace

extern "C" zr_status zr_column_sums(const void* x, zr_dtype dt, int64_t M, int64_t N, int64_t ldx, float* out,
                                    void* stream) {
  zr::clear_error();
  zr::Range range("zr_column_sums");
  if (!zr::dtype_ok(dt)) return fail(ZR_ERR_INVALID, "zr_column_sums: bad dtype %d", (int)dt);
  if (M < 0 || N < 0) return fail(ZR_ERR_INVALID, "zr_column_sums: negative size");
  if (ldx < N) return fail(ZR_ERR_INVALID, "zr_column_sums: the row stride is under the row");
  if (N == 0) return ZR_OK;
  if (!out || (M > 0 && !x)) return fail(ZR_ERR_INVALID, "zr_column_sums: null pointer");
  if (!zr::aligned16(x) || (reinterpret_cast<uintptr_t>(out) & 3))
    return fail(ZR_ERR_INVALID, "zr_column_sums: a pointer is not aligned");
  const int es = dt == ZR_F32 ? 4 : 2;
  if (N > (int64_t)1 << 33) return fail(ZR_ERR_UNSUPPORTED, "zr_column_sums: too many columns for one launch");
  const int sms = zr::sm_count("zr_column_sums");
  if (sms == 0) return ZR_ERR_CUDA;
  SumArgs a{x, out, M, N, ldx};
  const bool whole = ldx * es % 16 == 0 || M == 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == ZR_F16    ? launch<zr::DT_F16>(a, whole, sms, s)
                        : dt == ZR_BF16 ? launch<zr::DT_BF16>(a, whole, sms, s)
                                        : launch<zr::DT_F32>(a, whole, sms, s);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_column_sums: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}
