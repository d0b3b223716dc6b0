// Sums of a matrix's columns: a bias's gradient, the sum over tokens of its layer's output gradient.
//
// Each value is read once and the sums are small, so the matrix's read bounds it. A block takes a strip of
// columns and, in a cluster of C blocks, 1/C of the rows; a thread adds 16 bytes of each of its rows, and the
// parts are joined in shared memory, then between the cluster's blocks, in an order that the sizes decide.
// 8192 x 8192 bf16 in 23 us (5.8 TB/s; 82 with a test between a thread's eight loads), 8192 x 2048 in 6.3; rows off
// 16-byte boundaries, a value a thread, 8192 x 2049 in 10.8.
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

// LANES threads side by side take PER columns each.
template <int DT, int LANES, int PER, int C>
__global__ void __launch_bounds__(kThreads) column_kernel(const __grid_constant__ SumArgs a) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2, kCols = LANES * PER, kRows = kThreads / LANES, kOnce = 8;
  __shared__ float parts[kRows * kCols], sums[kCols];
  const int lane = threadIdx.x % LANES, r0 = threadIdx.x / LANES;
  zr::let_next_begin();
  zr::wait_for_previous();
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  const int64_t col0 = (int64_t)(blockIdx.x / C) * kCols, col = col0 + lane * PER;
  const int64_t share = (a.M + C - 1) / C, first = share * rank, end = first + share < a.M ? first + share : a.M;
  const int left = (int)(a.N - col < PER ? (a.N > col ? a.N - col : 0) : PER);
  const char* x = static_cast<const char*>(a.x) + col * es;
  float sum[PER] = {};
  auto add = [&](const float v[PER]) {
#pragma unroll
    for (int k = 0; k < PER; ++k) sum[k] = __fadd_rn(sum[k], v[k]);
  };
  auto open = [&](uint4 u) {
    float v[PER];
    if constexpr (PER == 8) {
      zr::unpack8<DT>(u, v);
    } else if constexpr (PER == 4) {
      v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
    }
    add(v);
  };
  const int64_t step = a.ld * es * kRows;
  const char* from = x + (first + r0) * a.ld * es;
  int64_t r = first + r0;
  if (PER > 1 && left == PER) {  // (not by the read-only path: the launch before may have written x since this one began)
    for (; r + (kOnce - 1) * kRows < end; r += kOnce * kRows, from += kOnce * step) {
      uint4 u[kOnce];
#pragma unroll
      for (int i = 0; i < kOnce; ++i) u[i] = zr::ld_row(from + i * step);
#pragma unroll
      for (int i = 0; i < kOnce; ++i) open(u[i]);
    }
    for (; r < end; r += kRows, from += step) open(zr::ld_row(from));
  } else if (left > 0) {
    for (; r + (kOnce - 1) * kRows < end; r += kOnce * kRows, from += kOnce * step) {
      float v[kOnce][PER];
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
#pragma unroll
        for (int k = 0; k < PER; ++k) v[i][k] = k < left ? zr::load1<DT>(from + i * step, k) : 0.0f;
#pragma unroll
      for (int i = 0; i < kOnce; ++i) add(v[i]);
    }
    for (; r < end; r += kRows, from += step) {
      float v[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) v[k] = k < left ? zr::load1<DT>(from, k) : 0.0f;
      add(v);
    }
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) parts[r0 * kCols + lane * PER + k] = sum[k];
  __syncthreads();
  // halves onto halves, down to one row
  for (int rows = kRows / 2; rows > 0; rows /= 2) {
    for (int i = threadIdx.x; i < rows * kCols; i += kThreads) parts[i] = __fadd_rn(parts[i], parts[i + rows * kCols]);
    __syncthreads();
  }
  if (threadIdx.x < kCols) sums[threadIdx.x] = parts[threadIdx.x];
  __syncthreads();
  if (C > 1) zr::cluster_sync();
  if (rank == 0 && threadIdx.x < kCols && col0 + threadIdx.x < a.N) {
    float s = sums[threadIdx.x];
#pragma unroll
    for (int r = 1; r < C; ++r)
      s = __fadd_rn(s, zr::cluster_load(zr::cluster_addr(zr::smem_u32(&sums[threadIdx.x]), r)));
    a.out[col0 + threadIdx.x] = s;
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
