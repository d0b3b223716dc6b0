// The distillation loss against a teacher's top logits and its gradient, from one read of the
// student's logits.
//
// With p = softmax(teacher / tau) over a row's kept entries and q = softmax(z / tau) over the
// vocabulary, loss = w tau^2 sum_k p_k (log p_k - log q_id(k)) and dloss/dz = w tau (q - p). A row
// is read once into shared memory (of one block, or of a cluster that shares the row), its
// maximum, its sum of exponentials and its gradient come from there, and the gradient is written
// once. All arithmetic is fp32; sums are taken in an order that the sizes alone decide.
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_device.cuh"
#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_nvtx.h"
#include "zr_plan.h"
#include "zr_tensor.cuh"

using zr::fail;

namespace {

constexpr int kMaxThreads = 512;
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct DistillArgs {
  const void* z;
  const void* ids;
  const void* teacher;
  const float* weight;  // null: 1
  const float* scale;   // null: 1 (a plan's loss scale, in device memory)
  float* loss;
  void* grad;           // null: the loss alone
  int64_t T, V, ldz, ldg, ldk;
  int64_t share;        // columns of each block of a row's cluster
  int K, wide_ids, tdt;
  int room;             // 16-byte words of a row's share that shared memory holds
  float tau, grad_scale;
};

// Not the read-only path: the gradient may replace the logits.
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp; 2^-inf = 0
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DT>
struct Word {
  static constexpr int per = DT == zr::DT_F32 ? 4 : 8;
  __device__ static void open(uint4 u, float f[per]) {
    if constexpr (DT == zr::DT_F32) {
      f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
      f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    } else {
      zr::unpack8<DT>(u, f);
    }
  }
  __device__ static uint4 close(const float f[per]) {
    if constexpr (DT == zr::DT_F32)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return zr::pack8<DT>(f);
  }
};

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (DT == zr::DT_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = zr::from_f32<DT == zr::DT_F32 ? zr::DT_BF16 : DT>(v);
}

struct Sum {
  __device__ static float of(float a, float b) { return __fadd_rn(a, b); }
};
struct Max {
  __device__ static float of(float a, float b) { return fmaxf(a, b); }
};

// The block's sum or maximum in every thread; `slots`: 32 floats that no one else uses meanwhile.
template <class OP>
__device__ float block_all(float v, float none, float* slots) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = OP::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? slots[threadIdx.x & 31] : none;
#pragma unroll
  for (int o = 16; o; o >>= 1) v = OP::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  return v;
}

// A row is handled in the 16-byte words of memory that hold it: word 0 begins at the boundary at
// or before its first value, so every load is aligned whatever the row stride; `lead` values of
// word 0 belong to the row before, and the last word may end past the row.
template <int DT, int C>
__global__ void __launch_bounds__(kMaxThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  using W = Word<DT>;
  constexpr int per = W::per, es = 16 / per;
  extern __shared__ __align__(16) char smem[];
  uint4* words = reinterpret_cast<uint4*>(smem);
  float* sp = reinterpret_cast<float*>(words + a.room);            // p of each entry
  int64_t* sid = reinterpret_cast<int64_t*>(sp + ((a.K + 1) & ~1));  // its column, or -1
  float* own = reinterpret_cast<float*>(sid + a.K);                // the gradient at that column
  float* slots = own + a.K;                                        // 32
  float* mine = slots + 32;                                        // what the cluster reads: max, sum, loss
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int64_t row = blockIdx.x / C;
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  const int64_t v0 = rank * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;  // may be empty: v0 >= v1
  const int64_t n = v1 > v0 ? v1 - v0 : 0;

  const float w = a.weight ? a.weight[row] : 1.0f;
  const float c = __fdiv_rn(kLog2E, a.tau);

  // ---- the teacher's entries: p over the kept ones
  bool some = false, beyond = false;
  float t_max = -INFINITY;
  if (w != 0.0f)
    for (int k = tid; k < a.K; k += nthr) {
      const int64_t at = row * a.ldk + k;
      const int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
      const float t = a.tdt == zr::DT_F32    ? zr::load1<zr::DT_F32>(a.teacher, at)
                      : a.tdt == zr::DT_BF16 ? zr::load1<zr::DT_BF16>(a.teacher, at)
                                             : zr::load1<zr::DT_F16>(a.teacher, at);
      sid[k] = id;
      sp[k] = t;
      some |= id >= 0 && !(t == -INFINITY);  // a masked entry is none
      beyond |= id >= a.V;
      if (id >= 0) t_max = fmaxf(t_max, t);
    }
  some = __syncthreads_or(some);
  void* grad = a.grad ? static_cast<char*>(a.grad) + (row * a.ldg + v0) * es : nullptr;
  const char* zrow = static_cast<const char*>(a.z) + (row * a.ldz + v0) * es;
  const int lead = (int)(reinterpret_cast<uintptr_t>(zrow) & 15) / es;
  const uint4* zw = reinterpret_cast<const uint4*>(zrow - lead * es);
  const int64_t nw = n > 0 ? (lead + n + per - 1) / per : 0;
  // the gradient's words are the logits' words, shifted: stored whole only where they coincide
  const bool same = grad && ((reinterpret_cast<uintptr_t>(grad) & 15) / es) == (uintptr_t)lead;

  if (!some) {  // no weight, or nothing kept: no loss and no gradient (uniform over the cluster)
    if (rank == 0 && tid == 0) a.loss[row] = 0.0f;
    if (grad)
      for (int64_t j = tid; j < nw; j += nthr) {
        const int64_t i0 = j * per - lead;
        if (same && i0 >= 0 && i0 + per <= n)
          *reinterpret_cast<uint4*>(static_cast<char*>(grad) + i0 * es) = make_uint4(0, 0, 0, 0);
        else
          for (int i = 0; i < per; ++i)
            if (i0 + i >= 0 && i0 + i < n) store1<DT>(grad, i0 + i, 0.0f);
      }
    return;
  }
  beyond = __syncthreads_or(beyond);

  // ---- the row into shared memory, and its maximum
  float m = -INFINITY;
  auto value_max = [&](int64_t j, uint4 u) {
    float f[per];
    W::open(u, f);
    const int64_t i0 = j * per - lead;
    if (i0 >= 0 && i0 + per <= n) {
#pragma unroll
      for (int i = 0; i < per; ++i) m = fmaxf(m, f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < per; ++i)
        if (i0 + i >= 0 && i0 + i < n) m = fmaxf(m, f[i]);
    }
  };
  {
    constexpr int kAhead = 8;
    int64_t j = tid;
    for (; j + (kAhead - 1) * nthr < nw; j += kAhead * nthr) {
      uint4 u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) u[i] = ld_row(zw + j + i * nthr);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (j + i * nthr < a.room) words[j + i * nthr] = u[i];
        value_max(j + i * nthr, u[i]);
      }
    }
    for (; j < nw; j += nthr) {
      const uint4 u = ld_row(zw + j);
      if (j < a.room) words[j] = u;
      value_max(j, u);
    }
  }
  auto word = [&](int64_t j) { return j < a.room ? words[j] : ld_row(zw + j); };
  t_max = block_all<Max>(t_max, -INFINITY, slots);
  float p_sum = 0.0f;
  for (int k = tid; k < a.K; k += nthr) {
    // an entry of -inf has p = 0; +inf or NaN leaves every p not a number
    const float e = sid[k] >= 0 ? exp2_fast((sp[k] - t_max) * c) : 0.0f;
    p_sum += e;
  }
  p_sum = block_all<Sum>(p_sum, 0.0f, slots);
  m = block_all<Max>(m, -INFINITY, slots);

  // ---- sum of 2^(z c - m c). The rounding of m c multiplies every term by the same factor, which
  // cancels in q and in log q.
  float mc = m == -INFINITY ? 0.0f : __fmul_rn(m, c);  // all masked so far: the terms are 0, or NaN where z is
  float sum = 0.0f;
  for (int64_t j = tid; j < nw; j += nthr) {
    float f[per];
    W::open(word(j), f);
    const int64_t i0 = j * per - lead;
    float part = 0.0f;
    if (i0 >= 0 && i0 + per <= n) {
#pragma unroll
      for (int i = 0; i < per; ++i) part = __fadd_rn(part, exp2_fast(__fmaf_rn(f[i], c, -mc)));
    } else {
#pragma unroll
      for (int i = 0; i < per; ++i)
        if (i0 + i >= 0 && i0 + i < n) part = __fadd_rn(part, exp2_fast(__fmaf_rn(f[i], c, -mc)));
    }
    sum = __fadd_rn(sum, part);
  }
  sum = block_all<Sum>(sum, 0.0f, slots);
  if (C > 1) {
    if (tid == 0) {
      mine[0] = m;
      mine[1] = sum;
    }
    __syncwarp();
    zr::cluster_sync();
    const uint32_t at = zr::smem_u32(mine);
    float ms[C], all = -INFINITY;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      ms[r] = zr::cluster_load(zr::cluster_addr(at, r));
      all = fmaxf(all, ms[r]);
    }
    mc = all == -INFINITY ? 0.0f : __fmul_rn(all, c);
    sum = 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const float s = zr::cluster_load(zr::cluster_addr(at + 4, r));
      sum = __fadd_rn(sum, ms[r] == -INFINITY ? s : __fmul_rn(s, exp2_fast(__fmul_rn(ms[r], c) - mc)));
    }
  }
  if (beyond) sum = NAN;  // an entry past the vocabulary: the row says so in its loss and its gradient

  // ---- the loss, by the entries in this block's columns; p stays in shared memory
  const float log_q = log2f(sum), log_p = log2f(p_sum);
  float loss = 0.0f;
  for (int k = tid; k < a.K; k += nthr) {
    const int64_t id = sid[k];
    const float t = (sp[k] - t_max) * c;
    const float p = id >= 0 ? __fdiv_rn(exp2_fast(t), p_sum) : 0.0f;
    sp[k] = p;
    if (id >= v0 && id < v1 && !(p == 0.0f)) {
      const int64_t i = lead + (id - v0), j = i / per;
      const float z = j < a.room ? zr::load1<DT>(smem, i) : zr::load1<DT>(zw, i);
      loss += p * ((t - log_p) - (__fmaf_rn(z, c, -mc) - log_q)) * kLn2;
    }
  }
  if (beyond) loss = NAN;
  loss = block_all<Sum>(loss, 0.0f, slots);  // and every p is written

  // ---- the gradient
  if (grad) {
    const float scale = a.scale ? __fmul_rn(a.grad_scale, *a.scale) : a.grad_scale;
    const float f = __fmul_rn(w, __fmul_rn(a.tau, scale));
    const float fq = __fdiv_rn(f, sum);
    // the entries' own columns first, from the logits as they were; stored behind the others
    for (int k = tid; k < a.K; k += nthr) {
      const int64_t id = sid[k];
      if (!(id >= v0 && id < v1)) continue;
      float p = 0.0f;
      for (int i = 0; i < a.K; ++i)
        if (sid[i] == id) p += sp[i];  // an id may stand twice: each of its entries finds the same sum
      const int64_t i = lead + (id - v0), j = i / per;
      const float z = j < a.room ? zr::load1<DT>(smem, i) : zr::load1<DT>(zw, i);
      own[k] = __fmul_rn(f, __fdiv_rn(exp2_fast(__fmaf_rn(z, c, -mc)), sum) - p);
    }
    __syncthreads();
    for (int64_t j = tid; j < nw; j += nthr) {
      float v[per];
      W::open(word(j), v);
#pragma unroll
      for (int i = 0; i < per; ++i) v[i] = __fmul_rn(exp2_fast(__fmaf_rn(v[i], c, -mc)), fq);
      const int64_t i0 = j * per - lead;
      if (same && i0 >= 0 && i0 + per <= n) {
        zr::st_once(static_cast<char*>(grad) + i0 * es, W::close(v));
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i)
          if (i0 + i >= 0 && i0 + i < n) store1<DT>(grad, i0 + i, v[i]);
      }
    }
    __syncthreads();
    for (int k = tid; k < a.K; k += nthr)
      if (sid[k] >= v0 && sid[k] < v1) store1<DT>(grad, sid[k] - v0, own[k]);
  }
  loss = __fmul_rn(loss, __fmul_rn(w, __fmul_rn(a.tau, a.tau)));
  if (C > 1) {
    if (tid == 0) mine[2] = loss;
    __syncwarp();
    zr::cluster_sync();
    if (rank == 0 && tid == 0) {
      loss = 0.0f;
#pragma unroll
      for (int r = 0; r < C; ++r) loss += zr::cluster_load(zr::cluster_addr(zr::smem_u32(mine + 2), r));
      a.loss[row] = loss;
    }
    __syncwarp();
    zr::cluster_sync();  // a block's shared memory stays until rank 0 has read it
  } else if (tid == 0) {
    a.loss[row] = loss;
  }
}

template <int DT, int C>
zr_status launch(const DistillArgs& a, int threads, int smem, cudaStream_t s) {
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_distill_topk", (const void*)distill_kernel<DT, C>, zr::kSmemMost)) return st;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(a.T * C));
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {C, 1, 1};
  c.attrs = &at;
  c.numAttrs = C > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&c, distill_kernel<DT, C>, a);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_distill_topk: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}

template <int DT>
zr_status launch_split(const DistillArgs& a, int split, int threads, int smem, cudaStream_t s) {
  if (split == 8) return launch<DT, 8>(a, threads, smem, s);
  if (split == 4) return launch<DT, 4>(a, threads, smem, s);
  if (split == 2) return launch<DT, 2>(a, threads, smem, s);
  return launch<DT, 1>(a, threads, smem, s);
}

}  // namespace

extern "C" zr_status zr_distill_topk(const void* logits, zr_dtype dt, int64_t T, int64_t V, int64_t ldz,
                                     const void* ids, int ids64, const void* teacher, zr_dtype teacher_dt, int K,
                                     int64_t ldk, const float* weight, float temperature, float grad_scale,
                                     const zr_plan* plan, float* loss, void* grad, int64_t ldg, void* stream) {
  zr::clear_error();
  zr::Range range("zr_distill_topk");
  if (!zr::dtype_ok(dt) || !zr::dtype_ok(teacher_dt)) return fail(ZR_ERR_INVALID, "zr_distill_topk: bad dtype");
  if (T < 0 || V < 1) return fail(ZR_ERR_INVALID, "zr_distill_topk: T must be >= 0 and V >= 1");
  if (K < 1 || K > ZR_DISTILL_MAX_TOP)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: K=%d outside [1, %d]", K, ZR_DISTILL_MAX_TOP);
  if (ldz < V || ldk < K || (grad && ldg < V)) return fail(ZR_ERR_INVALID, "zr_distill_topk: a row stride is under the row");
  if (!(temperature > 0.0f) || temperature > 1e6f || temperature < 1e-6f)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: temperature must lie in [1e-6, 1e6]");
  if (!(grad_scale == grad_scale) || grad_scale - grad_scale != 0.0f)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: grad_scale is not finite");
  if (T == 0) return ZR_OK;
  if (!logits || !ids || !teacher || !loss) return fail(ZR_ERR_INVALID, "zr_distill_topk: null pointer");
  if (!zr::aligned16(logits) || !zr::aligned16(ids) || !zr::aligned16(teacher) || !zr::aligned16(weight) ||
      !zr::aligned16(loss) || !zr::aligned16(grad))
    return fail(ZR_ERR_INVALID, "zr_distill_topk: a pointer is not 16-byte aligned");
  const int es = dt == ZR_F32 ? 4 : 2;
  const int64_t z_bytes = ((T - 1) * ldz + V) * es, g_bytes = ((T - 1) * ldg + V) * es;
  const char *zb = static_cast<const char*>(logits), *gb = static_cast<const char*>(grad);
  if (grad && !(gb == zb && ldg == ldz) && gb < zb + z_bytes && zb < gb + g_bytes)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: grad overlaps the logits without being them");
  const int sms = zr::sm_count("zr_distill_topk");
  if (sms == 0) return ZR_ERR_CUDA;
  DistillArgs a{};
  a.z = logits; a.ids = ids; a.teacher = teacher; a.weight = weight;
  a.scale = plan ? &plan->ctrl_dev->scale : nullptr;
  a.loss = loss; a.grad = grad;
  a.T = T; a.V = V; a.ldz = ldz; a.ldg = ldg; a.ldk = ldk;
  a.K = K; a.wide_ids = ids64; a.tdt = (int)teacher_dt;
  a.tau = temperature; a.grad_scale = grad_scale;
  // A row goes to one block where two rows fit an SM's shared memory and there are rows for every
  // SM; longer rows, or few of them, are shared by a cluster.
  const int fixed = ((K + 1) & ~1) * 4 + K * 12 + 36 * 4;
  const int64_t half = zr::kSmemMost / 2 - 1024 - fixed;
  int split = 1;
  while (split < 8 && ((V / split) * es > half || (T * split <= sms && V / split >= 4096))) split *= 2;
  if (T > 0x7FFFFFFF / split) return fail(ZR_ERR_UNSUPPORTED, "zr_distill_topk: too many rows for one launch");
  const int64_t unit = 16 / es;
  a.share = (V + split * unit - 1) / (split * unit) * unit;
  int64_t room = a.share / unit + 1;  // one more word where the row does not begin on a boundary
  const int64_t most = (zr::kSmemMost - fixed) / 16;
  a.room = (int)(room < most ? room : most);  // what does not fit is read again
  int threads = 64;
  while (threads < kMaxThreads && threads * 4 < room) threads *= 2;
  const int smem = a.room * 16 + fixed;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == ZR_F16) return launch_split<zr::DT_F16>(a, split, threads, smem, s);
  if (dt == ZR_BF16) return launch_split<zr::DT_BF16>(a, split, threads, smem, s);
  return launch_split<zr::DT_F32>(a, split, threads, smem, s);
}
