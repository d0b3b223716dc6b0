// The loss of pairs of sequences by their log-probability ratios, and its gradient.
//
// A sequence's reward is beta times the sum of logp - ref over its scored tokens; a pair's margin m is the
// chosen one's less the rejected one's, its loss -w ((1 - l) log s(m) + l log s(-m)) with the logistic s. The
// gradient of a row of it is f (1[v = a] - q_v), f = -+ w beta ((1 - l) s(-m) - l s(m)): it is known once all
// rows of the pair have been summed.
//
// So the logits are read twice and the gradient written once, by three launches that overlap at their ends: the
// rows' sums (139 us at 8192 x 50304 bf16), the pairs' (a block each, in the shadow of the others), the
// gradients (234 us). 373 us of the 366 that three passes take at a copy's rate; with a quarter of the rows not
// scored 321. Pairs are too long to stay on the chip between the two (a row is 100 KB, a pair hundreds of
// them); gradients that follow their pair's sums in one launch, from L2, were slower (409 us: each row's ticket,
// fence and arrival cost more than its second read from memory). The last rows' gradients come first, their
// logits are in L2 still. 61 rows of one pair: 10.8 us, three launches' latencies.
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_device.cuh"
#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_nvtx.h"
#include "zr_plan.h"
#include "zr_rows.cuh"
#include "zr_tensor.cuh"

using zr::fail;
using zr::Part;

namespace {

// What is kept of a scored row between its sum and its gradient.
struct __align__(16) RowSum {
  float m, sum;  // the largest logit; of the terms relative to it
  float others;  // 1 - q at the chosen token
  float unused;
};

struct PreferenceArgs {
  const void* z;
  const void* ids;
  const void* starts;
  const float* ref_logp;
  const float* weight;      // null: 1
  const float* loss_scale;  // null: 1 (a plan's, in device memory)
  float* loss;
  float* rewards;  // null: not wanted
  void* grad;      // null: the loss alone
  RowSum* sums;    // of each row
  float* ratio;    // logp - ref of each row, 0 where it is not scored
  float* slope;    // dloss/dlogp / tau of each sequence's rows, scaled
  int64_t T, V, ldz, ldg, share;
  int sequences, split;
  int wide_ids, wide_starts;
  zr::Scale scale;
  float beta, smoothing, grad_scale;
};

// The sequence that holds a row, -1 for none: the last that begins at or before it, by all lanes of a warp
// together, 32 looks at a time. Ends for starts in any order.
__device__ __forceinline__ int sequence_of(const PreferenceArgs& a, int64_t row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.sequences + 1;  // so many starts lie at or before the row
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const bool before = i < hi && zr::id_at(a.starts, a.wide_starts, i) <= row;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, before));
    hi = min(hi, lo + (n + 1) * step - 1);
    lo = min(lo + n * step, hi);
  }
  return lo == 0 || lo > a.sequences ? -1 : lo - 1;
}
__device__ __forceinline__ bool has_weight(const PreferenceArgs& a, int sequence) {
  return !a.weight || a.weight[sequence >> 1] != 0.0f;
}

// ---- each scored row's sum
template <int DT, int C>
__global__ void __launch_bounds__(384, 4) score_kernel(const __grid_constant__ PreferenceArgs a) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2;
  __shared__ zr::Parts sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / C;
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  if (C > 1) zr::cluster_arrived();
  zr::wait_for_previous();
  zr::let_next_begin();  // what begins from here on may read what was there before this call
  const int64_t id = zr::id_at(a.ids, a.wide_ids, row);
  const int sequence = sequence_of(a, row);
  if (id < 0 || sequence < 0 || !has_weight(a, sequence)) {
    if (C > 1) zr::cluster_wait();
    if (rank == 0 && tid == 0) a.ratio[row] = 0.0f;
    return;
  }
  const int64_t v0 = rank * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;
  const int n = v1 > v0 ? (int)(v1 - v0) : 0;
  const char* whole = static_cast<const char*>(a.z) + row * a.ldz * es;
  const float z_chosen = id < a.V ? zr::load1<DT>(whole, id) : 0.0f;
  const char* part = whole + v0 * es;
  const zr::RowWords<DT> words(part, n, tid);
  const Part mine =
      zr::read_part<DT, true, false>(words, part, id >= v0 && id < v1 ? (int)(id - v0) : -1, a.scale, tid, blockDim.x);
  Part rest = zr::join_all<false, C>(mine, a.scale, sh, rank);
  if (rank == 0 && tid == 0) {
    rest = zr::rebased<false>(rest, fmaxf(rest.m, z_chosen), a.scale);
    const zr::Base base(rest.m, a.scale);
    const float sum = __fadd_rn(rest.sum, zr::exp2_fast(base.exponent<true>(z_chosen, a.scale)));
    const zr::Pair logp = zr::log_chosen<true>(z_chosen, rest.sum, base, a.scale);
    a.ratio[row] = id < a.V ? (logp.value - a.ref_logp[row]) + logp.rest : NAN;
    a.sums[row] = RowSum{rest.m, sum, __fdiv_rn(rest.sum, sum), 0.0f};
  }
}

// ---- each pair's rewards, loss and slope: a block to a pair
// Sums in two words of 32 bits: a sequence's thousands of ratios would lose to one, and 64 bits are slow here (8 us a
// pair of 512 rows, most of them in a few dozen additions).
__device__ __forceinline__ zr::Pair across(zr::Pair a, int lanes) {
  return zr::plus(a, zr::Pair{__shfl_xor_sync(0xFFFFFFFFu, a.value, lanes), __shfl_xor_sync(0xFFFFFFFFu, a.rest, lanes)});
}
constexpr int kPairThreads = 256;
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ PreferenceArgs a) {
  __shared__ zr::Pair of_warp[2][kPairThreads / 32];
  const int pair = blockIdx.x, tid = threadIdx.x;
  zr::let_next_begin();
  int64_t at[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) at[i] = zr::id_at(a.starts, a.wide_starts, 2 * (int64_t)pair + i);
  const bool sound = at[0] >= 0 && at[0] <= at[1] && at[1] <= at[2] && at[2] <= a.T;
  zr::Pair sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
  zr::wait_for_previous();
  if (sound) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll 4
      for (int64_t r = at[i] + tid; r < at[i + 1]; r += kPairThreads) sum[i] = zr::plus(sum[i], zr::Pair{a.ratio[r], 0.0f});
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[i] = across(sum[i], o);
    if ((tid & 31) == 0) of_warp[i][tid >> 5] = sum[i];
  }
  __syncthreads();
  if (tid >= 32) return;
  const float w = a.weight ? a.weight[pair] : 1.0f;
  float reward[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    zr::Pair s = tid < kPairThreads / 32 ? of_warp[i][tid] : zr::Pair{0.0f, 0.0f};
#pragma unroll
    for (int o = kPairThreads / 64; o; o >>= 1) s = across(s, o);
    // (where one is infinite or no number so is the first word, and the second says nothing)
    const float whole = s.value - s.value == 0.0f ? __fmaf_rn(a.beta, s.rest, __fmul_rn(a.beta, s.value)) : __fmul_rn(a.beta, s.value);
    reward[i] = w == 0.0f ? 0.0f : sound ? whole : NAN;  // (a pair that does not count says nothing of its starts either)
  }
  if (tid != 0) return;
  if (a.rewards) a.rewards[2 * pair] = reward[0], a.rewards[2 * pair + 1] = reward[1];
  const float m = reward[0] - reward[1];
  // the logistic function on both sides, and the loss -log s(m) + l m = log(1 + e^-|m|) + |m| times l, or 1 - l where m < 0:
  // nothing cancels, and a share of nothing is nothing where the margin is infinite
  const float e = expf(-fabsf(m)), small = __fdiv_rn(e, 1.0f + e), large = __fdiv_rn(1.0f, 1.0f + e);
  const float up = m >= 0.0f ? large : small, down = m >= 0.0f ? small : large;
  const float share = m >= 0.0f ? a.smoothing : 1.0f - a.smoothing;
  const float value = log1pf(e) + (share > 0.0f ? __fmul_rn(share, fabsf(m)) : 0.0f);
  const float scale = a.loss_scale ? __fmul_rn(a.grad_scale, *a.loss_scale) : a.grad_scale;
  a.loss[pair] = w == 0.0f ? 0.0f : __fmul_rn(w, value);
  const float f = __fmul_rn(__fmul_rn(w, a.beta),
                            __fmul_rn(__fdiv_rn(scale, a.scale.tau), (1.0f - a.smoothing) * down - a.smoothing * up));
  a.slope[2 * pair] = -f;
  a.slope[2 * pair + 1] = f;
}

// ---- each row's gradient: the last rows first, which were summed last and are in L2 still. A block begins while the
// pairs are summed up and asks for its first words before it waits for them.
template <int DT>
__global__ void __launch_bounds__(384) gradient_kernel(const __grid_constant__ PreferenceArgs a) {
  using W = zr::Word<DT>;
  constexpr int per = W::per, es = 16 / per, kOnce = 4;
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int64_t place = blockIdx.x / a.split, row = a.T - 1 - place;
  const int64_t v0 = (blockIdx.x - place * a.split) * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;
  const int n = v1 > v0 ? (int)(v1 - v0) : 0;
  const char* zrow = static_cast<const char*>(a.z) + (row * a.ldz + v0) * es;
  char* grad = static_cast<char*>(a.grad) + (row * a.ldg + v0) * es;
  const zr::RowWords<DT> r(zrow, n, tid);
  uint4 u[kOnce];
  auto ask = [&](int j) {
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
      if (j + i * nthr < r.last) u[i] = zr::ld_row(r.words + j + i * nthr);
  };
  const int64_t id = zr::id_at(a.ids, a.wide_ids, row);
  const int sequence = sequence_of(a, row);
  const bool live = id >= 0 && sequence >= 0 && has_weight(a, sequence);
  if (live) ask(r.first + tid);
  zr::wait_for_previous();
  if (sequence < 0) return;  // left as it is
  // the gradient's words are the logits' words, shifted: stored whole only where they coincide
  const bool same = (int)(reinterpret_cast<uintptr_t>(grad) & 15) / es == r.lead;
  auto store = [&](int j, const float v[per]) {
    char* to = grad + (int64_t)(j * per - r.lead) * es;
    if (same) {
      zr::st_once(to, W::close(v));
    } else {
#pragma unroll
      for (int i = 0; i < per; ++i) zr::store1<DT>(to, i, v[i]);
    }
  };
  if (!live) {
    const float zeros[per] = {};
    for (int j = r.first + tid; j < r.last; j += nthr) store(j, zeros);
    if (r.single >= 0) zr::store1<DT>(grad, r.single, 0.0f);
    return;
  }
  const float f = a.slope[sequence];
  const RowSum row_sum = a.sums[row];
  const zr::Base base(row_sum.m, a.scale);
  const float by = -__fdiv_rn(f, row_sum.sum), own = __fmul_rn(f, row_sum.others);
  const int chosen = id >= v0 && id < v1 ? (int)(id - v0) : -1;
  const int hole = chosen < 0 ? -1 : (r.lead + chosen) / per, at = (r.lead + chosen) % per;
  const zr::Exponents<false> exponents(base, a.scale);
  const zr::Two by2(by, by);
  for (int j = r.first + tid; j < r.last; j += kOnce * nthr) {
    if (j != r.first + tid) ask(j);
#pragma unroll
    for (int i = 0; i < kOnce; ++i) {
      if (j + i * nthr >= r.last) break;
      float v[per];
      W::open(u[i], v);
      if (base.whole) {
#pragma unroll
        for (int k = 0; k < per; k += 2) {
          const zr::Two e = exponents.of(v[k], v[k + 1]);
          const zr::Two y = zr::mul2(zr::Two(zr::exp2_fast(e.lo()), zr::exp2_fast(e.hi())), by2);
          v[k] = y.lo();
          v[k + 1] = y.hi();
        }
      } else {
#pragma unroll
        for (int k = 0; k < per; ++k) v[k] = __fmul_rn(zr::exp2_fast(base.exponent<false>(v[k], a.scale)), by);
      }
      if (j + i * nthr == hole) {
#pragma unroll
        for (int k = 0; k < per; ++k)
          if (k == at) v[k] = own;
      }
      store(j + i * nthr, v);
    }
  }
  if (r.single >= 0) {
    const float z = zr::load1<DT>(zrow, r.single);
    zr::store1<DT>(grad, r.single,
                   r.single == chosen ? own : __fmul_rn(zr::exp2_fast(base.exponent<false>(z, a.scale)), by));
  }
}

template <int DT>
zr_status launch(PreferenceArgs& a, int sms, cudaStream_t s) {
  const zr::RowShape r = zr::streamed_rows(a.T, a.V, DT == zr::DT_F32 ? 4 : 2, sms);
  a.share = r.share;
  a.split = r.split;
  cudaError_t e = cudaSuccess;
  if (a.T > 0)
    e = r.split == 8   ? zr::launch(score_kernel<DT, 8>, a.T * 8, r.threads, 0, 8, true, s, a)
        : r.split == 4 ? zr::launch(score_kernel<DT, 4>, a.T * 4, r.threads, 0, 4, true, s, a)
        : r.split == 2 ? zr::launch(score_kernel<DT, 2>, a.T * 2, r.threads, 0, 2, true, s, a)
                       : zr::launch(score_kernel<DT, 1>, a.T, r.threads, 0, 1, true, s, a);
  // (behind a call's own sums it begins early: what it reads before it waits for them was there before the call)
  if (e == cudaSuccess) e = zr::launch(pair_kernel, a.sequences / 2, kPairThreads, 0, 1, a.T > 0, s, a);
  if (e == cudaSuccess && a.grad && a.T > 0)
    e = zr::launch(gradient_kernel<DT>, a.T * r.split, r.threads, 0, 1, true, s, a);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_preference_loss: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}

constexpr int64_t kMostRows = 0x7FFFFFFF / 8, kMostPairs = 1 << 28;

}  // namespace

extern "C" int64_t zr_preference_bytes(int64_t T, int64_t pairs) {
  if (T < 0 || pairs < 0 || T > kMostRows || pairs > kMostPairs) return -1;
  return T * 16 + (T + 2 * pairs + 3) / 4 * 16;
}

extern "C" zr_status zr_preference_loss(const void* logits, zr_dtype dt, int64_t T, int64_t V, int64_t ldz,
                                        const void* ids, int ids64, const void* starts, int starts64, int64_t pairs,
                                        const float* ref_logp, const float* weight, float beta, float smoothing,
                                        float temperature, float grad_scale, const zr_plan* plan, float* loss,
                                        float* rewards, void* grad, int64_t ldg, void* work, void* stream) {
  zr::clear_error();
  zr::Range range("zr_preference_loss");
  if (zr_status st = zr::check_logits("zr_preference_loss", dt, T, V, ldz, temperature)) return st;
  if (pairs < 0) return fail(ZR_ERR_INVALID, "zr_preference_loss: negative number of pairs");
  if (!zr::finite(beta) || !zr::finite(grad_scale))
    return fail(ZR_ERR_INVALID, "zr_preference_loss: beta or grad_scale is not finite");
  if (!(smoothing >= 0.0f && smoothing <= 1.0f))
    return fail(ZR_ERR_INVALID, "zr_preference_loss: smoothing must lie in [0, 1]");
  if (grad && ldg < V) return fail(ZR_ERR_INVALID, "zr_preference_loss: a row stride is under the row");
  if (T > kMostRows || pairs > kMostPairs)
    return fail(ZR_ERR_UNSUPPORTED, "zr_preference_loss: too many rows or pairs for one launch");
  if (pairs == 0) return ZR_OK;
  if (!starts || !loss || !work || (T > 0 && (!logits || !ids || !ref_logp)))
    return fail(ZR_ERR_INVALID, "zr_preference_loss: null pointer");
  if (!zr::aligned16(logits) || !zr::aligned16(grad) || !zr::aligned16(work) || !zr::aligned_to(ids, ids64 ? 8 : 4) ||
      !zr::aligned_to(starts, starts64 ? 8 : 4) || !zr::aligned_to(ref_logp, 4) || !zr::aligned_to(weight, 4) ||
      !zr::aligned_to(loss, 4) || !zr::aligned_to(rewards, 4))
    return fail(ZR_ERR_INVALID, "zr_preference_loss: a pointer is not aligned");
  if (T > 0)
    if (zr_status st = zr::check_gradient("zr_preference_loss", logits, grad, dt, T, V, ldz, ldg)) return st;
  const int sms = zr::sm_count("zr_preference_loss");
  if (sms == 0) return ZR_ERR_CUDA;
  PreferenceArgs a{};
  a.z = logits; a.ids = ids; a.starts = starts; a.ref_logp = ref_logp; a.weight = weight;
  a.loss_scale = plan ? &plan->ctrl_dev->scale : nullptr;
  a.loss = loss; a.rewards = rewards; a.grad = grad;
  a.sums = static_cast<RowSum*>(work);
  a.ratio = reinterpret_cast<float*>(a.sums + T);
  a.slope = a.ratio + T;
  a.T = T; a.V = V; a.ldz = ldz; a.ldg = ldg;
  a.sequences = 2 * (int)pairs;
  a.wide_ids = ids64; a.wide_starts = starts64;
  a.scale = zr::scale_of(temperature);
  a.beta = beta; a.smoothing = smoothing; a.grad_scale = grad_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == ZR_F16) return launch<zr::DT_F16>(a, sms, s);
  if (dt == ZR_BF16) return launch<zr::DT_BF16>(a, sms, s);
  return launch<zr::DT_F32>(a, sms, s);
}
