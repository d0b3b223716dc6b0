// The log-probabilities of chosen tokens, and the clipped policy loss with a KL term, forward and
// backward from one read of the logits.
//
// With q = softmax(z / tau) over the vocabulary and a the chosen column, logp = log q_a. The loss of a
// token is w (-min(r A, clip(r) A) + kl (e^d - d - 1)), r = e^(logp - old), d = ref - logp; it sees the
// row only through logp, so its gradient is dz_v = f (1[v = a] - q_v) with f = dloss/dlogp / tau, known
// once the row has been summed.
//
// A logit's bytes once, and for the loss its gradient's, bind both. Log-probabilities are summed as the rows
// come, through registers, four words of a thread on their way together and six blocks of 256 threads on an SM
// (the registers are held to 40 for that: 128 us at 8192 x 50304 bf16, 150 with the 56 that the compiler would
// take): 6.4 TB/s; with entropies 137 us, the exponentials' arithmetic in the way. The policy loss holds a row
// in shared memory between its sum and its gradient, 8192 x 50304 bf16 in 270 us, 6.1 TB/s, and 258 where a
// tenth of the rows carries no weight; shorter rows have as many at work as fit, 8192 x 8000 in 49 us, 1000 fp32
// in 14. 11 x 50257 fp32, a cluster of 8 blocks to a row: 5.5 us, the cluster's two waits about 1 each.
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

struct LogprobArgs {
  const void* z;
  const void* ids;
  float* logp;
  float* entropy;  // null: none
  int64_t T, V, ldz, share;
  int wide_ids;
  zr::Scale scale;
};

template <int DT, bool ENTROPY, int C>
__global__ void __launch_bounds__(384, 4) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int es = DT == zr::DT_F32 ? 4 : 2;
  __shared__ zr::Parts sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / C;
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  if (C > 1) zr::cluster_arrived();
  zr::wait_for_previous();
  const int64_t id = zr::id_at(a.ids, a.wide_ids, row);
  if (id < 0) {  // not scored, and not read (the same in the whole cluster)
    if (C > 1) zr::cluster_wait();
    if (rank == 0 && tid == 0) {
      a.logp[row] = 0.0f;
      if (ENTROPY) a.entropy[row] = 0.0f;
    }
    return;
  }
  const int64_t v0 = rank * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;
  const int n = v1 > v0 ? (int)(v1 - v0) : 0;
  const char* whole = static_cast<const char*>(a.z) + row * a.ldz * es;
  const float z_chosen = id < a.V ? zr::load1<DT>(whole, id) : 0.0f;
  const char* part = whole + v0 * es;
  const zr::RowWords<DT> words(part, n, tid);
  const Part mine =
      zr::read_part<DT, !ENTROPY, ENTROPY>(words, part, id >= v0 && id < v1 ? (int)(id - v0) : -1, a.scale, tid, blockDim.x);
  Part all = zr::join_all<ENTROPY, C>(mine, a.scale, sh, rank);
  if (rank == 0 && tid == 0) {
    all = zr::rebased<ENTROPY>(all, fmaxf(all.m, z_chosen), a.scale);
    const zr::Base base(all.m, a.scale);
    const float rest = ENTROPY ? all.trimmed(a.scale) : all.sum;
    const zr::Pair logp = zr::log_chosen<!ENTROPY>(z_chosen, rest, base, a.scale);
    a.logp[row] = id < a.V ? logp.value + logp.rest : NAN;
    if (ENTROPY) {
      // log sum less the mean exponent: two numbers of up to 1 in size where one token has nearly everything, so that what
      // rounding leaves of a smaller entropy may be under 0. Where it is the chosen one, e of its own against the
      // `rest`, the same without the difference: log(1 + rest/e) and how far the others' exponents lie under its own.
      const float x = base.exponent<false>(z_chosen, a.scale), e = zr::exp2_fast(x);
      float entropy;
      if (rest < e) {
        const float under = fmaxf(__fmaf_rn(x, rest, -all.ex), 0.0f);
        entropy = __fmaf_rn(zr::kLn2, __fdiv_rn(under, __fadd_rn(rest, e)), log1pf(__fdiv_rn(rest, e)));
      } else {
        zr::add_term<false, true>(all, base, a.scale, z_chosen);
        entropy = __fmul_rn(zr::kLn2, log2f(all.sum) - __fdiv_rn(all.ex, all.sum));
        entropy = entropy < 0.0f ? 0.0f : entropy;  // (no number stays so)
      }
      a.entropy[row] = id < a.V ? entropy : NAN;
    }
  }
}

struct PolicyArgs {
  const void* z;
  const void* ids;
  const float* old_logp;
  const float* ref_logp;  // null: no KL term
  const float* advantage;
  const float* weight;      // null: 1
  const float* loss_scale;  // null: 1 (a plan's, in device memory)
  float* loss;
  float* logp;  // null: not wanted
  void* grad;   // null: the loss alone
  int64_t T, V, ldz, ldg, share;
  int wide_ids;
  int room;  // 16-byte words of a row's share that shared memory holds
  zr::Scale scale;
  float low, high, kl, grad_scale;
};

// A row in the shared memory of a block, or of a cluster that shares it: one read, its sum, its gradient,
// one write. A thread copies, sums and stores the same words, so the passes need no barrier between them.
// The chosen value is taken out of the row (-inf in its place): the sum is of all others, which is what its
// own gradient, 1 - q_a, keeps its accuracy from where the token is almost certain.
template <int DT, int C>
__global__ void __launch_bounds__(1024) policy_kernel(const __grid_constant__ PolicyArgs a) {
  using W = zr::Word<DT>;
  constexpr int per = W::per, es = 16 / per;
  extern __shared__ __align__(16) char smem[];
  uint4* words = reinterpret_cast<uint4*>(smem);
  zr::Parts& sh = *reinterpret_cast<zr::Parts*>(words + a.room);
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int64_t row = blockIdx.x / C;
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  if (C > 1) zr::cluster_arrived();  // a block's shared memory may be written to once it has begun
  const int64_t v0 = rank * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;
  const int n = v1 > v0 ? (int)(v1 - v0) : 0;  // this block's columns; the last blocks may have none
  const char* whole = static_cast<const char*>(a.z) + row * a.ldz * es;
  const char* zrow = whole + v0 * es;
  char* grad = a.grad ? static_cast<char*>(a.grad) + (row * a.ldg + v0) * es : nullptr;
  const zr::RowWords<DT> r(zrow, n, tid);
  // the gradient's words are the logits' words, shifted: stored whole only where they coincide
  const bool same = grad && (int)(reinterpret_cast<uintptr_t>(grad) & 15) / es == r.lead;
  zr::wait_for_previous();
  const float w = a.weight ? a.weight[row] : 1.0f;
  const int64_t id = zr::id_at(a.ids, a.wide_ids, row);

  if (w == 0.0f || id < 0) {  // no loss and no gradient, whatever the logits hold (the same in the whole cluster)
    if (rank == 0 && tid == 0) {
      a.loss[row] = 0.0f;
      if (a.logp) a.logp[row] = 0.0f;
    }
    if (grad) {
      for (int j = r.first + tid; j < r.last; j += nthr) {
        char* to = grad + (int64_t)(j * per - r.lead) * es;
        if (same)
          zr::st_once(to, make_uint4(0, 0, 0, 0));
        else
          for (int i = 0; i < per; ++i) zr::store1<DT>(to, i, 0.0f);
      }
      if (r.single >= 0) zr::store1<DT>(grad, r.single, 0.0f);
    }
    __syncwarp();
    if (C > 1) zr::cluster_wait();
    return;
  }

  // ---- on the way to shared memory: the words that it holds
  const int kept = min(r.last, a.room);
  for (int j = r.first + tid; j < kept; j += nthr) zr::copy16(zr::smem_u32(words + j), r.words + j);
  const bool known = id < a.V;
  const float z_chosen = known ? zr::load1<DT>(whole, id) : 0.0f;
  const float old_logp = a.old_logp[row], advantage = a.advantage[row];
  const float ref_logp = a.ref_logp ? a.ref_logp[row] : 0.0f;
  const int chosen = id >= v0 && id < v1 ? (int)(id - v0) : -1;
  const int hole = chosen < 0 ? -1 : (r.lead + chosen) / per, at = (r.lead + chosen) % per;
  float z_single = -INFINITY;
  if (r.single >= 0 && r.single != chosen) z_single = zr::load1<DT>(zrow, r.single);

  // ---- each thread's maximum, and its sum relative to it: of the words without room first, meanwhile
  zr::RowWords<DT> beyond = r;
  beyond.first = r.first + max(kept - r.first - tid + nthr - 1, 0) / nthr * nthr;  // this thread's first, less its place
  beyond.single = -1;
  Part p = zr::read_part<DT, false, false>(beyond, zrow, chosen, a.scale, tid, nthr);
  zr::copies_done();
  if (hole >= r.first && hole < kept && (hole - r.first) % nthr == tid) words[hole] = zr::without<DT>(words[hole], at);
  {
    uint32_t most = W::lowest();
    for (int j = r.first + tid; j < kept; j += nthr) most = W::larger(most, words[j]);
    p = zr::rebased<false>(p, fmaxf(fmaxf(p.m, W::largest(most)), z_single), a.scale);
    const zr::Base mine(p.m, a.scale);
    zr::add_words<DT, false, false>(p, mine, a.scale, [&](auto add) {
      for (int j = r.first + tid; j < kept; j += nthr) add(words[j]);
    });
    zr::add_term<false, false>(p, mine, a.scale, z_single);
  }

  // ---- the row's: all other terms, the chosen one's exponent, and what the loss makes of it
  Part rest = zr::join_all<false, C>(p, a.scale, sh, rank);
  rest = zr::rebased<false>(rest, fmaxf(rest.m, z_chosen), a.scale);
  const zr::Base base(rest.m, a.scale);
  const float sum = known ? __fadd_rn(rest.sum, zr::exp2_fast(base.exponent<false>(z_chosen, a.scale))) : NAN;
  const zr::Pair of = zr::log_chosen<false>(z_chosen, rest.sum, base, a.scale);
  const float logp = known ? of.value + of.rest : NAN;
  const float ratio = expf(logp - old_logp), free = __fmul_rn(ratio, advantage);
  const float bound = __fmul_rn(fminf(fmaxf(ratio, a.low), a.high), advantage);
  const bool clipped = free > bound;  // (not where one is no number, which stays so)
  float value = clipped ? -bound : -free, slope = clipped ? 0.0f : -free;
  if (a.ref_logp) {
    const float far = ref_logp - logp, more = expm1f(far);
    value += __fmul_rn(a.kl, more - far);
    slope -= __fmul_rn(a.kl, more);
  }
  if (rank == 0 && tid == 0) {
    a.loss[row] = __fmul_rn(w, value);
    if (a.logp) a.logp[row] = logp;
  }

  // ---- the gradient: all columns, then the chosen one's own
  if (grad) {
    const float scale = a.loss_scale ? __fmul_rn(a.grad_scale, *a.loss_scale) : a.grad_scale;
    const float f = __fmul_rn(__fmul_rn(w, slope), __fdiv_rn(scale, a.scale.tau)), by = -__fdiv_rn(f, sum);
    const zr::Exponents<false> exponents(base, a.scale);
    const zr::Two by2(by, by);
    auto put = [&](int j, uint4 u) {
      float v[per];
      W::open(u, v);
      if (base.whole) {
#pragma unroll
        for (int i = 0; i < per; i += 2) {
          const zr::Two e = exponents.of(v[i], v[i + 1]);
          const zr::Two y = zr::mul2(zr::Two(zr::exp2_fast(e.lo()), zr::exp2_fast(e.hi())), by2);
          v[i] = y.lo();
          v[i + 1] = y.hi();
        }
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) v[i] = __fmul_rn(zr::exp2_fast(base.exponent<false>(v[i], a.scale)), by);
      }
      char* to = grad + (int64_t)(j * per - r.lead) * es;
      if (same) {
        zr::st_once(to, W::close(v));
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) zr::store1<DT>(to, i, v[i]);
      }
    };
    constexpr int kOnce = 4;
    for (int j = beyond.first + tid; j < r.last; j += kOnce * nthr) {
      uint4 u[kOnce];
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (j + i * nthr < r.last) u[i] = zr::ld_row(r.words + j + i * nthr);
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (j + i * nthr < r.last) put(j + i * nthr, u[i]);
    }
    for (int j = r.first + tid; j < kept; j += nthr) put(j, words[j]);
    if (r.single >= 0 && r.single != chosen)
      zr::store1<DT>(grad, r.single, __fmul_rn(zr::exp2_fast(base.exponent<false>(z_single, a.scale)), by));
    __syncthreads();
    if (chosen >= 0 && tid == 0) zr::store1<DT>(grad, chosen, __fmul_rn(f, __fdiv_rn(rest.sum, sum)));
  }
}

template <int DT, int C>
zr_status launch_policy(const PolicyArgs& a, int threads, int smem, cudaStream_t s) {
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_policy_loss", (const void*)policy_kernel<DT, C>, zr::kSmemMost)) return st;
  cudaError_t e = zr::launch(policy_kernel<DT, C>, a.T * C, threads, smem, C, true, s, a);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_policy_loss: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}
template <int DT>
zr_status launch_policy(const PolicyArgs& a, int split, int threads, int smem, cudaStream_t s) {
  if (split == 8) return launch_policy<DT, 8>(a, threads, smem, s);
  if (split == 4) return launch_policy<DT, 4>(a, threads, smem, s);
  if (split == 2) return launch_policy<DT, 2>(a, threads, smem, s);
  return launch_policy<DT, 1>(a, threads, smem, s);
}

template <int DT, bool ENTROPY>
zr_status launch_logprobs(const LogprobArgs& a, const zr::RowShape& r, cudaStream_t s) {
  cudaError_t e = r.split == 8   ? zr::launch(logprob_kernel<DT, ENTROPY, 8>, a.T * 8, r.threads, 0, 8, true, s, a)
                  : r.split == 4 ? zr::launch(logprob_kernel<DT, ENTROPY, 4>, a.T * 4, r.threads, 0, 4, true, s, a)
                  : r.split == 2 ? zr::launch(logprob_kernel<DT, ENTROPY, 2>, a.T * 2, r.threads, 0, 2, true, s, a)
                                 : zr::launch(logprob_kernel<DT, ENTROPY, 1>, a.T, r.threads, 0, 1, true, s, a);
  if (e != cudaSuccess) return fail(ZR_ERR_CUDA, "zr_token_logprobs: launch failed: %s", cudaGetErrorString(e));
  return ZR_OK;
}
template <int DT>
zr_status launch_logprobs(const LogprobArgs& a, const zr::RowShape& r, cudaStream_t s) {
  return a.entropy ? launch_logprobs<DT, true>(a, r, s) : launch_logprobs<DT, false>(a, r, s);
}

}  // namespace

extern "C" zr_status zr_token_logprobs(const void* logits, zr_dtype dt, int64_t T, int64_t V, int64_t ldz,
                                       const void* ids, int ids64, float temperature, float* logp, float* entropy,
                                       void* stream) {
  zr::clear_error();
  zr::Range range("zr_token_logprobs");
  if (zr_status st = zr::check_logits("zr_token_logprobs", dt, T, V, ldz, temperature)) return st;
  if (T == 0) return ZR_OK;
  if (!logits || !ids || !logp) return fail(ZR_ERR_INVALID, "zr_token_logprobs: null pointer");
  if (!zr::aligned16(logits) || !zr::aligned_to(ids, ids64 ? 8 : 4) || !zr::aligned_to(logp, 4) ||
      !zr::aligned_to(entropy, 4))
    return fail(ZR_ERR_INVALID, "zr_token_logprobs: a pointer is not aligned");
  const int sms = zr::sm_count("zr_token_logprobs");
  if (sms == 0) return ZR_ERR_CUDA;
  const zr::RowShape r = zr::streamed_rows(T, V, dt == ZR_F32 ? 4 : 2, sms);
  if (T > 0x7FFFFFFF / r.split) return fail(ZR_ERR_UNSUPPORTED, "zr_token_logprobs: too many rows for one launch");
  LogprobArgs a{};
  a.z = logits; a.ids = ids; a.logp = logp; a.entropy = entropy;
  a.T = T; a.V = V; a.ldz = ldz; a.share = r.share;
  a.wide_ids = ids64; a.scale = zr::scale_of(temperature);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == ZR_F16) return launch_logprobs<zr::DT_F16>(a, r, s);
  if (dt == ZR_BF16) return launch_logprobs<zr::DT_BF16>(a, r, s);
  return launch_logprobs<zr::DT_F32>(a, r, s);
}

extern "C" zr_status zr_policy_loss(const void* logits, zr_dtype dt, int64_t T, int64_t V, int64_t ldz,
                                    const void* ids, int ids64, const float* old_logp, const float* advantage,
                                    const float* weight, float clip_low, float clip_high, const float* ref_logp,
                                    float kl, float temperature, float grad_scale, const zr_plan* plan, float* loss,
                                    float* logp, void* grad, int64_t ldg, void* stream) {
  zr::clear_error();
  zr::Range range("zr_policy_loss");
  if (zr_status st = zr::check_logits("zr_policy_loss", dt, T, V, ldz, temperature)) return st;
  if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f && clip_high <= 1e30f))
    return fail(ZR_ERR_INVALID, "zr_policy_loss: clip_low must lie in [0, 1], clip_high in [0, 1e30]");
  if (!zr::finite(kl)) return fail(ZR_ERR_INVALID, "zr_policy_loss: kl is not finite");
  if (kl != 0.0f && !ref_logp && T > 0) return fail(ZR_ERR_INVALID, "zr_policy_loss: kl without ref_logp");
  if (!zr::finite(grad_scale)) return fail(ZR_ERR_INVALID, "zr_policy_loss: grad_scale is not finite");
  if (grad && ldg < V) return fail(ZR_ERR_INVALID, "zr_policy_loss: a row stride is under the row");
  if (T == 0) return ZR_OK;
  if (!logits || !ids || !old_logp || !advantage || !loss) return fail(ZR_ERR_INVALID, "zr_policy_loss: null pointer");
  if (!zr::aligned16(logits) || !zr::aligned16(grad) || !zr::aligned_to(ids, ids64 ? 8 : 4) ||
      !zr::aligned_to(old_logp, 4) || !zr::aligned_to(advantage, 4) || !zr::aligned_to(weight, 4) ||
      !zr::aligned_to(ref_logp, 4) || !zr::aligned_to(loss, 4) || !zr::aligned_to(logp, 4))
    return fail(ZR_ERR_INVALID, "zr_policy_loss: a pointer is not aligned");
  if (zr_status st = zr::check_gradient("zr_policy_loss", logits, grad, dt, T, V, ldz, ldg)) return st;
  const int sms = zr::sm_count("zr_policy_loss");
  if (sms == 0) return ZR_ERR_CUDA;
  const int es = dt == ZR_F32 ? 4 : 2, fixed = (int)sizeof(zr::Parts);
  const zr::RowShape r = zr::held_rows(T, V, es, fixed, sms);
  if (T > 0x7FFFFFFF / r.split) return fail(ZR_ERR_UNSUPPORTED, "zr_policy_loss: too many rows for one launch");
  PolicyArgs a{};
  a.z = logits; a.ids = ids; a.old_logp = old_logp; a.advantage = advantage; a.weight = weight;
  a.ref_logp = kl != 0.0f ? ref_logp : nullptr;
  a.loss_scale = plan ? &plan->ctrl_dev->scale : nullptr;
  a.loss = loss; a.logp = logp; a.grad = grad;
  a.T = T; a.V = V; a.ldz = ldz; a.ldg = ldg; a.share = r.share;
  a.wide_ids = ids64; a.room = r.room; a.scale = zr::scale_of(temperature);
  a.low = 1.0f - clip_low; a.high = 1.0f + clip_high; a.kl = kl; a.grad_scale = grad_scale;
  const int smem = r.room * 16 + fixed;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == ZR_F16) return launch_policy<zr::DT_F16>(a, r.split, r.threads, smem, s);
  if (dt == ZR_BF16) return launch_policy<zr::DT_BF16>(a, r.split, r.threads, smem, s);
  return launch_policy<zr::DT_F32>(a, r.split, r.threads, smem, s);
}
