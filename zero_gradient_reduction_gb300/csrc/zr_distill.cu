// The distillation loss against a teacher's top logits and its gradient, from one read of the
// student's logits.
//
// With p = softmax(teacher / tau) over a row's kept entries and q = softmax(z / tau) over the
// vocabulary, loss = w tau^2 sum_k p_k (log p_k - log q_id(k)) and dloss/dz = w tau (q - p). A row
// is read once into shared memory (of one block, or of a cluster that shares the row), its
// maximum, its sum of exponentials and its gradient come from there, and the gradient is written
// once; what a long row has beyond that room is summed as it is read, and read again from L2 for its
// gradient. All arithmetic is fp32; sums are taken in an order that the sizes alone decide.
//
// Two bytes (or four) a logit each way bind it: 8192 x 50304 bf16 in 263 us, 6.3 TB/s of the 6.7 that
// a copy reaches, and in 248 us where a tenth of the rows carries no weight and is not read (6.3, too),
// with two rows at work on each multiprocessor (101 KB each), one read while the other is summed. In
// the logits' place 272 us; the loss alone 175, 4.7 TB/s. A thousand entries a row, which one warp
// takes, cost more than a row: 658 us, 311 with 256. Of the case with a tenth of the rows without weight
// a first form with loads through registers and fp32 one at a time took 724 us, asynchronous copies 344,
// two exponentials' arithmetic in one instruction and results under 2^-126 to zero 310, the teacher's
// entries in a warp of their own 263. Shorter rows have as many at work as fit:
// 8192 x 8000 bf16 in 55 us with ten, 104 with three. Blocks that stay and fetch the next row's words
// into the places of the gradient's were slower (307 and 67 us): they all read, then all sum, together.
// 13 x 50257 fp32, a cluster of 8 blocks to a row: 8.8 us, of which a launch is 2.5 and each wait of the
// cluster about 1.
#include <cuda_runtime.h>

#include <cstdint>

#include "zr_device.cuh"
#include "zr_internal.h"
#include "zr_launch.h"
#include "zr_nvtx.h"
#include "zr_plan.h"
#include "zr_rows.cuh"
#include "zr_tensor.cuh"

using zr::add2;
using zr::exp2_fast;
using zr::fail;
using zr::fma2;
using zr::kLn2;
using zr::kLog2E;
using zr::ld_row;
using zr::mul2;
using zr::store1;
using zr::Two;
using zr::warp_max;
using zr::warp_sum;
using zr::Word;

namespace {

constexpr int kMaxThreads = 1024;  // the last warp for the teacher's entries, the others for a row's words

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
  int K, K4, wide_ids, tdt;  // K4: K to a multiple of 4
  int slot_bits;             // log2 of the slots of an entry's column: at least 2 K of them
  int room;             // 16-byte words of a row's share that shared memory holds
  float tau, grad_scale;
};

// A sum of exponentials is kept relative to the maximum m of its z, in base 2 and as one
// multiply-add: sum of 2^(z c - mc), mc = m c rounded. That rounding multiplies every term by the
// same factor, which cancels in q and in log q. Where m c is so large that the factor would be
// anything (logits of 10^4 at a temperature of 0.01, a mask of the type's lowest value) the terms are
// 2^((z - m) c). A part that is all masked has m = -inf; its terms are taken relative to 0: 0, or NaN
// where z is.
struct Base {
  float m, mc, c;
  bool fused;
  __device__ Base(float largest, float c_) : c(c_) {
    m = largest == -INFINITY ? 0.0f : largest;
    mc = __fmul_rn(m, c);
    fused = fabsf(mc) < 1e6f;  // a factor of at most 2^(1/32); not where m is NaN or infinite either
  }
  __device__ float exponent(float z) const { return fused ? __fmaf_rn(z, c, -mc) : __fmul_rn(z - m, c); }
};
// A sum relative to the maximum m, relative to a larger one: each as it is kept.
__device__ __forceinline__ float rescaled(float m, float sum, const Base& to) {
  if (m == -INFINITY) return sum;
  const Base from(m, to.c);
  const float e = from.fused ? (to.fused ? from.mc - to.mc : __fmaf_rn(-to.m, to.c, from.mc)) : to.exponent(from.m);
  return __fmul_rn(sum, exp2_fast(e));
}

// Which columns stand in a row's entries more than once: a table of the columns in shared memory,
// filled by one warp in any order, the sign marking those taken again. Looking through all K
// entries for each of them cost 8192 rows of 256 entries as much again as the row itself.
constexpr int kNoColumn = 0x7FFFFFFF;
__device__ __forceinline__ int slot_of(int id, int bits) { return (int)((uint32_t)id * 2654435761u >> (32 - bits)); }
// Goes on from a slot that held `was` when an entry came to it.
__device__ __forceinline__ void take_slot(int* slots, int bits, int id, int at, int was) {
  const int mask = (1 << bits) - 1;
  while (was != kNoColumn) {  // ends: half the slots stay free
    if ((was & 0x7FFFFFFF) == id) {
      if (was >= 0) atomicOr(slots + at, (int)0x80000000);
      return;
    }
    at = (at + 1) & mask;
    was = atomicCAS(slots + at, kNoColumn, id);
  }
}
__device__ __forceinline__ bool several(const int* slots, int bits, int id, int at, int there) {
  const int mask = (1 << bits) - 1;
  while ((there & 0x7FFFFFFF) != id) there = slots[at = (at + 1) & mask];
  return there < 0;
}

// The exponentials of a word's logits relative to a maximum, summed: two by two where that is one
// multiply-add.
template <int DT>
__device__ __forceinline__ Two terms(uint4 u, Two c, Two less) {
  constexpr int per = Word<DT>::per;
  float f[per];
  Word<DT>::open(u, f);
  Two part(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < per; i += 2) {
    const Two x = fma2(Two(f[i], f[i + 1]), c, less);
    part = add2(part, Two(exp2_fast(x.lo()), exp2_fast(x.hi())));
  }
  return part;
}
template <int DT>
__device__ __forceinline__ float terms(uint4 u, const Base& base) {
  if (base.fused) {
    const Two part = terms<DT>(u, Two(base.c, base.c), Two(-base.mc, -base.mc));
    return __fadd_rn(part.lo(), part.hi());
  }
  constexpr int per = Word<DT>::per;
  float f[per], sum = 0.0f;
  Word<DT>::open(u, f);
#pragma unroll
  for (int i = 0; i < per; ++i) sum = __fadd_rn(sum, exp2_fast(base.exponent(f[i])));
  return sum;
}

// A row's entries as they stand in memory, to shared memory: ids of 4 or 8 bytes, and the words of 4
// bytes that hold the logits (of a word that the row's last entry begins, 2 bytes: the array may end
// there). They are asked for before the row is, and all together: behind a row's copies each turn of
// loads waits for 100 KB (8192 rows of 50304 with 256 entries each took 413 us in eight turns).
__device__ __forceinline__ void ask_for_entries(const DistillArgs& a, int64_t row, int lane, void* ids, void* logits) {
  const int half = a.tdt != zr::DT_F32;
  for (int k = lane; k < a.K; k += 32) {
    const int64_t at = row * a.ldk + k;
    if (a.wide_ids)
      zr::copy8(zr::smem_u32(static_cast<int64_t*>(ids) + k), static_cast<const int64_t*>(a.ids) + at);
    else
      zr::copy4(zr::smem_u32(static_cast<int32_t*>(ids) + k), static_cast<const int32_t*>(a.ids) + at);
    zr::copy_of<4>(zr::smem_u32(static_cast<uint32_t*>(logits) + k), static_cast<const uint32_t*>(a.teacher) + (at >> half),
                   half && k == a.K - 1 && !(at & 1) ? 2 : 4);
  }
}
__device__ __forceinline__ float teacher_logit(const DistillArgs& a, int64_t row, int k, uint32_t w) {
  if (a.tdt == zr::DT_F32) return __uint_as_float(w);
  const uint16_t v = (uint16_t)(w >> ((row * a.ldk + k) & 1) * 16);
  return a.tdt == zr::DT_BF16 ? zr::to_f32<zr::DT_BF16>(v) : zr::to_f32<zr::DT_F16>(v);
}

struct Shared {      // what the block's warps, and the cluster's blocks, tell each other
  float m[32], sum[32], loss[32];  // of each warp
  float row_m[8], row_sum[8], row_loss[8];  // of the cluster's blocks: each tells all, the loss the first
  int some, no_answer;
};

// A row is handled in the 16-byte words of memory that hold it: word 0 begins at the boundary at
// or before its first value, so every load is aligned whatever the row stride; `lead` values of
// word 0 belong to the row before, and the last word may end past the row. A thread copies, sums
// and stores the same words, so the passes need no barrier between them; the last warp has no words
// and reads the teacher's entries while the row is on its way.
template <int DT, int C>
__global__ void __launch_bounds__(kMaxThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  using W = Word<DT>;
  constexpr int per = W::per, es = 16 / per;
  extern __shared__ __align__(16) char smem[];
  uint4* words = reinterpret_cast<uint4*>(smem);
  int* sid = reinterpret_cast<int*>(words + a.room);  // an entry's column, or -1
  float* sp = reinterpret_cast<float*>(sid + a.K4);   // its p
  float* own = sp + a.K4;                             // its log2 p, then the gradient at its column
  float* all = own + a.K4;                            // the p of all entries at its column
  int* slots = reinterpret_cast<int*>(all + a.K4);    // the columns, by hash
  Shared& sh = *reinterpret_cast<Shared*>(slots + (1 << a.slot_bits));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthr = blockDim.x - 32;  // those that share the words
  const int64_t row = blockIdx.x / C;
  const int rank = C > 1 ? (int)zr::cluster_rank() : 0;
  const int64_t v0 = rank * a.share, v1 = v0 + a.share < a.V ? v0 + a.share : a.V;
  const int n = v1 > v0 ? (int)(v1 - v0) : 0;  // this block's columns; the last blocks may have none

  if (C > 1) zr::cluster_arrived();  // a block's shared memory may be written to once it has begun
  const float w = a.weight ? a.weight[row] : 1.0f;
  const float c = __fdiv_rn(kLog2E, a.tau);
  char* grad = a.grad ? static_cast<char*>(a.grad) + (row * a.ldg + v0) * es : nullptr;
  const char* zrow = static_cast<const char*>(a.z) + (row * a.ldz + v0) * es;
  const int lead = (int)(reinterpret_cast<uintptr_t>(zrow) & 15) / es;
  const uint4* zw = reinterpret_cast<const uint4*>(zrow - lead * es);
  const int nw = n > 0 ? (lead + n + per - 1) / per : 0;
  // the gradient's words are the logits' words, shifted: stored whole only where they coincide
  const bool same = grad && (int)(reinterpret_cast<uintptr_t>(grad) & 15) / es == lead;

  // whole words [first, last) and, before and behind them, under a word's worth of single values:
  // those go to one thread each, which keeps its value in a register
  const int first = lead > 0 ? 1 : 0, last = (lead + n) / per;
  const int head = lead > 0 ? min(n, per - lead) : 0, behind = max(head, last * per - lead);
  const int single = tid < head ? tid : tid >= 8 && tid - 8 < n - behind ? behind + tid - 8 : -1;
  float z_single = -INFINITY;

  if (tid >= nthr) ask_for_entries(a, row, lane, own, sp);  // (ids of 8 bytes reach over `all`)
  bool some = w != 0.0f;
  if (some) {
    for (int j = first + tid; tid < nthr && j < min(last, a.room); j += nthr)
      zr::copy16(zr::smem_u32(words + j), zw + j);
    if (single >= 0) {
      if (single == 0 && first == 1) zr::copy16(zr::smem_u32(words), zw);
      if (single == n - 1 && last >= first && last < min(nw, a.room)) zr::copy16(zr::smem_u32(words + last), zw + last);
      z_single = zr::load1<DT>(zrow, single);
    }
    if (tid >= nthr) {
      // ---- the teacher's entries: p over the kept ones
      float t_max = -INFINITY;
      int any = 0, no_answer = 0;
      for (int i = lane; i < 1 << a.slot_bits; i += 32) slots[i] = kNoColumn;
      zr::copies_done();
      for (int k = lane; k < a.K4; k += 32) {  // (an entry's bytes are this lane's own copies)
        int64_t id = -1;
        float t = 0.0f;
        if (k < a.K) {
          id = a.wide_ids ? reinterpret_cast<const int64_t*>(own)[k] : reinterpret_cast<const int32_t*>(own)[k];
          t = teacher_logit(a, row, k, __float_as_uint(sp[k]));
        }
        const bool kept = id >= 0;
        no_answer |= id >= a.V || (kept && !(t < INFINITY));
        any |= kept && !(t == -INFINITY);  // a masked entry is none
        if (kept) t_max = fmaxf(t_max, t);
        sid[k] = kept && id < a.V ? (int)id : -1;
        sp[k] = kept ? t : -INFINITY;
      }
      __syncwarp();
      any = __any_sync(0xFFFFFFFFu, any);
      no_answer = __any_sync(0xFFFFFFFFu, no_answer);
      t_max = warp_max(t_max);
      // an entry of -inf has p = 0
      constexpr int kEntries = 4;  // of a lane, so that their first looks at the table overlap
      float p_sum = 0.0f;
      for (int k0 = lane; k0 < a.K4; k0 += 32 * kEntries) {
        int id[kEntries], at[kEntries], was[kEntries];
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const int k = k0 + 32 * i;
          id[i] = k < a.K4 ? sid[k] : -1;
          at[i] = slot_of(id[i], a.slot_bits);
          was[i] = id[i] >= 0 ? atomicCAS(slots + at[i], kNoColumn, id[i]) : kNoColumn;
        }
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const int k = k0 + 32 * i;
          if (k < a.K4) p_sum += sp[k] = exp2_fast(own[k] = (sp[k] - t_max) * c);
        }
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
          if (id[i] >= 0) take_slot(slots, a.slot_bits, id[i], at[i], was[i]);
      }
      p_sum = warp_sum(p_sum);
      const float log_p = log2f(p_sum);
      for (int k = lane; k < a.K4; k += 32) {
        sp[k] = __fdiv_rn(sp[k], p_sum);
        own[k] -= log_p;
      }
      __syncwarp();
      for (int k0 = lane; k0 < a.K; k0 += 32 * kEntries) {
        int id[kEntries], at[kEntries], there[kEntries];
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const int k = k0 + 32 * i;
          id[i] = k < a.K ? sid[k] : -1;
          at[i] = slot_of(id[i], a.slot_bits);
          there[i] = slots[at[i]];
        }
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const int k = k0 + 32 * i;
          if (k >= a.K) break;
          float p = sp[k];
          if (id[i] >= 0 && several(slots, a.slot_bits, id[i], at[i], there[i])) {  // each of them finds the same sum
            p = 0.0f;
            for (int j = 0; j < a.K; ++j)
              if (sid[j] == id[i]) p += sp[j];
          }
          all[k] = p;
        }
      }
      if (lane == 0) {
        sh.some = any;
        sh.no_answer = no_answer;
      }
    }
  }

  auto value = [&](int i) {  // the i-th logit of this block's columns
    i += lead;
    return i / per < a.room ? zr::load1<DT>(smem, i) : zr::load1<DT>(zw, i);
  };
  // the words that shared memory holds, and the first of this thread's that it does not
  const int kept = min(last, a.room);
  const int more = first + tid + max(kept - first - tid + nthr - 1, 0) / nthr * nthr;
  constexpr int kOnce = 4;  // of the others, on their way together

  if (some && tid < nthr) {
    // ---- each thread's maximum, and its sum relative to it: of the words without room first, while
    // the others are on their way
    float m = -INFINITY, sum = 0.0f;
    for (int j = more; j < last; j += kOnce * nthr) {
      uint4 u[kOnce];
      uint32_t most = W::lowest();
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        u[i] = j + i * nthr < last ? ld_row(zw + j + i * nthr)
                                   : make_uint4(W::lowest(), W::lowest(), W::lowest(), W::lowest());
#pragma unroll
      for (int i = 0; i < kOnce; ++i) most = W::larger(most, u[i]);
      const float m_all = fmaxf(m, W::largest(most));
      const Base mine(m_all, c);
      if (m_all != m) sum = rescaled(m, sum, mine);
      m = m_all;
#pragma unroll
      for (int i = 0; i < kOnce; ++i) sum = __fadd_rn(sum, terms<DT>(u[i], mine));
    }
    zr::copies_done();
    uint32_t most = W::lowest();
    for (int j = first + tid; j < kept; j += nthr) most = W::larger(most, words[j]);
    const float m_over = m;
    m = fmaxf(fmaxf(m, W::largest(most)), z_single);
    const Base mine(m, c);
    sum = rescaled(m_over, sum, mine);
    if (mine.fused) {
      const Two cc(c, c), less(-mine.mc, -mine.mc);
      Two total(0.0f, 0.0f);
      for (int j = first + tid; j < kept; j += nthr) total = add2(total, terms<DT>(words[j], cc, less));
      sum = __fadd_rn(sum, __fadd_rn(total.lo(), total.hi()));
    } else {
      for (int j = first + tid; j < kept; j += nthr) sum = __fadd_rn(sum, terms<DT>(words[j], mine));
    }
    sum = __fadd_rn(sum, exp2_fast(mine.exponent(z_single)));
    const float wm = warp_max(m);
    sum = warp_sum(rescaled(m, sum, Base(wm, c)));
    if (lane == 0) {
      sh.m[warp] = wm;
      sh.sum[warp] = sum;
    }
  }
  if (some) {
    __syncthreads();
    some = sh.some;
  }

  if (!some && tid >= nthr) zr::copies_done();
  if (!some) {  // no weight, or nothing kept: no loss and no gradient (the same in the whole cluster)
    if (rank == 0 && tid == 0) a.loss[row] = 0.0f;
    if (grad && tid < nthr) {
      for (int j = first + tid; j < last; j += nthr) {
        char* to = grad + (int64_t)(j * per - lead) * es;
        if (same)
          zr::st_once(to, make_uint4(0, 0, 0, 0));
        else
          for (int i = 0; i < per; ++i) store1<DT>(to, i, 0.0f);
      }
      if (single >= 0) store1<DT>(grad, single, 0.0f);
    }
    __syncwarp();
    if (C > 1) zr::cluster_wait();
    return;
  }

  const bool has = lane < (nthr >> 5);
  float wm = has ? sh.m[lane] : -INFINITY, m = warp_max(wm);
  float sum = warp_sum(has ? rescaled(wm, sh.sum[lane], Base(m, c)) : 0.0f);
  if (C > 1) {
    __syncwarp();
    zr::cluster_wait();
    if (tid < C) {
      zr::cluster_store(zr::cluster_addr(zr::smem_u32(&sh.row_m[rank]), tid), m);
      zr::cluster_store(zr::cluster_addr(zr::smem_u32(&sh.row_sum[rank]), tid), sum);
    }
    __syncwarp();
    zr::cluster_sync();
    m = -INFINITY;
#pragma unroll
    for (int r = 0; r < C; ++r) m = fmaxf(m, sh.row_m[r]);
    sum = 0.0f;
#pragma unroll
    for (int r = 0; r < C; ++r) sum = __fadd_rn(sum, rescaled(sh.row_m[r], sh.row_sum[r], Base(m, c)));
  }
  const Base base(m, c);
  if (sh.no_answer) sum = NAN;  // an entry past the vocabulary, or no number: so are the loss and the whole gradient

  // ---- the entries in this block's columns: their loss, and the gradient there
  const float scale = a.scale ? __fmul_rn(a.grad_scale, *a.scale) : a.grad_scale;
  const float f = __fmul_rn(w, __fmul_rn(a.tau, scale));
  const float log_q = log2f(sum);
  float loss = 0.0f;
  for (int k = tid; k < a.K; k += blockDim.x) {
    const int id = sid[k];
    if (id >= v0 && id < v1) {
      const float zc = base.exponent(value((int)(id - v0)));
      if (!(sp[k] == 0.0f)) loss += sp[k] * (own[k] - (zc - log_q)) * kLn2;
      own[k] = __fmul_rn(f, __fdiv_rn(exp2_fast(zc), sum) - all[k]);
    }
  }
  loss = warp_sum(loss);
  if (lane == 0) sh.loss[warp] = loss;
  if (C > 1 || nw > a.room) __syncthreads();  // the entries' logits are read before the gradient may replace them
  if (C > 1) {  // the blocks' parts of the loss travel while the gradient is written
    if (warp == 0) {
      loss = warp_sum(lane <= (nthr >> 5) ? sh.loss[lane] : 0.0f);
      if (lane == 0) zr::cluster_store(zr::cluster_addr(zr::smem_u32(&sh.row_loss[rank]), 0), loss);
    }
    __syncwarp();
    zr::cluster_arrived();
  }

  // ---- the gradient: all columns, then the entries' own
  if (grad) {
    const float fq = __fdiv_rn(f, sum);
    const Two cc(c, c), less(-base.mc, -base.mc), by(fq, fq);
    auto put = [&](int j, uint4 u) {
      float v[per];
      W::open(u, v);
      if (base.fused) {
#pragma unroll
        for (int i = 0; i < per; i += 2) {
          const Two x = fma2(Two(v[i], v[i + 1]), cc, less);
          const Two y = mul2(Two(exp2_fast(x.lo()), exp2_fast(x.hi())), by);
          v[i] = y.lo();
          v[i + 1] = y.hi();
        }
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) v[i] = __fmul_rn(exp2_fast(base.exponent(v[i])), fq);
      }
      char* to = grad + (int64_t)(j * per - lead) * es;
      if (same) {
        zr::st_once(to, W::close(v));
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) store1<DT>(to, i, v[i]);
      }
    };
    if (tid < nthr) {
      for (int j = more; j < last; j += kOnce * nthr) {
        uint4 u[kOnce];
#pragma unroll
        for (int i = 0; i < kOnce; ++i)
          if (j + i * nthr < last) u[i] = ld_row(zw + j + i * nthr);
#pragma unroll
        for (int i = 0; i < kOnce; ++i)
          if (j + i * nthr < last) put(j + i * nthr, u[i]);
      }
      for (int j = first + tid; j < kept; j += nthr) put(j, words[j]);
    }
    if (single >= 0) store1<DT>(grad, single, __fmul_rn(exp2_fast(base.exponent(z_single)), fq));
  }
  __syncthreads();
  if (grad)
    for (int k = tid; k < a.K; k += blockDim.x)
      if (sid[k] >= v0 && sid[k] < v1) store1<DT>(grad, sid[k] - v0, own[k]);
  if (C > 1) {
    __syncwarp();
    zr::cluster_wait();
  }
  if (rank == 0 && warp == 0) {
    if (C > 1) {
      loss = 0.0f;
#pragma unroll
      for (int r = 0; r < C; ++r) loss = __fadd_rn(loss, sh.row_loss[r]);
    } else {
      loss = warp_sum(lane <= (nthr >> 5) ? sh.loss[lane] : 0.0f);
    }
    if (lane == 0) a.loss[row] = sh.no_answer ? NAN : __fmul_rn(loss, __fmul_rn(w, __fmul_rn(a.tau, a.tau)));
  }
}

template <int DT, int C>
zr_status launch(const DistillArgs& a, int threads, int smem, cudaStream_t s) {
  static zr::SmemAllowance allowance;
  if (zr_status st = allowance.allow("zr_distill_topk", (const void*)distill_kernel<DT, C>, zr::kSmemMost)) return st;
  cudaError_t e = zr::launch(distill_kernel<DT, C>, a.T * C, threads, smem, C, false, s, a);
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
  if (T < 0 || V < 1 || V > 0x7FFFFF00)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: T must be >= 0 and V in [1, 2^31 - 256]");
  if (K < 1 || K > ZR_DISTILL_MAX_TOP)
    return fail(ZR_ERR_INVALID, "zr_distill_topk: K=%d outside [1, %d]", K, ZR_DISTILL_MAX_TOP);
  if (ldz < V || ldk < K || (grad && ldg < V))
    return fail(ZR_ERR_INVALID, "zr_distill_topk: a row stride is under the row");
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
  a.K = K; a.K4 = (K + 3) & ~3; a.wide_ids = ids64; a.tdt = (int)teacher_dt;
  a.tau = temperature; a.grad_scale = grad_scale;
  // How many blocks share a row, and how many an SM has at once. Its memory holds so many words of a row
  // each; what a row has beyond them is read again, from L2. One block takes a row of up to 1.2 times
  // what two blocks to an SM hold (7229 x 57000 bf16 in 270 us, 372 with one) or of what one holds;
  // longer rows go to as few blocks as have up to 1.2 times the half each. Where rows leave SMs free
  // each is shared as far as those go and its parts stay 24 KB long.
  // A quarter full the table of columns is walked less than half full (256 entries by 8192 x 8000 in 75 us
  // against 98), as long as it is small.
  a.slot_bits = 1;
  while (1 << a.slot_bits < 2 * K || (1 << a.slot_bits < 4 * K && a.slot_bits < 11)) ++a.slot_bits;  // up to 8 KB
  const int fixed = a.K4 * 16 + (4 << a.slot_bits) + (int)sizeof(Shared);
  auto held = [&](int blocks) { return ((zr::kSmemMost + 1024) / blocks - 1024 - fixed) / 16; };
  const int unit = 16 / es;
  auto words = [&](int split) { return (V + split * unit - 1) / (split * unit) + 1; };  // 1: it may begin inside a word
  auto nearly = [&](int64_t n, int blocks) { return n * 5 <= (int64_t)held(blocks) * 6; };
  int split = 1;
  if (words(1) > held(1) && !nearly(words(1), 2))
    while (split < 8 && !nearly(words(split), 2)) split *= 2;
  while (split < 8 && T * split * 2 <= sms && words(split) > 3000) split *= 2;
  if (T > 0x7FFFFFFF / split) return fail(ZR_ERR_UNSUPPORTED, "zr_distill_topk: too many rows for one launch");
  const int64_t room = words(split);
  a.share = (room - 1) * unit;
  // One more block than fit whole where it nearly does: for a row of its own the second only, in a
  // cluster, which waits more, others too (1373 x 150000 fp32 in 296 us with 3, 348 with 2). A thread has
  // 20 words at most: 8192 x 8000 bf16 in 55 us with 10 blocks of 2 warps, 71 with 14 of one.
  int blocks = 1;
  while (blocks < 16 && T * split > (int64_t)blocks * sms && room <= 20 * (1024 / (blocks + 1) / 32 * 32 - 32) &&
         (room <= held(blocks + 1) || ((blocks == 1 || split > 1) && nearly(room, blocks + 1)))) ++blocks;
  a.room = (int)(room < held(blocks) ? room : held(blocks));
  // They share the SM's registers, 64 a thread. A row that has its SM to itself takes fewer threads, as
  // barriers cost more than words then (13 x 50257 fp32 in 9.0 us with 384, 9.9 with 1024).
  int threads = T * split <= sms ? 384 : 1024 / blocks / 32 * 32;
  if (threads > (room + 31) / 32 * 32 + 32) threads = (int)((room + 31) / 32 * 32 + 32);
  const int smem = a.room * 16 + fixed;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == ZR_F16) return launch_split<zr::DT_F16>(a, split, threads, smem, s);
  if (dt == ZR_BF16) return launch_split<zr::DT_BF16>(a, split, threads, smem, s);
  return launch_split<zr::DT_F32>(a, split, threads, smem, s);
}
