// Rows of logits as the losses read them: in the 16-byte words of memory that hold them, with sums of
// exponentials kept relative to a maximum.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "zr_device.cuh"
#include "zr_launch.h"
#include "zr_tensor.cuh"

namespace zr {

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// Not the read-only path: the gradient may replace the logits, and a launch that begins early may find them still being
// written. Nor is it moved across a wait.
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// 2^x to 2 ulp, results under 2^-126 to zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
struct Two {
  uint64_t v;
  __device__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ explicit Two(uint64_t w) : v(w) {}
  __device__ float lo() const { return __uint_as_float((uint32_t)v); }
  __device__ float hi() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
  return Two(r);
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return Two(r);
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return Two(r);
}

template <int DT>
struct Word {
  static constexpr int per = DT == DT_F32 ? 4 : 8;
  __device__ static void open(uint4 u, float f[per]) {
    if constexpr (DT == DT_F32) {
      f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
      f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    } else {
      unpack8<DT>(u, f);
    }
  }
  // The larger of m and the word's values, two at a time in 16 bits; `m` starts as lowest().
  __device__ static uint32_t lowest() {
    return DT == DT_F32 ? 0xFF800000u : DT == DT_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  }
  __device__ static uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (DT == DT_F32) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (DT == DT_BF16) {
      const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  __device__ static uint32_t larger(uint32_t m, uint4 u) {
    return larger(larger(m, larger(u.x, u.y)), larger(u.z, u.w));
  }
  __device__ static float largest(uint32_t m) {
    if constexpr (DT == DT_F32)
      return __uint_as_float(m);
    else
      return fmaxf(to_f32<DT>((uint16_t)m), to_f32<DT>((uint16_t)(m >> 16)));
  }
  __device__ static uint4 close(const float f[per]) {
    if constexpr (DT == DT_F32)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return pack8<DT>(f);
  }
};

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (DT == DT_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = from_f32<DT == DT_F32 ? DT_BF16 : DT>(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// 1/tau times log2(e): in one number of 32 bits, in two (the upper 12 bits and the next 24), and what the one
// is short of, as a share of it, in units of a term's logarithm.
struct Scale {
  float c, hi, lo, trim, tau;
};
inline Scale scale_of(float tau) {
  const double c = 1.4426950408889634 / tau;
  Scale s{(float)c, 0.0f, 0.0f, 0.0f, tau};
  uint64_t bits;
  std::memcpy(&bits, &c, 8);
  bits &= ~((uint64_t)0x1FFFFFFFFFF);  // downwards, so that the rest is positive: an infinity times it keeps its sign
  double upper;
  std::memcpy(&upper, &bits, 8);
  s.hi = (float)upper;
  s.lo = c > upper ? (float)(c - upper) : 1e-37f;
  s.trim = (float)((c - s.c) / s.c * 0.6931471805599453);
  return s;
}

// A sum of exponentials is kept in base 2 relative to the whole number M at or over m c, m the largest z
// and c = log2(e)/tau: sum of 2^(z c - M). M is whole so that a sum moves to another maximum by an exact power
// of two. Where M is so large that its own rounding would count (logits of 10^4, a low temperature, a mask of
// the type's lowest value) the terms are 2^((z - m) c). A part that is all masked has m = -inf; its terms
// are taken relative to 0: 0, or NaN where z is.
// A c of 24 bits is off by the same for every term, and a row's log-probability by some 10^-7, always the same
// way; a sequence adds thousands of them. So exponents may be FINE, two multiply-adds with both parts of c
// while M is under 32 (the first is rounded like M): they cost a row that is only read nothing (8192 x 50304
// bf16 in 130 us, 128), but one that is held and written 19 us of 268. A sum with its entropy needs none,
// the entropy says what c's error has made of it (Part::trimmed).
struct Base {
  float m, M, hi, lo;
  bool whole, fine;
  __device__ Base(float largest, const Scale& k) {
    m = largest == -INFINITY ? 0.0f : largest;
    M = ceilf(__fmul_rn(m, k.c));
    whole = fabsf(M) <= 256.0f;  // (not where m is infinite)
    fine = fabsf(M) <= 32.0f;
    hi = fine ? k.hi : k.c;
    lo = fine ? k.lo : 1e-37f;  // no part in a sum, and an infinity with a logit of -inf
  }
  template <bool FINE>
  __device__ float exponent(float z, const Scale& k) const {
    if (!whole) return __fmul_rn(z - m, k.c);
    return FINE ? __fmaf_rn(z, hi, __fmaf_rn(z, lo, -M)) : __fmaf_rn(z, k.c, -M);
  }
  // How far a term of m lies under 1 with the c of 24 bits, as an exponent.
  __device__ float below(const Scale& k) const { return whole ? __fmaf_rn(m, k.c, -M) : 0.0f; }
};
// The exponents of two values, where M is whole.
template <bool FINE>
struct Exponents {
  Two by, low, less;
  __device__ Exponents(const Base& b, const Scale& k)
      : by(FINE ? b.hi : k.c, FINE ? b.hi : k.c), low(b.lo, b.lo), less(-b.M, -b.M) {}
  __device__ Two of(float a, float b) const {
    const Two z(a, b);
    return fma2(z, by, FINE ? fma2(z, low, less) : less);
  }
};

// 2^d for whole d <= 0, exactly (0 under 2^-126).
__device__ __forceinline__ float power_of(float d) {
  return d < -126.0f ? 0.0f : __int_as_float((127 + (int)d) << 23);
}

// What is kept of a part of a row: the largest z, the sum of its terms and, for an entropy, the sum of the
// terms times their exponents.
struct Part {
  float m, sum, ex;
  // The sum less what c's error has added to it relative to m's term, by its first derivative (of a part with
  // its entropy).
  __device__ float trimmed(const Scale& k) const {
    return __fmaf_rn(k.trim, ex - __fmul_rn(Base(m, k).below(k), sum), sum);
  }
};

// A part relative to a larger maximum m.
template <bool ENTROPY>
__device__ __forceinline__ Part rebased(const Part& p, float m, const Scale& k) {
  if (p.m == -INFINITY) return Part{m, p.sum, p.ex};
  const Base from(p.m, k), to(m, k);
  float down, by;
  if (from.whole && to.whole) {
    down = from.M - to.M;
    by = power_of(down);
  } else {
    down = from.whole ? __fmaf_rn(-to.m, k.c, from.M) : to.exponent<false>(from.m, k);
    by = exp2_fast(down);
  }
  Part r{m, __fmul_rn(p.sum, by), 0.0f};
  // every exponent falls by the same, kept finite: a term too small to be one has no part in it
  if (ENTROPY) r.ex = __fmul_rn(by, __fmaf_rn(p.sum, fmaxf(down, -1000.0f), p.ex));
  return r;
}

// One more term.
template <bool FINE, bool ENTROPY>
__device__ __forceinline__ void add_term(Part& p, const Base& base, const Scale& k, float z) {
  const float x = base.exponent<FINE>(z, k), t = exp2_fast(x);
  p.sum = __fadd_rn(p.sum, t);
  if (ENTROPY) p.ex = __fmaf_rn(t, fmaxf(x, -1000.0f), p.ex);  // (an exponent of -inf has no term)
}

// The terms of the words that `next` gives to what it is called with.
template <int DT, bool FINE, bool ENTROPY, class Next>
__device__ __forceinline__ void add_words(Part& p, const Base& base, const Scale& k, Next next) {
  using W = Word<DT>;
  constexpr int per = W::per;
  float f[per];
  if (base.whole) {
    const Exponents<FINE> exponents(base, k);
    Two sum(0.0f, 0.0f), ex(0.0f, 0.0f);
    next([&](uint4 u) {
      W::open(u, f);
#pragma unroll
      for (int j = 0; j < per; j += 2) {
        const Two x = exponents.of(f[j], f[j + 1]);
        const Two t(exp2_fast(x.lo()), exp2_fast(x.hi()));
        sum = add2(sum, t);
        if (ENTROPY) ex = fma2(t, Two(fmaxf(x.lo(), -1000.0f), fmaxf(x.hi(), -1000.0f)), ex);
      }
    });
    p.sum = __fadd_rn(p.sum, __fadd_rn(sum.lo(), sum.hi()));
    if (ENTROPY) p.ex = __fadd_rn(p.ex, __fadd_rn(ex.lo(), ex.hi()));
  } else {
    next([&](uint4 u) {
      W::open(u, f);
#pragma unroll
      for (int j = 0; j < per; ++j) add_term<FINE, ENTROPY>(p, base, k, f[j]);
    });
  }
}

// A row's place in memory: word 0 begins at the 16-byte boundary at or before its first value, so that
// every load is aligned whatever the row's stride. Words [first, last) are whole; before and behind
// them are under a word's worth of single values, each one thread's (`single`, -1 for none).
template <int DT>
struct RowWords {
  static constexpr int per = Word<DT>::per, es = 16 / per;
  const uint4* words;
  int lead, first, last, single;
  __device__ RowWords(const char* row, int n, int tid) {
    lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / es;
    words = reinterpret_cast<const uint4*>(row - lead * es);
    first = lead > 0 ? 1 : 0;
    last = (lead + n) / per;
    const int head = lead > 0 ? min(n, per - lead) : 0, behind = max(head, last * per - lead);
    single = tid < head ? tid : tid >= 8 && tid - 8 < n - behind ? behind + tid - 8 : -1;
  }
};

// A word with its value `at` replaced by -inf.
template <int DT>
__device__ __forceinline__ uint4 without(uint4 u, int at) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_F32) {
      if (at == i) w[i] = 0xFF800000u;
    } else {
      const uint32_t low = DT == DT_BF16 ? 0xFF80u : 0xFC00u;
      if (at == 2 * i) w[i] = (w[i] & 0xFFFF0000u) | low;
      if (at == 2 * i + 1) w[i] = (w[i] & 0xFFFFu) | low << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's part of a row that is read once, and kept nowhere; the value in column `chosen` (-1: none
// here) is left out of it.
template <int DT, bool FINE, bool ENTROPY>
__device__ __forceinline__ Part read_part(const RowWords<DT>& r, const char* row, int chosen, const Scale& k, int tid,
                                          int nthr) {
  using W = Word<DT>;
  constexpr int per = W::per, kOnce = 4;  // words on their way together
  Part p{-INFINITY, 0.0f, 0.0f};
  const int hole = chosen < 0 ? -1 : (r.lead + chosen) / per, at = (r.lead + chosen) % per;
  for (int j = r.first + tid; j < r.last; j += kOnce * nthr) {
    uint4 u[kOnce];
    uint32_t most = W::lowest();
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
      u[i] = j + i * nthr < r.last ? ld_row(r.words + j + i * nthr)
                                   : make_uint4(W::lowest(), W::lowest(), W::lowest(), W::lowest());
#pragma unroll
    for (int i = 0; i < kOnce; ++i) {
      if (j + i * nthr == hole) u[i] = without<DT>(u[i], at);
      most = W::larger(most, u[i]);
    }
    const float m = fmaxf(p.m, W::largest(most));
    if (m != p.m) p = rebased<ENTROPY>(p, m, k);
    p.m = m;
    add_words<DT, FINE, ENTROPY>(p, Base(m, k), k, [&](auto add) {
#pragma unroll
      for (int i = 0; i < kOnce; ++i) add(u[i]);
    });
  }
  if (r.single >= 0 && r.single != chosen) {
    const float z = load1<DT>(row, r.single), m = fmaxf(p.m, z);
    p = rebased<ENTROPY>(p, m, k);
    add_term<FINE, ENTROPY>(p, Base(m, k), k, z);
  }
  return p;
}

// The parts of all lanes of a warp as one, the same in each of them.
template <bool ENTROPY>
__device__ __forceinline__ Part join_warp(const Part& p, const Scale& k) {
  Part r = rebased<ENTROPY>(p, warp_max(p.m), k);
  r.sum = warp_sum(r.sum);
  if (ENTROPY) r.ex = warp_sum(r.ex);
  return r;
}

// What the blocks of a row's cluster tell each other: the parts of a block's warps, those of the blocks.
struct Parts {
  Part warp[32], block[8];
};

// The parts of all threads of a block, or of a cluster of C of them, as one, the same in each: each warp
// joins the warps' parts, and each block the blocks', in the same order. The cluster's blocks have
// arrived once before it (cluster_arrived).
template <bool ENTROPY, int C>
__device__ __forceinline__ Part join_all(const Part& mine, const Scale& k, Parts& sh, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Part w = join_warp<ENTROPY>(mine, k);
  if (lane == 0) sh.warp[warp] = w;
  __syncthreads();
  Part all = join_warp<ENTROPY>(lane < (int)(blockDim.x >> 5) ? sh.warp[lane] : Part{-INFINITY, 0.0f, 0.0f}, k);
  if constexpr (C > 1) {
    __syncwarp();
    cluster_wait();
    if (threadIdx.x < C) {
      const uint32_t to = cluster_addr(smem_u32(&sh.block[rank]), threadIdx.x);
      cluster_store(to, all.m);
      cluster_store(to + 4, all.sum);
      if (ENTROPY) cluster_store(to + 8, all.ex);
    }
    __syncwarp();
    cluster_sync();
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < C; ++r) m = fmaxf(m, sh.block[r].m);
    all = Part{m, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const Part b = rebased<ENTROPY>(sh.block[r], m, k);
      all.sum = __fadd_rn(all.sum, b.sum);
      if (ENTROPY) all.ex = __fadd_rn(all.ex, b.ex);
    }
  }
  return all;
}

// a + b, and what rounding has taken from it.
struct Pair {
  float value, rest;
};
__device__ __forceinline__ Pair exact_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  const Pair s = exact_sum(a.value, b.value);
  return Pair{s.value, s.rest + (a.rest + b.rest)};
}

// ln s in two words: with s = 2^k f and t = (f - 1)/(f + 1), k ln 2 + 2 (t + t^3/3 + t^5/5 + ...), of which k ln 2
// and 2 t are taken to twice 24 bits. One number's last half unit would be much the same for rows of much the
// same sum.
constexpr float kLn2Rest = -1.904654323148236e-9f;  // ln 2 less kLn2
__device__ __forceinline__ Pair log_pair(float s) {
  if (!(s > 1e-37f)) return Pair{logf(s), 0.0f};
  const int bits = __float_as_int(s), k = (bits - 0x3F3504F3) >> 23;  // f from about sqrt(1/2) to sqrt(2)
  const float f = __int_as_float(bits - (k << 23)), n = f - 1.0f;
  const Pair d = exact_sum(f, 1.0f);
  const float t = __fdiv_rn(n, d.value), t2 = __fmul_rn(t, t);
  const float t_rest = __fdiv_rn(__fmaf_rn(-t, d.value, n) - __fmul_rn(t, d.rest), d.value);
  float series = __fmaf_rn(t2, 2.0f / 11.0f, 2.0f / 9.0f);
  series = __fmaf_rn(t2, series, 2.0f / 7.0f);
  series = __fmaf_rn(t2, series, 2.0f / 5.0f);
  series = __fmaf_rn(t2, series, 2.0f / 3.0f);
  const float kf = (float)k, a = __fmul_rn(kf, kLn2);
  const Pair sum = exact_sum(a, 2.0f * t);
  const float low = __fmaf_rn(kf, kLn2Rest, __fmaf_rn(kf, kLn2, -a)) + 2.0f * t_rest;
  return Pair{sum.value, sum.rest + (low + __fmul_rn(__fmul_rn(t, t2), series))};
}

// log softmax at the chosen value z from the sum of all other terms, in two words. Where the chosen one has
// most of the sum, the sum's logarithm would keep nothing of the rest. Elsewhere it is z's exponent less the
// sum's logarithm: of fine exponents z c - M itself; of others the difference to m, which c's error leaves as
// it is. ex2.approx gives results that are too small by 5.0e-8 of themselves on average (as measured here over
// a million arguments in each of eight intervals), which the sum's logarithm gets back.
template <bool FINE>
__device__ __forceinline__ Pair log_chosen(float z, float rest, const Base& base, const Scale& k) {
  constexpr float kShort = 5.0e-8f;
  const float e = exp2_fast(base.exponent<FINE>(z, k));
  if (rest < e) return Pair{-log1pf(__fdiv_rn(rest, e)), 0.0f};
  const Pair log_sum = log_pair(rest + e);
  // So far under the maximum that the logarithm is nothing beside the difference, masked, or no number; halves, because
  // the difference of two that are far from zero may have no number of 32 bits where its share of tau has one.
  if (!(z - base.m > -1e30f))
    return Pair{__fdiv_rn(0.5f * z - 0.5f * base.m, 0.5f * k.tau) - log_sum.value, 0.0f};
  const float short_of = log_sum.rest + kShort;
  if (!(FINE && base.fine)) {
    const Pair d = exact_sum(__fdiv_rn(z - base.m, k.tau), -log_sum.value);
    return Pair{d.value, d.rest + __fmaf_rn(base.below(k), kLn2, -short_of)};
  }
  const float p = __fmul_rn(z, base.hi);
  const Pair x = exact_sum(p, -base.M);
  const Pair y = exact_sum(x.value, __fmaf_rn(z, base.lo, __fmaf_rn(z, base.hi, -p) + x.rest));
  const float q = __fmul_rn(y.value, kLn2), q_rest = __fmaf_rn(y.value, kLn2, -q);
  const Pair d = exact_sum(q, -log_sum.value);
  return Pair{d.value, d.rest + (__fmaf_rn(y.rest, kLn2, __fmaf_rn(y.value, kLn2Rest, q_rest)) - short_of)};
}

// Column ids of 4 or 8 bytes.
__device__ __forceinline__ int64_t id_at(const void* ids, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// How a launch shares rows out: the blocks of a row's cluster, each block's columns, how many blocks an SM
// has at once and the 16-byte words that each then holds, threads of a block.
struct RowShape {
  int split, blocks, room, threads;
  int64_t share;
};

// Rows that are held in shared memory while their gradient is not known. An SM's memory holds so many
// words of a row for each of its blocks; what a row has beyond them is read again, from L2. One block takes
// a row of up to 1.2 times what two blocks to an SM hold or of what one holds; longer rows go to as few
// blocks as have up to 1.2 times the half each. Where rows leave SMs free each is shared, as far as three
// blocks to an SM go and its parts stay 24 KB long (200 x 50257 fp32 in 18.6 us, 22.6 with one).
// One more block than fit whole where it nearly does: for a row of its own the second only, in a
// cluster, which waits more, others too. A thread has 20 words at most (8192 x 1000 fp32 in 13.8 us with 32
// blocks, 21.0 with 16).
inline RowShape held_rows(int64_t T, int64_t V, int es, int fixed, int sms) {
  auto held = [&](int blocks) { return ((kSmemMost + 1024) / blocks - 1024 - fixed) / 16; };
  const int unit = 16 / es;
  auto words = [&](int split) { return (V + split * unit - 1) / (split * unit) + 1; };  // 1: it may begin inside a word
  auto nearly = [&](int64_t n, int blocks) { return n * 5 <= (int64_t)held(blocks) * 6; };
  int split = 1;
  if (words(1) > held(1) && !nearly(words(1), 2))
    while (split < 8 && !nearly(words(split), 2)) split *= 2;
  while (split < 8 && T * split * 2 <= 3 * sms && words(split) > 3000) split *= 2;
  const int64_t room = words(split);
  RowShape r{};
  r.split = split;
  r.share = (room - 1) * unit;
  r.blocks = 1;
  while (r.blocks < 32 && T * split > (int64_t)r.blocks * sms && room <= 20 * (1024 / (r.blocks + 1) / 32 * 32) &&
         (room <= held(r.blocks + 1) || ((r.blocks == 1 || split > 1) && nearly(room, r.blocks + 1))))
    ++r.blocks;
  r.room = (int)(room < held(r.blocks) ? room : held(r.blocks));
  // They share the SM's registers, 64 a thread. A row that has its SM to itself takes fewer threads, as
  // barriers cost more than words then.
  r.threads = T * split <= sms ? 384 : 1024 / r.blocks / 32 * 32;
  if (r.threads > (room + 31) / 32 * 32) r.threads = (int)((room + 31) / 32 * 32);
  return r;
}

// Rows that are read as they come. A thread has about 16 words (8192 x 8000 bf16 in 25 us, 34 with 4), of rows that
// leave SMs free 4; those are shared by clusters as far as two blocks to an SM go and the parts stay 32 KB long
// (100 x 50257 fp32 in 7.0 us, 8.0 with one block to an SM).
inline RowShape streamed_rows(int64_t T, int64_t V, int es, int sms) {
  const int unit = 16 / es;
  auto words = [&](int split) { return (V + split * unit - 1) / (split * unit) + 1; };
  RowShape r{};
  r.split = 1;
  while (r.split < 8 && T * r.split <= sms && words(r.split) > 2000) r.split *= 2;
  const int64_t room = words(r.split);
  r.share = (room - 1) * unit;
  const int each = T * r.split <= 2 * sms ? 4 : 16, most = T * r.split <= 2 * sms ? 384 : 256;
  r.threads = (int)(room < each * most ? (room + each * 32 - 1) / (each * 32) * 32 : most);
  return r;
}

// ---- what the losses refuse alike
inline bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool finite(float x) { return x - x == 0.0f; }

inline zr_status check_logits(const char* what, zr_dtype dt, int64_t T, int64_t V, int64_t ldz, float temperature) {
  if (!dtype_ok(dt)) return fail(ZR_ERR_INVALID, "%s: bad dtype %d", what, (int)dt);
  if (T < 0 || V < 1 || V > 0x7FFFFF00)
    return fail(ZR_ERR_INVALID, "%s: T must be >= 0 and V in [1, 2^31 - 256]", what);
  if (ldz < V) return fail(ZR_ERR_INVALID, "%s: a row stride is under the row", what);
  if (!(temperature >= 1e-6f && temperature <= 1e6f))
    return fail(ZR_ERR_INVALID, "%s: temperature must lie in [1e-6, 1e6]", what);
  return ZR_OK;
}

// A gradient is the logits themselves, or lies apart from them.
inline zr_status check_gradient(const char* what, const void* logits, const void* grad, zr_dtype dt, int64_t T, int64_t V,
                                int64_t ldz, int64_t ldg) {
  if (!grad || (grad == logits && ldg == ldz)) return ZR_OK;
  const int es = dt == ZR_F32 ? 4 : 2;
  const __int128 z_bytes = ((__int128)(T - 1) * ldz + V) * es, g_bytes = ((__int128)(T - 1) * ldg + V) * es;
  const __int128 z = (__int128)reinterpret_cast<uintptr_t>(logits), g = (__int128)reinterpret_cast<uintptr_t>(grad);
  if (g < z + z_bytes && z < g + g_bytes)
    return fail(ZR_ERR_INVALID, "%s: grad overlaps the logits without being them", what);
  return ZR_OK;
}

}  // namespace zr
