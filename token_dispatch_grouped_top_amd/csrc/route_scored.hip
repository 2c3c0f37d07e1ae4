// route_scored.hip -- the scored route (softmax or sigmoid scores, balance
// bias, expert groups, renormalised weights), its backward and the update of
// the bias.
//
// The order of two experts is that of their choice values c = s + bias in
// fp64, because fp32 does not always tell them apart (about one batch of 16384
// tokens over 256 experts in four has a token that fp32 picks for differently).
// An fp64 exponential of every logit costs more than all the rest, so a token's
// experts go through two steps:
//   1. fp32 keys (c with a known error; without a bias the logits
//      themselves, whose order is the scores') find a value t0 that at least k
//      experts reach, and the candidates are those with a key of at least
//      t0 less twice the error: all that could be among the k largest c, seldom more than
//      k + 1;
//   2. the candidates, one to a lane, get c in fp64, and each counts the
//      candidates before it, by all bits of c and the lane, which is its place
//      among the picks.
// Groups are ranked by fp32 values; where the values at the border are nearer
// than their error, the groups' values are formed in fp64 (exact_groups).
// Where more candidates are left than lanes, the wave takes the plain way
// (exact_picks): fp64 for every expert and k rounds of argmax.  That is so with
// many equal logits; and as a lane keeps its four largest keys, with any logits
// where the open groups' lanes keep fewer than k in all (4 m top_groups < k, m the
// lanes of a group), and now and then where they keep little more.
// Reductions over lanes are of integers in the floats' order: one DPP
// instruction a level.
//
// Times over four sets of buffers in turn.  65536 tokens, 256 experts in 8 groups,
// 27.6 us: bound by the issue of vector instructions, 760 a wave of four tokens (a
// key takes 15, the rest is the same for any number of experts; the logits alone
// take 13 us at the rate of a large copy).  16384 tokens 11.2 us, of which 5.1 are
// issue, 3.3 the logits and 1.9 the launch, one after the other: four waves a SIMD
// start together and each loads, computes, stores.  384 experts without groups
// 11.9 and 34.9 us, 73728 tokens 38.5.  One token 4.1 us, half of it the launch.
// The plain way: 16384 tokens over 256 experts with all logits equal 53 us; over
// 512 in 8 groups, k = 12, four open 17.7 us, two 59 (some waves), one 100 (all).
// (A first version with an fp64 score of every logit, k rounds of argmax over 64
// lanes and an atomic for each pick took 174 us for 16384 tokens with their load.)
//
// Lanes.  A token has kL = 16 or 64 lanes.  Every group of experts gets m
// neighbouring lanes (the largest power of two with m G <= kL), each a run of
// `chunk` experts of its group, so that a group's value is a reduction over m
// lanes, a lane's experts are open or shut together, and experts in lane order
// are in id order.
#include <type_traits>

#include "scored_adamw.h"

namespace mok {

namespace {

constexpr int kWaves = 4;
constexpr float kNegInf = -__builtin_inff();
constexpr double kNegInf64 = -__builtin_inf();
// Error of an fp32 key.  Sigmoid, s = 1 / (1 + 2^(-x log2 e)): of e^-x the
// relative error |x| 1.25 2^-24 (the exponent) + 2^-23 (its power), of which
// s (1 - s) <= 1/4 and |x| s (1 - s) <= 0.23 reach s, of the sum and its
// reciprocal 1.5 2^-23: below 1.9 2^-23.  Softmax: |x| 2.25 2^-24 + 2^-22 of
// p <= 1, with p |x| <= 0.37: below 2.5 2^-23.  The sum with the bias adds 2^-24
// of itself (kRel, doubled).
constexpr float kSigmoidErr = 0x1p-22f, kSoftmaxErr = 0x1p-21f;
constexpr float kRel = 0x1p-23f;
constexpr float kLog2e = 1.44269504f;
// Tokens from which four share a wave, 16 lanes a token against 64 (us, buffers in
// turn).  Forward: 2048 tokens over 160 experts 4.55 and 5.0, 256 5.3 and 5.4, 384
// 4.8 and 5.0, 512 6.2 and 5.0; 16384 tokens 8.0 and 17.9, 10.5 and 19.7, 11.2 and
// 19.0, 16.1 and 19.2 (512 gain from 4096 tokens on).  Sparse backward, fp32: 256
// experts, 4096 tokens 3.6 and 3.5, 8192 4.6 and 4.9, 16384 7.3 and 8.6; 512
// experts 4.3 and 4.1, 6.9 and 6.7, 9.4 and 10.1.  Dense backward, fp32: 160
// experts, 16384 tokens 9.0 and 9.1, 32768 13.7 and 14.6, 65536 22.2 and 25.8; 256
// experts 10.8 and 9.7, 16.2 and 15.1, 32.6 and 35.2 (bf16 13.9 and 15.2 at 32768);
// above 256 experts 64 lanes are faster at every size: 384 experts 30.8 and 27.6 at
// 32768, 512 35.4 and 29.3.
constexpr int kManyTokens = 2048, kManySparse = 8192, kManyDense = 32768;
// Picks up to which each adds to the load by itself: about 1 ns a pick on the
// same few lines, against a second launch of 2.2 to 3 us.
constexpr int kDirectPicks = 2048;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* __restrict__ p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else
    return static_cast<const float*>(p)[i];
}

// NaN and -inf: not eligible (-inf); +inf: the largest finite value.
__device__ __forceinline__ float clean_logit(float l) {
  return l > kNegInf ? fminf(l, 3.402823466e38f) : kNegInf;
}

// Integers in the floats' order (zeros of either sign alike), and back.
__device__ __forceinline__ int key_of(float f) {
  const int b = __builtin_bit_cast(int, f + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_key(int k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kNoKey = static_cast<int>(0x807fffff);   // key_of(-inf)

// e^x for x <= 0 (and -inf: 0): 2^(x log2 e), the rounding of the exponent made good.
__device__ __forceinline__ float exp32(float x) {
  x = fmaxf(x, -256.0f);
  const float y = x * kLog2e;
  const float more = fmaf(x, kLog2e, -y) + x * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e, more * 0.693147181f, e);
}

__device__ __forceinline__ bool better(double v, int e, double bv, int be) {
  return v > bv || (v == bv && e < be);
}

// ------------------------------------------------- reductions over kL lanes
// Within a row of 16 lanes by DPP (xor 1, xor 2, i with 7 - i, i with 15 - i:
// each level's two sides are uniform in themselves); the four rows of a wave
// through scalars.  Every lane gets the result.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const int2 b = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(dpp<CTRL>(b.x), dpp<CTRL>(b.y)));
}
constexpr int kX1 = 0xB1, kX2 = 0x4E, kX4 = 0x141, kX8 = 0x140;   // quad_perm, row_half_mirror, row_mirror

__device__ __forceinline__ float lane_value(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ int lane_value(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double lane_value(double v, int l) {
  const int2 b = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(b.x, l), __builtin_amdgcn_readlane(b.y, l)));
}

template <int kL, class T, class F>
__device__ __forceinline__ T reduce(T v, F f) {
  v = f(v, dpp<kX1>(v));
  v = f(v, dpp<kX2>(v));
  v = f(v, dpp<kX4>(v));
  v = f(v, dpp<kX8>(v));
  if constexpr (kL == 64)
    v = f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
  return v;
}
struct MaxI { __device__ __forceinline__ int operator()(int a, int b) const { return a > b ? a : b; } };
struct MinI { __device__ __forceinline__ int operator()(int a, int b) const { return a < b ? a : b; } };
struct MaxF { __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct Add { template <class T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; } };

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// The picks' shares u: `valid` lanes hold the logits l of the picks (one at
// least in each token that has any); the other lanes get 0.  sigmoid: s / sum
// s, formed from exp(l) where every s is as small as exp(l) itself (below
// e^-60), so that nothing underflows.  softmax: exp(l - max) / sum.
template <int kL>
__device__ __forceinline__ double share(bool valid, float l, bool sigmoid, double s) {
  const float lmax = reduce<kL>(valid ? l : kNegInf, MaxF());
  double a = s;
  if (!sigmoid || lmax <= -60.0f) a = exp(static_cast<double>(l) - static_cast<double>(lmax));
  a = valid ? a : 0.0;
  const double sum = reduce<kL>(a, Add());
  return valid ? a / sum : 0.0;
}

// One token's row as its lanes see it.
struct Row {
  int sl;         // lane within the token
  int g, part;    // its group, and its run in the group
  int first, n;   // its experts [first, first + n)
};

template <int kL>
__device__ __forceinline__ Row row_of(const RouterArgs& r, int lane) {
  Row o;
  o.sl = lane & (kL - 1);
  o.g = o.sl >> r.log_m;
  o.part = o.sl & ((1 << r.log_m) - 1);
  const int from = o.part * r.chunk;
  o.first = o.g * r.gsize + from;
  o.n = o.g < r.G && from < r.gsize ? (r.gsize - from < r.chunk ? r.gsize - from : r.chunk) : 0;
  return o;
}

// Largest and second largest of the m lanes of each group, in every lane.
template <class T, class F>
__device__ __forceinline__ void merge_top2(T& a, T& b, int log_m, F max2) {
  auto step = [&](T oa, T ob) {
    const T lo = oa < a ? oa : a;
    a = max2(a, oa);
    b = max2(lo, max2(b, ob));
  };
  if (log_m > 0) step(dpp<kX1>(a), dpp<kX1>(b));
  if (log_m > 1) step(dpp<kX2>(a), dpp<kX2>(b));
  if (log_m > 2) step(dpp<kX4>(a), dpp<kX4>(b));
  if (log_m > 3) step(dpp<kX8>(a), dpp<kX8>(b));
  if (log_m > 4) step(__shfl_xor(a, 16), __shfl_xor(b, 16));
}

// The plain way, for every token of the wave: c in fp64 for every expert, group
// values in fp64, k rounds of argmax.  Returns the pick of rank sl, or -1.
template <int kL, int V, bool BF16>
__device__ __forceinline__ int exact_picks(const RouterArgs& r, const void* __restrict__ logits,
                                           int64_t at, const float* __restrict__ bias, float top) {
  const int lane = lane_id();
  const Row w = row_of<kL>(r, lane);
  double c[V], sum = 0.0;                  // the logits are read again: registers
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float l = i < w.n ? clean_logit(load_logit<BF16>(logits, at + w.first + i)) : kNegInf;
    c[i] = kNegInf64;
    if (l > kNegInf) {
      c[i] = static_cast<double>(l);
      if (bias && !r.sigmoid) sum += exp(c[i] - static_cast<double>(top));
    }
  }
  sum = reduce<kL>(sum, Add());
  auto score = [&](double x) {             // without a bias exp(x - top): a common factor orders nothing
    const double s = r.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(top));
    return bias && !r.sigmoid ? s / sum : s;
  };
  if (bias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] > kNegInf64) c[i] = score(c[i]) + static_cast<double>(bias[w.first + i]);
  }
  if (r.G > 1) {
    double a = kNegInf64, b = kNegInf64;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b = c[i] > a ? a : (c[i] > b ? c[i] : b);
      a = c[i] > a ? c[i] : a;
    }
    merge_top2(a, b, r.log_m, [](double x, double y) { return x > y ? x : y; });
    if (r.top2 && !bias) {
      a = a > kNegInf64 ? score(a) : a;
      b = b > kNegInf64 ? score(b) : b;
    }
    const double gv = r.top2 && b > kNegInf64 ? a + b : a;
    int rank = 0;
    for (int g = 0; g < r.G; ++g) {
      const double ov = __shfl(gv, (lane & ~(kL - 1)) + (g << r.log_m));
      rank += better(ov, g, gv, w.g) ? 1 : 0;
    }
    if (rank >= r.top_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = kNegInf64;
    }
  }
  int mine = -1;
  for (int j = 0; j < r.k; ++j) {
    double bv = kNegInf64;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] > bv) { bv = c[i]; be = w.first + i; }
#pragma unroll
    for (int o = 1; o < kL; o <<= 1) {
      const double ov = __shfl_xor(bv, o);
      const int oe = __shfl_xor(be, o);
      if (better(ov, oe, bv, be)) { bv = ov; be = oe; }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (w.first + i == be) c[i] = kNegInf64;
    if (w.sl == j && bv > kNegInf64) mine = be;
  }
  return mine;
}

// How many of lanes [kFrom, kTo) of the token's row of 16 come before this one by
// (value, lane).  Both launches of 16384 tokens over 256 experts with load 12.8 us,
// 65536 over 256 22.9, 73728 over 384 36.8; with 15 rotations in place of the lanes
// that hold a candidate 13.05, 23.6 and 37.7 (keys, without a bias: 65536 over 256
// 19.0 and 19.4).
template <int kFrom, int kTo, class T>
__device__ __forceinline__ int count_of16(T v, int sl) {
  if constexpr (kFrom == kTo) {
    return 0;
  } else {
    const T o = dpp<0x150 + kFrom>(v);                    // row_newbcast:kFrom
    return ((o > v) | ((o == v) & (sl > kFrom)) ? 1 : 0) + count_of16<kFrom + 1, kTo>(v, sl);
  }
}

// Groups before this lane's by (value, id), where every lane holds its group's
// value and kM lanes are a group: rotations by whole groups.  The source of
// row_ror:R is below lane sl if sl >= R.
template <int kM, int R>
__device__ __forceinline__ int groups_before16(int own, int sl) {
  if constexpr (R >= 16) return 0;
  else return (dpp<0x120 + R>(own) > own - (sl >= R ? 1 : 0) ? 1 : 0) + groups_before16<kM, R + kM>(own, sl);
}

// Whether the lane's group is among the top_groups, from values in fp64 of the
// experts whose keys could be its two largest.  Every lane of the wave calls it.
template <int kL, int V, bool BF16>
__device__ __forceinline__ bool exact_groups(const RouterArgs& r, const Row& w, const void* __restrict__ logits,
                                             int64_t at, const float* __restrict__ bias, float top,
                                             double inv, const float (&c)[V], int ga, int gb) {
  const int lane = lane_id();
  auto score = [&](double x) {
    return r.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(top)) * inv;
  };
  double a = kNegInf64, b = kNegInf64;
  if (bias) {
    const float low = of_key(r.top2 && gb > kNoKey ? gb : ga);
    const float from = low - 2.0f * ((r.sigmoid ? kSigmoidErr : kSoftmaxErr) + kRel * fabsf(low));
    // a lane's few, one a turn (the largest V in passes of 32)
#pragma unroll
    for (int i0 = 0; i0 < V; i0 += 32) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = i0; i < V && i < i0 + 32; ++i)
        if (c[i] >= from && c[i] > kNegInf) bits |= 1u << (i - i0);
      while (bits) {
        const int e = w.first + i0 + __ffs(static_cast<int>(bits)) - 1;
        bits &= bits - 1;
        const double x = score(static_cast<double>(clean_logit(load_logit<BF16>(logits, at + e)))) +
                         static_cast<double>(bias[e]);
        b = x > a ? a : (x > b ? x : b);
        a = x > a ? x : a;
      }
    }
    merge_top2(a, b, r.log_m, [](double x, double y) { return x > y ? x : y; });
  } else {                       // keys are logits: these are the two
    if (ga > kNoKey) a = score(static_cast<double>(of_key(ga)));
    if (gb > kNoKey) b = score(static_cast<double>(of_key(gb)));
  }
  const double gv = r.top2 && b > kNegInf64 ? a + b : a;
  int rank = 0;
  for (int g = 0; g < r.G; ++g) {
    const double ov = __shfl(gv, (lane & ~(kL - 1)) + (g << r.log_m));
    rank += better(ov, g, gv, w.g) ? 1 : 0;
  }
  return rank < r.top_groups;
}

template <int kL, int V, bool BF16>
__global__ __launch_bounds__(kWaves * kWave)
void k_route_scored(RouterArgs r, const void* __restrict__ logits, int64_t ld,
                    const float* __restrict__ bias, int32_t T, int32_t* __restrict__ idx,
                    float* __restrict__ gate, int32_t* __restrict__ load, RouteCount rc) {
  constexpr int kTok = kWave / kL;                      // tokens of a wave
  // a candidate: its id, and for few tokens, where a second read's latency counts, its logit and bias
  constexpr bool kCarry = kL == 64 && V <= 16;
  using Slot = typename std::conditional<kCarry, float4, uint16_t>::type;
  __shared__ Slot slots[kWaves][kTok][kL];
  const int lane = lane_id(), wave = threadIdx.x / kWave, sub = lane / kL;
  const Row w = row_of<kL>(r, lane);
  const int64_t t_mine = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTok + sub;
  const bool live = t_mine < T;
  const int64_t t = live ? t_mine : T - 1;              // a wave's spare lanes repeat the last token
  const int64_t at = t * ld;
  float l[V];
  if (r.wide) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float4 q = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
      if (i < w.n) {
        if constexpr (BF16) {
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + at + w.first + i);
          q = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                          __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
        } else {
          q = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + at + w.first + i);
        }
      }
      l[i] = q.x; l[i + 1] = q.y; l[i + 2] = q.z; l[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < w.n ? load_logit<BF16>(logits, at + w.first + i) : kNegInf;
  }
  float bv[V];
  if (bias) {
    if (r.wide && r.wide_bias) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < w.n) q = *reinterpret_cast<const float4*>(bias + w.first + i);
        bv[i] = q.x; bv[i + 1] = q.y; bv[i + 2] = q.z; bv[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) bv[i] = i < w.n ? bias[w.first + i] : 0.0f;
    }
  }
  if (!(bias && r.sigmoid)) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = clean_logit(l[i]);
  }

  // softmax: the row's largest logit and its sum (fp64 where the order needs it)
  float top = 0.0f;
  double inv = 1.0;
  if (!r.sigmoid) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    top = of_key(reduce<kL>(key_of(m), MaxI()));
    if (bias) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l[i] > kNegInf) sum += exp(static_cast<double>(l[i]) - static_cast<double>(top));
      sum = reduce<kL>(sum, Add());
      inv = sum > 0.0 ? 1.0 / sum : 0.0;
    } else if (!r.renorm) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] > kNegInf ? exp32(l[i] - top) : 0.0f;
      sum = reduce<kL>(sum, Add());
      inv = sum > 0.0f ? 1.0 / static_cast<double>(sum) : 0.0;
    }
  }
  const float inv32 = static_cast<float>(inv);
  auto sigmoid32 = [](float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
  };
  auto softmax32 = [&](float x) { return __builtin_amdgcn_exp2f(kLog2e * (x - top)) * inv32; };

  // keys, and the four largest of the lane's
  float c[V], f1 = kNegInf, f2 = kNegInf, f3 = kNegInf, f4 = kNegInf;
  if (!bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  } else if (r.sigmoid) {                    // +inf: 1, NaN and -inf: shut
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] > kNegInf ? sigmoid32(l[i]) + bv[i] : kNegInf;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] > kNegInf ? softmax32(l[i]) + bv[i] : kNegInf;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f4 = __builtin_amdgcn_fmed3f(f3, f4, c[i]);
    f3 = __builtin_amdgcn_fmed3f(f2, f3, c[i]);
    f2 = __builtin_amdgcn_fmed3f(f1, f2, c[i]);
    f1 = c[i] > f1 ? c[i] : f1;
  }
  int a1 = key_of(f1), a2 = key_of(f2), a3 = key_of(f3), a4 = key_of(f4);

  const float delta = r.sigmoid ? kSigmoidErr : kSoftmaxErr;
  bool open = w.n > 0;
  if (r.G > 1) {
    int ga = a1, gb = a2;
    merge_top2(ga, gb, r.log_m, MaxI());
    const float fa = of_key(ga);
    float gv = fa, err = bias ? delta + kRel * fabsf(fa) : 0.0f;
    if (r.top2) {
      float fb = of_key(gb);
      if (!bias) {               // keys are logits: the sum is of scores
        gv = ga > kNoKey ? (r.sigmoid ? sigmoid32(fa) : softmax32(fa)) : kNegInf;
        fb = gb > kNoKey ? (r.sigmoid ? sigmoid32(fb) : softmax32(fb)) : kNegInf;
      }
      if (gb > kNoKey) gv += fb;
      err = 2.0f * delta + 2.0f * kRel * (bias ? fabsf(fa) + (gb > kNoKey ? fabsf(fb) : 0.0f) : gv);
      // without a bias the relative error counts too, below 2^-16 for |x| < 104 (and 2^-120 for
      // exponentials that leave the normal numbers)
      if (!bias) err = fminf(err, 0x1p-16f * gv) + 0x1p-120f;
    }
    const bool counts = w.g < r.G && ga > kNoKey;
    const int gk = counts ? key_of(gv) : kNoKey;
    int before = 0;
    if constexpr (kL == 16) {
      if (r.log_m == 0) before = groups_before16<1, 1>(gk, w.sl);
      else if (r.log_m == 1) before = groups_before16<2, 2>(gk, w.sl);
      else if (r.log_m == 2) before = groups_before16<4, 4>(gk, w.sl);
      else before = groups_before16<8, 8>(gk, w.sl);
    } else {
      for (int g = 0; g < r.G; ++g) {
        const int o = lane_value(gk, g << r.log_m);
        before += o > gk || (o == gk && g < w.g) ? 1 : 0;
      }
    }
    bool chosen = counts && before < r.top_groups;
    if (bias || r.top2) {
      const int last = reduce<kL>(chosen ? key_of(gv - err) : 0x7fffffff, MinI());
      const int next = reduce<kL>(!chosen && counts ? key_of(gv + err) : kNoKey, MaxI());
      const bool near = next > kNoKey && next >= last;
      if (__ballot(near)) {
        const bool sure = exact_groups<kL, V, BF16>(r, w, logits, at, bias, top, inv, c, ga, gb);
        chosen = near ? sure : chosen;
      }
    }
    open = open && chosen;
    if (!open) a1 = a2 = a3 = a4 = kNoKey;
  }

  // t0: after k rounds of taking the largest heads off, at least k keys were >= it
  int t0 = kNoKey;
  for (int j = 0; j < r.k; ++j) {
    t0 = reduce<kL>(a1, MaxI());
    const bool off = a1 == t0;
    a1 = off ? a2 : a1;
    a2 = off ? a3 : a2;
    a3 = off ? a4 : a3;
    a4 = off ? kNoKey : a4;
  }
  int thr = t0;
  if (bias && t0 > kNoKey) {
    const float f = of_key(t0);
    thr = key_of(f - 2.0f * (delta + kRel * fabsf(f)));
  }
  // every eligible expert, where k are not there (the lowest finite value); none of a shut group
  const float from = open ? of_key(thr > kNoKey ? thr : kNoKey + 1) : __builtin_inff();

  // candidates, in id order
  uint32_t bits = 0;                                    // kL = 16: element i at bit V - 1 - i
  int have = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (kL == 16) bits = bits + bits + (c[i] >= from ? 1u : 0u);
    else have += c[i] >= from ? 1 : 0;
  }
  if constexpr (kL == 16) have = __popc(bits);
  int slot = have;                                      // inclusive prefix over the token's lanes
  slot += dpp<0x111>(slot);                             // row_shr:1, 2, 4, 8 (0 from outside)
  slot += dpp<0x112>(slot);
  slot += dpp<0x114>(slot);
  slot += dpp<0x118>(slot);
  int n_cand;
  if constexpr (kL == 16) {
    n_cand = reduce<16>(slot, MaxI());
  } else {
    const int r0 = lane_value(slot, 15), r1 = lane_value(slot, 31), r2 = lane_value(slot, 47);
    const int row = lane >> 4;
    slot += (row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0);
    n_cand = lane_value(slot, 63);
  }
  slot -= have;
  Slot* mine = slots[wave][sub];
  if constexpr (kL == 16) {
    bits <<= 32 - V;                                    // the lowest id at the top
    while (bits) {
      const int i = __clz(static_cast<int>(bits));
      bits &= ~(0x80000000u >> i);
      if (slot < kL) mine[slot] = static_cast<uint16_t>(w.first + i);
      ++slot;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] >= from) {
        if (slot < kL) {
          if constexpr (kCarry) mine[slot] = make_float4(l[i], bias ? bv[i] : 0.0f, __int_as_float(w.first + i), 0.0f);
          else mine[slot] = static_cast<uint16_t>(w.first + i);
        }
        ++slot;
      }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const bool plain = n_cand > kL;

  // fp64 values of the candidates, one to a lane, and their places
  int e = -1, place = w.sl;
  float le = kNegInf, be = 0.0f;
  double s = 0.0;
  const auto read = [&]() {                 // the logit and bias of expert e
    le = e >= 0 ? clean_logit(load_logit<BF16>(logits, at + e)) : kNegInf;
    be = bias && e >= 0 ? bias[e] : 0.0f;
  };
  const auto score64 = [&]() {
    s = 0.0;
    if (e >= 0)
      s = r.sigmoid ? sigmoid64(le) : exp(static_cast<double>(le) - static_cast<double>(top)) * inv;
  };
  if constexpr (!kCarry) {
    if (!plain && w.sl < n_cand) e = mine[w.sl];
    read();
  } else if (!plain && w.sl < n_cand) {
    const float4 q = mine[w.sl];
    le = clean_logit(q.x);
    be = q.y;
    e = __float_as_int(q.z);
  }
  score64();
  {
    double v = kNegInf64;
    if (e >= 0) v = bias ? s + static_cast<double>(be) : static_cast<double>(le);
    // all bits of v count; equal values in id order, which is lane order
    if constexpr (kL == 16) {
      const uint64_t any = __ballot(e >= 0);              // seldom many more candidates than k
      const auto count = [&](auto x) {
        int n = count_of16<0, 8>(x, w.sl);
        if (any & 0xff00ff00ff00ff00ull) n += count_of16<8, 12>(x, w.sl);
        if (any & 0xf000f000f000f000ull) n += count_of16<12, 16>(x, w.sl);
        return n;
      };
      place = bias ? count(v) : count(key_of(le));
    } else {
      place = 0;
      const int n = n_cand < kL ? n_cand : kL;
      for (int j = 0; j < n; ++j) {
        const double o = lane_value(v, j);
        place += (o > v) | ((o == v) & (j < w.sl)) ? 1 : 0;
      }
    }
  }
  if (__ballot(plain)) {
    const int pe = exact_picks<kL, V, BF16>(r, logits, at, bias, top);
    if (plain) {
      e = pe;
      place = w.sl;
      read();
      score64();
    }
  }
  const bool valid = e >= 0 && place < r.k;
  if (r.renorm) s = share<kL>(valid, le, r.sigmoid, s);
  if (!live) return;
  const int64_t to = t * r.k;
  if (valid) {
    idx[to + place] = e;
    gate[to + place] = static_cast<float>(static_cast<double>(r.scale) * s);
    if (load) __hip_atomic_fetch_add(load + e, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the fused layer's schedule counts
    const int local = e - rc.base;
    if (rc.blk_counts && local >= 0 && local < rc.n_local)
      __hip_atomic_fetch_add(rc.blk_counts + static_cast<int64_t>(local) * rc.nblk +
                                 (to + place) / kSchedChunk,
                             1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else if (e < 0 && w.sl < r.k) {           // fewer candidates than k: the places behind them
    idx[to + w.sl] = -1;
    gate[to + w.sl] = 0.0f;
  }
}

// The load of many picks: a workgroup counts its share in LDS and adds each
// expert's count once: 131072 picks of 256 experts in 2.6 us (one atomic a pick:
// 130 us).
constexpr int kLoadThreads = 1024, kLoadPicks = 4 * kLoadThreads;

__global__ __launch_bounds__(kLoadThreads)
void k_load_count(const int32_t* __restrict__ idx, int64_t n, int32_t E, int32_t* __restrict__ load) {
  __shared__ int32_t hist[4096];
  for (int e = threadIdx.x; e < E; e += kLoadThreads) hist[e] = 0;
  __syncthreads();
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kLoadPicks; i0 < n;
       i0 += static_cast<int64_t>(gridDim.x) * kLoadPicks) {
    int e[kLoadPicks / kLoadThreads];
#pragma unroll
    for (int j = 0; j < kLoadPicks / kLoadThreads; ++j) {
      const int64_t i = i0 + j * kLoadThreads + threadIdx.x;
      e[j] = i < n ? idx[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < kLoadPicks / kLoadThreads; ++j)
      if (e[j] >= 0) atomicAdd(&hist[e[j]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kLoadThreads)
    if (hist[e]) __hip_atomic_fetch_add(load + e, hist[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The backward.  Lane j of a token has its pick j; the token's row lies in LDS,
// zero but for what the picks put there, and is written from there in whole
// 16-byte pieces: the sparse gradients (V = 0) are the picks' own.  Dense
// (softmax without renorm): with the picks' weights w in the row,
//   D = sum_e s_e w_e,  dl_e = s_e (w_e - D),
// the logits in registers, V of them to a lane, four neighbours at a time.
// Bound by the row's write (and for the dense form its read).  Buffers in turn,
// 256 experts: 16384 tokens sparse 7.4 us in fp32, 6.1 in bf16, dense 9.9 and 9.6;
// 65536 sparse 25.5 us, dense 31.2.  Zeros written before the picks' values instead
// of a row in LDS, over the same buffers again and again: 3.6 us where this takes
// 3.7 at 4096 tokens, 19.7 where it takes 18.1 at 65536.
template <int kL, int V, bool BF16>
__global__ __launch_bounds__(kWaves * kWave)
void k_route_scored_bwd(RouterArgs r, const void* __restrict__ logits, int64_t ld, int32_t T,
                        const int32_t* __restrict__ idx, const float* __restrict__ dgate,
                        void* __restrict__ dlogits, int64_t ldd, bool wide_in, bool wide_out) {
  extern __shared__ float rows[];                       // [kWaves][tokens][E, a multiple of 4]
  constexpr int kTok = kWave / kL;
  const int lane = lane_id(), wave = threadIdx.x / kWave, sub = lane / kL, sl = lane & (kL - 1);
  const int E = r.E, Ep = (E + 3) & ~3;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTok;
  if (t0 >= T) return;
  const int64_t t = t0 + sub < T ? t0 + sub : T - 1;
  float* row = rows + (wave * kTok + sub) * Ep;
  const auto fence = []() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };

  int e = sl < r.k ? idx[t * r.k + sl] : -1;
  if (e < 0 || e >= E) e = -1;
  float x = e >= 0 ? r.scale * dgate[t * r.k + sl] : 0.0f;
  float lv[V > 0 ? V : 1];
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int c = i * kL + 4 * sl;
      float4 q = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
      if (wide_in) {
        if (c < E) {
          if constexpr (BF16) {
            const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + t * ld + c);
            q = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                            __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
          } else {
            q = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + t * ld + c);
          }
        }
      } else {
        if (c < E) q.x = load_logit<BF16>(logits, t * ld + c);
        if (c + 1 < E) q.y = load_logit<BF16>(logits, t * ld + c + 1);
        if (c + 2 < E) q.z = load_logit<BF16>(logits, t * ld + c + 2);
        if (c + 3 < E) q.w = load_logit<BF16>(logits, t * ld + c + 3);
      }
      lv[i] = clean_logit(q.x); lv[i + 1] = clean_logit(q.y);
      lv[i + 2] = clean_logit(q.z); lv[i + 3] = clean_logit(q.w);
    }
  }
  for (int c = 4 * sl; c < Ep; c += 4 * kL)
    *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

  if constexpr (V == 0) {
    const float l = e >= 0 ? clean_logit(load_logit<BF16>(logits, t * ld + e)) : kNegInf;
    if (!(l > kNegInf)) {
      e = -1;
      x = 0.0f;
    }
    const bool valid = e >= 0;
    float s = 0.0f, not_s = 1.0f, big = 1.0f;
    if (r.sigmoid) {
      const float ex = exp32(-fabsf(l));                // of the smaller of s and 1 - s
      big = 1.0f / (1.0f + ex);
      const float small = ex * big;
      s = l > 0.0f ? big : small;
      not_s = l > 0.0f ? small : big;
    }
    if (r.renorm) {
      const float lmax = of_key(reduce<kL>(valid ? key_of(l) : kNoKey, MaxI()));
      // shares from exp(l - max); sigmoid: s = e^l / (1 + e^l), so that no s leaves the normal
      // numbers while its share does not
      float a = s;
      if (!r.sigmoid || lmax <= 0.0f) a = exp32(l - lmax) * big;
      a = valid ? a : 0.0f;
      const float sum = reduce<kL>(a, Add());
      const float u = valid ? a / sum : 0.0f;
      x = u * not_s * (x - reduce<kL>(x * u, Add()));
    } else {
      x = s * not_s * x;
    }
    x = valid ? x : 0.0f;
  }

  // the picks into the row: each writes its lane and looks whether another was there
  const bool valid = e >= 0;
  fence();
  if (valid) row[e] = __int_as_float(sl);
  fence();
  const bool twice = valid && __float_as_int(row[e]) != sl;
  fence();
  if (__ballot(twice) == 0) {
    if (valid) row[e] = x;
  } else {                                              // an id twice: added in the picks' order
    if (valid) row[e] = 0.0f;
    fence();
    for (int j = 0; j < r.k; ++j) {
      if (valid && sl == j) row[e] += x;
      fence();
    }
  }
  fence();
  __builtin_amdgcn_wave_barrier();

  if constexpr (V > 0) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, lv[i]);
    const float top = of_key(reduce<kL>(key_of(m), MaxI()));
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int c = i * kL + 4 * sl;
      const float4 w = c < Ep ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = lv[i + j] > kNegInf ? exp32(lv[i + j] - top) : 0.0f;
        sum += p;
        dot += lv[i + j] > kNegInf ? p * wv[j] : 0.0f;
        lv[i + j] = lv[i + j] > kNegInf ? p : -1.0f;    // not eligible: no gradient
      }
    }
    sum = reduce<kL>(sum, Add());
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float D = reduce<kL>(dot, Add()) * inv;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int c = i * kL + 4 * sl;
      if (c >= Ep) continue;
      const float4 w = *reinterpret_cast<const float4*>(row + c);
      const float4 o = make_float4(lv[i] >= 0.0f ? lv[i] * inv * (w.x - D) : 0.0f,
                                   lv[i + 1] >= 0.0f ? lv[i + 1] * inv * (w.y - D) : 0.0f,
                                   lv[i + 2] >= 0.0f ? lv[i + 2] * inv * (w.z - D) : 0.0f,
                                   lv[i + 3] >= 0.0f ? lv[i + 3] * inv * (w.w - D) : 0.0f);
      *reinterpret_cast<float4*>(row + c) = o;
    }
    fence();
    __builtin_amdgcn_wave_barrier();
  }

#pragma unroll
  for (int u = 0; u < kTok; ++u) {
    if (t0 + u >= T) break;
    const float* from = rows + (wave * kTok + u) * Ep;
    const int64_t to = (t0 + u) * ldd;
    if (wide_out) {
      for (int c = 4 * lane; c < E; c += 4 * kWave) {
        const float4 q = *reinterpret_cast<const float4*>(from + c);
        if constexpr (BF16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + to + c) =
              make_uint2(pack_bf16x2(q.x, q.y), pack_bf16x2(q.z, q.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(dlogits) + to + c) = q;
      }
    } else {
      for (int c = lane; c < E; c += kWave) {
        if constexpr (BF16) static_cast<uint16_t*>(dlogits)[to + c] = f32_to_bf16(from[c]);
        else static_cast<float*>(dlogits)[to + c] = from[c];
      }
    }
  }
}

// The bias update: one workgroup per layer, an expert to a thread as far as
// 1024 threads go.  The load's sum in 64-bit integers, then the bias.  Bound by
// latency: 1.9 us for one layer of 384 experts, 3.5 us for 60 of 1000.
constexpr int kBiasThreads = 1024;

__global__ __launch_bounds__(kBiasThreads)
void k_bias_update(int32_t* __restrict__ load, int32_t E, float rate, float* __restrict__ bias,
                   int32_t clear_load) {
  __shared__ int64_t part[kBiasThreads / kWave];
  load += static_cast<int64_t>(blockIdx.x) * E;
  bias += static_cast<int64_t>(blockIdx.x) * E;
  const int n = blockDim.x, first = threadIdx.x;
  const int32_t mine = first < E ? load[first] : 0;
  const float old = first < E ? bias[first] : 0.0f;
  int64_t sum = mine;
  for (int e = first + n; e < E; e += n) sum += load[e];
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o);
  if (lane_id() == 0) part[first / kWave] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < n / kWave; ++w) sum += part[w];
  for (int e = first; e < E; e += n) {
    const int64_t d = sum - static_cast<int64_t>(E) * (e == first ? mine : load[e]);
    const float b = e == first ? old : bias[e];
    bias[e] = b + (d > 0 ? rate : d < 0 ? -rate : 0.0f);
    if (clear_load) load[e] = 0;
  }
}

template <int kL, int V>
hipError_t launch_scored_v(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                           const float* bias, int32_t T, int32_t* idx, float* gate, int32_t* load,
                           const RouteCount& rc, hipStream_t s) {
  constexpr int kTok = kWaves * (kWave / kL);           // tokens of a workgroup
  const dim3 grid((T + kTok - 1) / kTok), block(kWaves * kWave);
  const int64_t picks = static_cast<int64_t>(T) * r.k;
  int32_t* direct = picks <= kDirectPicks ? load : nullptr;
  if (bf16)
    hipLaunchKernelGGL((k_route_scored<kL, V, true>), grid, block, 0, s, r, logits, ld, bias, T,
                       idx, gate, direct, rc);
  else
    hipLaunchKernelGGL((k_route_scored<kL, V, false>), grid, block, 0, s, r, logits, ld, bias, T,
                       idx, gate, direct, rc);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && load && !direct) {
    const int64_t blocks = (picks + kLoadPicks - 1) / kLoadPicks;
    hipLaunchKernelGGL(k_load_count, dim3(blocks < 64 ? blocks : 64), dim3(kLoadThreads), 0, s, idx,
                       picks, r.E, load);
    e = hipGetLastError();
  }
  return e;
}

// The split of a row over kL lanes; false: not possible within max_chunk.
bool split_row(RouterArgs& r, int kL, int max_chunk) {
  if (r.G > kL) return false;
  r.log_m = 0;
  while ((r.G << (r.log_m + 1)) <= kL) ++r.log_m;
  const int m = 1 << r.log_m;
  r.chunk = (r.gsize + m - 1) / m;
  if (r.chunk % 4 != 0 && r.gsize % 4 == 0 && (r.chunk + 3) / 4 * 4 <= max_chunk)
    r.chunk = (r.chunk + 3) / 4 * 4;                    // runs of whole 16-byte loads
  return r.chunk <= max_chunk;
}

template <int kL, int V>
hipError_t launch_bwd_v(const RouterArgs& r, const void* logits, bool bf16, int64_t ld, int32_t T,
                        const int32_t* idx, const float* dgate, void* dlogits, int64_t ldd,
                        hipStream_t s) {
  constexpr int kTok = kWaves * (kWave / kL);
  const dim3 grid((T + kTok - 1) / kTok), block(kWaves * kWave);
  const size_t lds = static_cast<size_t>(kTok) * ((r.E + 3) & ~3) * sizeof(float);
  const uintptr_t bytes = bf16 ? 8 : 16;
  const bool in = r.E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % bytes == 0;
  const bool out = r.E % 4 == 0 && ldd % 4 == 0 && reinterpret_cast<uintptr_t>(dlogits) % bytes == 0;
  if (bf16)
    hipLaunchKernelGGL((k_route_scored_bwd<kL, V, true>), grid, block, lds, s, r, logits, ld, T, idx,
                       dgate, dlogits, ldd, in, out);
  else
    hipLaunchKernelGGL((k_route_scored_bwd<kL, V, false>), grid, block, lds, s, r, logits, ld, T, idx,
                       dgate, dlogits, ldd, in, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouterArgs& router, const void* logits, bool bf16, int64_t ld,
                               const float* bias, int32_t T, int32_t* idx, float* gate,
                               int32_t* load, const RouteCount& rc, hipStream_t s) {
  if (T == 0) return hipSuccess;
  RouterArgs r = router;
  const auto wide = [&]() {
    const uintptr_t bytes = bf16 ? 8 : 16;
    r.wide = r.chunk % 4 == 0 && r.gsize % 4 == 0 && ld % 4 == 0 &&
             reinterpret_cast<uintptr_t>(logits) % bytes == 0;
    r.wide_bias = reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  };
  if (T >= kManyTokens && r.k <= 14 && split_row(r, 16, 32)) {
    wide();
    if (r.chunk <= 4) return launch_scored_v<16, 4>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
    if (r.chunk <= 8) return launch_scored_v<16, 8>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
    if (r.chunk <= 12) return launch_scored_v<16, 12>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
    if (r.chunk <= 16) return launch_scored_v<16, 16>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
    if (r.chunk <= 24) return launch_scored_v<16, 24>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
    return launch_scored_v<16, 32>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  }
  if (!split_row(r, 64, 128)) return hipErrorInvalidValue;
  wide();
  if (r.chunk <= 4) return launch_scored_v<64, 4>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (r.chunk <= 8) return launch_scored_v<64, 8>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (r.chunk <= 16) return launch_scored_v<64, 16>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (r.chunk <= 32) return launch_scored_v<64, 32>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (r.chunk <= 64) return launch_scored_v<64, 64>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  return launch_scored_v<64, 128>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
}

hipError_t launch_route_scored_bwd(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                                   int32_t T, const int32_t* idx, const float* dgate,
                                   void* dlogits, int64_t ldd, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int E = r.E;
  const bool dense = !r.sigmoid && !r.renorm;
  if (T >= (dense ? kManyDense : kManySparse) && r.k <= 16 && E <= 512) {   // four tokens to a wave
    if (!dense) return launch_bwd_v<16, 0>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
    if (E <= 64) return launch_bwd_v<16, 4>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
    if (E <= 128) return launch_bwd_v<16, 8>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
    if (E <= 256) return launch_bwd_v<16, 16>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
    return launch_bwd_v<16, 32>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  }
  if (!dense) return launch_bwd_v<64, 0>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 256) return launch_bwd_v<64, 4>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 512) return launch_bwd_v<64, 8>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 1024) return launch_bwd_v<64, 16>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 2048) return launch_bwd_v<64, 32>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  return launch_bwd_v<64, 64>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
}

hipError_t launch_bias_update(int32_t* load, int32_t n_layers, int32_t E, float rate, float* bias,
                              bool clear_load, hipStream_t s) {
  if (n_layers == 0) return hipSuccess;
  const int threads = E < kBiasThreads ? (E + kWave - 1) / kWave * kWave : kBiasThreads;
  hipLaunchKernelGGL(k_bias_update, dim3(n_layers), dim3(threads), 0, s, load, E, rate, bias,
                     clear_load ? 1 : 0);
  return hipGetLastError();
}

}  // namespace mok
