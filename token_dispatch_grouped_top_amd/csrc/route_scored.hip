// route_scored.hip -- the scored route (softmax or sigmoid scores, balance
// bias, expert groups, renormalised weights), its backward and the update of
// the bias.
//
// One wave per token.  Lane l holds the logits l, l + 64, ... in registers.
// Choice values c = s + bias are formed in fp64: the order of two experts is
// that of their real scores, which fp32 does not tell apart often enough (of
// 16384 tokens over 256 experts about one has two neighbours in its order
// within fp32's error).
#include "mok_internal.h"

namespace mok {

namespace {

constexpr int kWaves = 4;
constexpr float kNegInf = -__builtin_inff();

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

__device__ __forceinline__ bool better(double v, int e, double bv, int be) {
  return v > bv || (v == bv && e < be);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// The picks' shares u: lanes below n hold the logits l of the picks (n >= 1),
// largest first or not; the other lanes get 0.  sigmoid: s / sum s, formed
// from exp(l) where every s is as small as exp(l) itself (below 2^-60 of 1),
// so that nothing underflows.  softmax: exp(l - max) / sum.
__device__ __forceinline__ double share(bool valid, float l, bool sigmoid, double s) {
  const float lmax = wave_max(valid ? l : kNegInf);
  double a;
  if (sigmoid && lmax > -60.0f) a = valid ? s : 0.0;
  else a = valid ? exp(static_cast<double>(l) - static_cast<double>(lmax)) : 0.0;
  return a / wave_sum(a);
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kWaves * kWave)
void k_route_scored(RouterArgs r, const void* __restrict__ logits, int64_t ld,
                    const float* __restrict__ bias, int32_t T, int32_t* __restrict__ idx,
                    float* __restrict__ gate, int32_t* __restrict__ load, RouteCount rc) {
  extern __shared__ double lds[];           // groups: [waves][E] choice values
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / kWave) + w;
  if (t >= T) return;
  const int E = r.E;
  float l[VPL];
  double c[VPL];
  float lmax = kNegInf;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + kWave * i;
    l[i] = e < E ? clean_logit(load_logit<BF16>(logits, t * ld + e)) : kNegInf;
    lmax = fmaxf(lmax, l[i]);
  }
  double inv = 1.0;                         // softmax: 1 / sum
  const double top = static_cast<double>(wave_max(lmax));
  if (!r.sigmoid) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (l[i] > kNegInf) sum += exp(static_cast<double>(l[i]) - top);
    sum = wave_sum(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + kWave * i;
    const double x = static_cast<double>(l[i]);
    double s = r.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) * inv;
    if (bias && e < E) s += static_cast<double>(bias[e]);
    c[i] = l[i] > kNegInf ? s : -__builtin_inf();
  }
  if (r.G > 1) {
    double* row = lds + w * E;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + kWave * i < E) row[lane + kWave * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    double gv = -__builtin_inf();
    if (lane < r.G) {
      double g2 = -__builtin_inf();
      for (int j = 0; j < r.gsize; ++j) {
        const double v = row[lane * r.gsize + j];
        if (v > gv) { g2 = gv; gv = v; }
        else if (v > g2) g2 = v;
      }
      if (r.top2 && g2 > -__builtin_inf()) gv += g2;
    }
    int rank = 0;                           // groups before this one
    for (int g = 0; g < r.G; ++g) {
      const double ov = __shfl(gv, g);
      rank += g != lane && better(ov, g, gv, lane);
    }
    const uint64_t open = __ballot(lane < r.G && rank < r.top_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + kWave * i;
      if (e < E && !((open >> (e / r.gsize)) & 1ull)) c[i] = -__builtin_inf();
    }
  }
  int mine_e = -1;
  uint64_t taken = 0;
  for (int j = 0; j < r.k; ++j) {
    double bv = -__builtin_inf();
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + kWave * i;
      if (!((taken >> i) & 1ull) && c[i] > -__builtin_inf() && better(c[i], e, bv, be)) {
        bv = c[i];
        be = e;
      }
    }
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const double ov = __shfl_xor(bv, o);
      const int oe = __shfl_xor(be, o);
      if (better(ov, oe, bv, be)) { bv = ov; be = oe; }
    }
    if (be == 0x7fffffff) break;
    if ((be & (kWave - 1)) == lane) taken |= 1ull << (be / kWave);
    if (lane == j) mine_e = be;
  }
  const bool valid = mine_e >= 0;
  const float ml = valid ? clean_logit(load_logit<BF16>(logits, t * ld + mine_e)) : kNegInf;
  double s = 0.0;
  if (valid)
    s = r.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(ml)))
                  : exp(static_cast<double>(ml) - top) * inv;
  if (r.renorm && __ballot(valid)) s = share(valid, ml, r.sigmoid, s);
  if (lane < r.k) {
    idx[t * r.k + lane] = mine_e;
    gate[t * r.k + lane] = static_cast<float>(static_cast<double>(r.scale) * s);
  }
  if (valid && load)
    __hip_atomic_fetch_add(load + mine_e, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  // the fused layer's schedule counts
  const int le = mine_e - rc.base;
  if (valid && rc.blk_counts && le >= 0 && le < rc.n_local)
    __hip_atomic_fetch_add(rc.blk_counts + static_cast<int64_t>(le) * rc.nblk +
                               (t * r.k + lane) / kSchedChunk,
                           1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kWaves * kWave)
void k_route_scored_bwd(RouterArgs r, const void* __restrict__ logits, int64_t ld, int32_t T,
                        const int32_t* __restrict__ idx, const float* __restrict__ dgate,
                        void* __restrict__ dlogits, int64_t ldd) {
  const int lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / kWave;
  if (t >= T) return;
  const int E = r.E;
  int e = lane < r.k ? idx[t * r.k + lane] : -1;
  float l = kNegInf;
  if (e >= 0 && e < E) l = clean_logit(load_logit<BF16>(logits, t * ld + e));
  const bool valid = l > kNegInf;
  if (!valid) e = -1;
  const double x = static_cast<double>(l);
  const double wg = valid ? static_cast<double>(r.scale) * static_cast<double>(dgate[t * r.k + lane]) : 0.0;
  double s = 0.0, d = 0.0, rest = 0.0, top = 0.0;
  double dense[VPL];                        // softmax without renorm: s of every expert
#pragma unroll
  for (int i = 0; i < VPL; ++i) dense[i] = 0.0;
  if (r.sigmoid && valid) s = 1.0 / (1.0 + exp(-x));
  const double not_s = r.sigmoid ? (valid ? 1.0 / (1.0 + exp(x)) : 0.0) : 1.0;
  if (r.renorm) {
    if (__ballot(valid)) {
      const double u = share(valid, l, r.sigmoid, s);
      d = u * not_s * (wg - wave_sum(wg * u));
    }
  } else if (r.sigmoid) {
    d = s * not_s * wg;
  } else {
    float lv[VPL], m = kNegInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int o = lane + kWave * i;
      lv[i] = o < E ? clean_logit(load_logit<BF16>(logits, t * ld + o)) : kNegInf;
      m = fmaxf(m, lv[i]);
    }
    top = static_cast<double>(wave_max(m));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      dense[i] = lv[i] > kNegInf ? exp(static_cast<double>(lv[i]) - top) : 0.0;
      sum += dense[i];
    }
    sum = wave_sum(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
    s = valid ? exp(x - top) * inv : 0.0;
    d = s * wg;
    rest = wave_sum(d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) dense[i] *= -inv * rest;
  }
  for (int j = 0; j < r.k; ++j) {
    const int ej = __shfl(e, j);
    const double dj = __shfl(d, j);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + kWave * i == ej) dense[i] += dj;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int o = lane + kWave * i;
    if (o >= E) continue;
    if constexpr (BF16)
      static_cast<uint16_t*>(dlogits)[t * ldd + o] = f32_to_bf16(static_cast<float>(dense[i]));
    else
      static_cast<float*>(dlogits)[t * ldd + o] = static_cast<float>(dense[i]);
  }
}

constexpr int kBiasThreads = 256;

// One workgroup per layer: the load's sum in 64-bit integers, then the bias.
__global__ __launch_bounds__(kBiasThreads)
void k_bias_update(int32_t* __restrict__ load, int32_t E, float rate, float* __restrict__ bias,
                   int32_t clear_load) {
  __shared__ int64_t part[kBiasThreads / kWave];
  load += static_cast<int64_t>(blockIdx.x) * E;
  bias += static_cast<int64_t>(blockIdx.x) * E;
  int64_t sum = 0;
  for (int e = threadIdx.x; e < E; e += kBiasThreads) sum += load[e];
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o);
  if (lane_id() == 0) part[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kBiasThreads / kWave; ++w) sum += part[w];
  for (int e = threadIdx.x; e < E; e += kBiasThreads) {
    const int64_t d = sum - static_cast<int64_t>(E) * load[e];
    if (d != 0) bias[e] += d > 0 ? rate : -rate;
    if (clear_load) load[e] = 0;
  }
}

template <int VPL>
hipError_t launch_scored_vpl(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                             const float* bias, int32_t T, int32_t* idx, float* gate,
                             int32_t* load, const RouteCount& rc, hipStream_t s) {
  const int waves = r.E <= 2048 ? kWaves : 2;   // at most 64 KiB of choice values
  const dim3 grid((T + waves - 1) / waves), block(waves * kWave);
  const size_t lds = r.G > 1 ? sizeof(double) * waves * r.E : 0;
  if (bf16)
    hipLaunchKernelGGL((k_route_scored<VPL, true>), grid, block, lds, s, r, logits, ld, bias, T,
                       idx, gate, load, rc);
  else
    hipLaunchKernelGGL((k_route_scored<VPL, false>), grid, block, lds, s, r, logits, ld, bias, T,
                       idx, gate, load, rc);
  return hipGetLastError();
}

template <int VPL>
hipError_t launch_bwd_vpl(const RouterArgs& r, const void* logits, bool bf16, int64_t ld, int32_t T,
                          const int32_t* idx, const float* dgate, void* dlogits, int64_t ldd,
                          hipStream_t s) {
  const dim3 grid((T + kWaves - 1) / kWaves), block(kWaves * kWave);
  if (bf16)
    hipLaunchKernelGGL((k_route_scored_bwd<VPL, true>), grid, block, 0, s, r, logits, ld, T, idx,
                       dgate, dlogits, ldd);
  else
    hipLaunchKernelGGL((k_route_scored_bwd<VPL, false>), grid, block, 0, s, r, logits, ld, T, idx,
                       dgate, dlogits, ldd);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                               const float* bias, int32_t T, int32_t* idx, float* gate,
                               int32_t* load, const RouteCount& rc, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int E = r.E;
  if (E <= 64) return launch_scored_vpl<1>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (E <= 128) return launch_scored_vpl<2>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (E <= 256) return launch_scored_vpl<4>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (E <= 512) return launch_scored_vpl<8>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (E <= 1024) return launch_scored_vpl<16>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  if (E <= 2048) return launch_scored_vpl<32>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
  return launch_scored_vpl<64>(r, logits, bf16, ld, bias, T, idx, gate, load, rc, s);
}

hipError_t launch_route_scored_bwd(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                                   int32_t T, const int32_t* idx, const float* dgate,
                                   void* dlogits, int64_t ldd, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int E = r.E;
  if (E <= 64) return launch_bwd_vpl<1>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 128) return launch_bwd_vpl<2>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 256) return launch_bwd_vpl<4>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 512) return launch_bwd_vpl<8>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 1024) return launch_bwd_vpl<16>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  if (E <= 2048) return launch_bwd_vpl<32>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
  return launch_bwd_vpl<64>(r, logits, bf16, ld, T, idx, dgate, dlogits, ldd, s);
}

hipError_t launch_bias_update(int32_t* load, int32_t n_layers, int32_t E, float rate, float* bias,
                              bool clear_load, hipStream_t s) {
  if (n_layers == 0) return hipSuccess;
  hipLaunchKernelGGL(k_bias_update, dim3(n_layers), dim3(kBiasThreads), 0, s, load, E, rate, bias,
                     clear_load ? 1 : 0);
  return hipGetLastError();
}

}  // namespace mok
