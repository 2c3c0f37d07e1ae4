// adamw.hip -- one AdamW step over many tensors, states in fp32 or in E4M3 codes
// with a scale per 32 elements: one launch for each of the two.
//
// A table in device memory, written once for a program's buffers, holds the
// tensors' addresses and factors, and the first unit of each: the 1024 elements
// (2048 with 8-bit states) of one workgroup.  A workgroup finds its tensor with
// one load per lane and a ballot for each power of 64 in the number of tensors,
// and works out the step's factors while its elements are on their way.  A
// thread has four consecutive elements, so that every access of a wave is
// contiguous and the 32 elements of an 8-bit block lie in eight lanes.
//
// Bound by HBM: 28 bytes an element with fp32 states, bf16 gradients and copy:
// 352 M in 1.53 ms, 6.45 TB/s; 16 1/8 with 8-bit states: 88 M in 0.25 ms, 5.6 TB/s
// (a large copy moves 5.2).  What counts is how near to each other the runs of
// memory are that are read and written at a time:
//   - small units: fp32 states in units of 8192 elements 1.85 ms, and 2.0 where
//     2048 workgroups take the units in turn and drift apart;
//   - few waves in flight: fp32 states 1.72 ms with 8 waves a SIMD, 1.60 with 5
//     or 4, 1.75 with 3; with 8-bit states latency counts more: 0.25 ms with 7
//     waves, 0.27 with 6, 0.29 with 5;
//   - 64 units in a row for each XCD: 1.60 -> 1.53 ms (128: 1.61; with 8-bit
//     states no gain);
//   - nontemporal loads and stores: 6 and 4 %.
// With 8-bit states two units of loads are under way at once (0.25 ms; one 0.30,
// three 0.28), and the vector instructions are near: 80 an element, 0.2 ms.  What
// is rare (a value that is not finite, r below 2^-50, a code below 2^-6 of the
// scale) is left to a second path that a whole wave takes.
// One tensor of 2048 elements 2.6 us (fp32) and 4.4 us, 200 tensors of 4096 to
// 13000 elements 11 us.
//
// The order of the fp32 operations on the states is fixed (no contraction): the
// 8-bit codes follow from the bits of m and v.
#include <cmath>

#include "scored_adamw.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = kThreads * 4;              // elements of a workgroup at a time
constexpr int kBatch = 40;                        // tensors of one table-writing launch
constexpr int kF32Waves = 5, kMxWaves = 7;        // a SIMD
constexpr uint32_t kXcds = 8, kRun = 64;          // units that follow each other on one XCD
constexpr int kMxGroups = 2;                      // groups of a unit with 8-bit states

struct TensorArg {
  float* p;
  uint16_t* pb;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  uint32_t flags;                                 // kBf16Grad, kWide
  uint32_t number;                                // of the tensor in the caller's list
  float lr_scale, weight_decay;
  int64_t unit0;
};
constexpr uint32_t kBf16Grad = 1, kWide = 2;

struct TableArg {
  int32_t first, count;
  TensorArg t[kBatch];
};
static_assert(sizeof(TableArg) <= 4096, "kernel argument");

// The table: n first units, then n descriptors.
size_t descriptors_at(int64_t n) { return (static_cast<size_t>(n) * 8 + 15) / 16 * 16; }

__global__ void k_adamw_table(TableArg a, int64_t* units, TensorArg* t) {
  const int i = threadIdx.x;
  if (i >= a.count) return;
  units[a.first + i] = a.t[i].unit0;
  t[a.first + i] = a.t[i];
}

struct StepArg {
  double lr, beta1, beta2;
  double per_m;                                   // lr / (1 - beta1^t), and
  float inv_bc2;                                  // 1 / sqrt(1 - beta2^t), of the host's step
  uint32_t step_key;
  float b1, c1, b2, c2, eps, grad_scale;
  uint32_t seed;
  const mok_adamw_scalars* scalars;
  const int64_t* units;
  const TensorArg* tensors;
  int32_t n_tensors;
};

__host__ __device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x9E3779B1u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// beta^t by repeated squaring, in fp64.
__device__ __forceinline__ double power(double b, uint32_t t) {
  double r = 1.0;
  for (; t; t >>= 1) {
    if (t & 1u) r *= b;
    b *= b;
  }
  return r;
}

// The smallest E with amax <= 448 * 2^E (448 = 1.75 * 2^8), -127 at least.
__device__ __forceinline__ int state_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(code), 0);
}

__device__ __forceinline__ bool finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
}

// (b + 0.5) / 65536, exact.
__device__ __forceinline__ float unit_of(uint32_t b16) {
  return fmaf(static_cast<float>(b16), 1.0f / 65536.0f, 0.5f / 65536.0f);
}

// Codes of any value, and of those that most are: finite, a in [2^-6, 448]
// (an E4M3 number without a subnormal, so its neighbours are cut from its bits).
__device__ __forceinline__ uint32_t encode_m(float m, int E, uint32_t b16) {
#pragma clang fp contract(off)
  if (!finite(m)) return 0x7fu;
  const float a = __builtin_amdgcn_ldexpf(fabsf(m), -E);
  const uint32_t normal = ((__float_as_uint(a) + 16u * b16 + 8u) >> 20) - 960u;
  const uint32_t tiny = static_cast<uint32_t>(a * 512.0f + unit_of(b16));
  const uint32_t code = a >= 0.015625f ? normal : tiny;
  return m < 0.0f ? code | 0x80u : code;
}
__device__ __forceinline__ uint32_t encode_m_normal(float a, float m, uint32_t b16) {
  const uint32_t code = (__float_as_uint(a) + 16u * b16 + (8u - (960u << 20))) >> 20;
  return code | ((__float_as_uint(m) >> 24) & 0x80u);
}

__device__ __forceinline__ uint32_t encode_r(float r, int E, uint32_t b16) {
#pragma clang fp contract(off)
  if (!finite(r)) return 0x7fu;
  const float a = __builtin_amdgcn_ldexpf(r, -E);
  uint32_t code = a >= 0.015625f ? (__float_as_uint(a) >> 20) - 960u
                                 : static_cast<uint32_t>(a * 512.0f);
  const float low = e4m3_value(code);
  const float high = code == 0x7eu ? 480.0f : e4m3_value(code + 1u);
  const float have = (a - low) * (a + low), span = (high - low) * (high + low);
  code += have > unit_of(b16) * span ? 1u : 0u;
  return r > 0.0f && code == 0u ? 1u : code;
}
__device__ __forceinline__ uint32_t encode_r_normal(float a, uint32_t b16) {
#pragma clang fp contract(off)
  const uint32_t u = __float_as_uint(a) & 0xfff00000u;
  const float low = __uint_as_float(u), high = __uint_as_float(u + 0x100000u);
  const float have = (a - low) * (a + low), span = fmaf(high, high, -(low * low));   // exact
  return (u >> 20) + (have > unit_of(b16) * span ? 1u - 960u : 0u - 960u);
}

struct Factors {
  float b1, c1, b2, c2, gs, keep, rate, inv_bc2, eps;
};

// New m and v of one element.
__device__ __forceinline__ void states(const Factors& f, float g, float& m, float& v) {
#pragma clang fp contract(off)
  g = g * f.gs;
  m = f.b1 * m + f.c1 * g;
  v = f.b2 * v + f.c2 * g * g;
}

// sqrt of a normal number: rsq and one step (rounds as sqrtf but for an odd case in 2^20).
__device__ __forceinline__ float sqrt_normal(float v) {
  const float y = __builtin_amdgcn_rsqf(v), s = v * y;
  return fmaf(fmaf(-s, s, v), 0.5f * y, s);
}

__device__ __forceinline__ float parameter(const Factors& f, float p, float m, float r) {
  const float d = fmaf(r, f.inv_bc2, f.eps);
  return fmaf(-f.rate, m * __builtin_amdgcn_rcpf(d), p * f.keep);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Largest of the eight lanes that share a block of 32 elements.
__device__ __forceinline__ float max8(float v) {
  int b = __builtin_bit_cast(int, v);                    // not negative: ordered as integers
  auto up = [&](int o) { b = o > b ? o : b; };
  up(__builtin_amdgcn_update_dpp(0, b, 0xB1, 0xF, 0xF, true));
  up(__builtin_amdgcn_update_dpp(0, b, 0x4E, 0xF, 0xF, true));
  up(__builtin_amdgcn_update_dpp(0, b, 0x141, 0xF, 0xF, true));
  return __builtin_bit_cast(float, b);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four elements as they are loaded.
template <bool MX>
struct Group {
  f32x4 p;
  f32x4 g;                       // bf16: two words
  f32x4 m, v;                    // MX: one word of codes
  int em, ev;                    // MX: old scales
};

// `have` of the four exist (0..4); whole: all, aligned.
template <bool MX>
__device__ __forceinline__ void load(const TensorArg& t, int64_t i0, int have, bool wide, Group<MX>& o) {
  const uint16_t* gb = static_cast<const uint16_t*>(t.g);
  const float* gf = static_cast<const float*>(t.g);
  const uint8_t* mc = static_cast<const uint8_t*>(t.m);
  const uint8_t* vc = static_cast<const uint8_t*>(t.v);
  const float* mf = static_cast<const float*>(t.m);
  const float* vf = static_cast<const float*>(t.v);
  const bool bf16 = t.flags & kBf16Grad;
  o.p = o.g = o.m = o.v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  o.em = o.ev = 0;
  if (wide && have == 4) {
    o.p = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(t.p + i0));
    if (bf16) {
      const u32x2 b = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(gb + i0));
      o.g.x = __uint_as_float(b.x << 16); o.g.y = __uint_as_float(b.x & 0xffff0000u);
      o.g.z = __uint_as_float(b.y << 16); o.g.w = __uint_as_float(b.y & 0xffff0000u);
    } else {
      o.g = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(gf + i0));
    }
    if (MX) {
      o.m.x = __uint_as_float(__builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(mc + i0)));
      o.v.x = __uint_as_float(__builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(vc + i0)));
    } else {
      o.m = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(mf + i0));
      o.v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(vf + i0));
    }
  } else {
    uint32_t mw = 0, vw = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= have) break;
      o.p[j] = t.p[i0 + j];
      o.g[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(gb[i0 + j]) << 16) : gf[i0 + j];
      if (MX) {
        mw |= static_cast<uint32_t>(mc[i0 + j]) << (8 * j);
        vw |= static_cast<uint32_t>(vc[i0 + j]) << (8 * j);
      } else {
        o.m[j] = mf[i0 + j];
        o.v[j] = vf[i0 + j];
      }
    }
    if (MX) {
      o.m.x = __uint_as_float(mw);
      o.v.x = __uint_as_float(vw);
    }
  }
  if (MX && have > 0) {
    o.em = t.ms[i0 >> 5];
    o.ev = t.vs[i0 >> 5];
  }
}

template <bool MX>
__device__ __forceinline__ void work(const TensorArg& t, const Factors& f, uint32_t key, int64_t i0,
                                     int have, bool wide, Group<MX>& o) {
  float m[4], v[4], r[4], p[4];
  uint32_t mw = __float_as_uint(o.m.x), vw = __float_as_uint(o.v.x);
  if (MX) {
#pragma clang fp contract(off)
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 m01 = __builtin_amdgcn_cvt_pk_f32_fp8(mw, false), m23 = __builtin_amdgcn_cvt_pk_f32_fp8(mw, true);
    const f32x2 v01 = __builtin_amdgcn_cvt_pk_f32_fp8(vw, false), v23 = __builtin_amdgcn_cvt_pk_f32_fp8(vw, true);
    m[0] = m01.x; m[1] = m01.y; m[2] = m23.x; m[3] = m23.y;
    v[0] = v01.x; v[1] = v01.y; v[2] = v23.x; v[3] = v23.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = __builtin_amdgcn_ldexpf(m[j], o.em - 127);
      const float q = __builtin_amdgcn_ldexpf(v[j], o.ev - 127);
      v[j] = q * q;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) { m[j] = o.m[j]; v[j] = o.v[j]; }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    states(f, o.g[j], m[j], v[j]);
    if (MX && j >= have) m[j] = v[j] = 0.0f;
  }
  // the plain way for a wave with a v that is not finite, or below the range of rsq (v is not
  // negative: its bits are in its order, a NaN's above all)
  const uint32_t b0 = __float_as_uint(v[0]), b1 = __float_as_uint(v[1]), b2 = __float_as_uint(v[2]),
                 b3 = __float_as_uint(v[3]);
  const uint32_t most = umax(umax(umax(b0, b1), b2), b3), lowest = umin(umin(umin(b0, b1), b2), b3);
  const bool odd = __ballot(most >= 0x7f800000u || lowest < 0x0d800000u) != 0;   // inf; 2^-100
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = odd ? sqrtf(v[j]) : sqrt_normal(v[j]);
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = parameter(f, o.p[j], m[j], r[j]);
  if (MX) {
    float am = 0.0f, ar = 0.0f;
    if (odd) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (finite(m[j])) am = fmaxf(am, fabsf(m[j]));
        if (finite(r[j])) ar = fmaxf(ar, r[j]);
      }
    } else {
      am = fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])), fmaxf(fabsf(m[2]), fabsf(m[3])));
      ar = fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
    }
    const int em = state_scale_exp(max8(am)), er = state_scale_exp(max8(ar));
    uint32_t h[4];
    // four neighbours never lie on both sides of a multiple of 2^32
    const uint32_t at = static_cast<uint32_t>(i0) +
                        static_cast<uint32_t>(static_cast<uint64_t>(i0) >> 32) * 0x6A09E667u + key;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = hash32(at + j);
    float a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __builtin_amdgcn_ldexpf(fabsf(m[j]), -em);
      b[j] = __builtin_amdgcn_ldexpf(r[j], -er);
    }
    const float least = fminf(fminf(fminf(a[0], a[1]), fminf(a[2], a[3])),
                              fminf(fminf(b[0], b[1]), fminf(b[2], b[3])));
    // (a NaN among the m would not show in `least`)
    const bool plain = !(least >= 0.015625f && (a[0] + a[1]) + (a[2] + a[3]) < 2048.0f);
    mw = vw = 0;
    if (odd || __ballot(plain)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mw |= encode_m(m[j], em, h[j] & 0xffffu) << (8 * j);
        vw |= encode_r(r[j], er, h[j] >> 16) << (8 * j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mw |= encode_m_normal(a[j], m[j], h[j] & 0xffffu) << (8 * j);
        vw |= encode_r_normal(b[j], h[j] >> 16) << (8 * j);
      }
    }
    if (have > 0 && (i0 & 31) == 0) {
      t.ms[i0 >> 5] = static_cast<uint8_t>(em + 127);
      t.vs[i0 >> 5] = static_cast<uint8_t>(er + 127);
    }
  }
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  float* mf = static_cast<float*>(t.m);
  float* vf = static_cast<float*>(t.v);
  if (wide && have == 4) {
    __builtin_nontemporal_store(f32x4{p[0], p[1], p[2], p[3]}, reinterpret_cast<f32x4*>(t.p + i0));
    if (MX) {
      __builtin_nontemporal_store(mw, reinterpret_cast<uint32_t*>(mc + i0));
      __builtin_nontemporal_store(vw, reinterpret_cast<uint32_t*>(vc + i0));
    } else {
      __builtin_nontemporal_store(f32x4{m[0], m[1], m[2], m[3]}, reinterpret_cast<f32x4*>(mf + i0));
      __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(vf + i0));
    }
    if (t.pb)
      __builtin_nontemporal_store(u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])},
                                  reinterpret_cast<u32x2*>(t.pb + i0));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= have) break;
      t.p[i0 + j] = p[j];
      if (MX) {
        mc[i0 + j] = static_cast<uint8_t>(mw >> (8 * j));
        vc[i0 + j] = static_cast<uint8_t>(vw >> (8 * j));
      } else {
        mf[i0 + j] = m[j];
        vf[i0 + j] = v[j];
      }
      if (t.pb) t.pb[i0 + j] = f32_to_bf16(p[j]);
    }
  }
}

// The table is read through the scalar cache: every wave works on one tensor.
typedef const __attribute__((address_space(4))) TensorArg* TablePtr;

// The last tensor whose first unit is not behind u.
__device__ __forceinline__ int tensor_of(const int64_t* __restrict__ units, int count, int64_t u) {
  const int lane = lane_id();
  int first = 0;
  while (count > 1) {
    const int step = (count + kWave - 1) / kWave;
    const bool starts = lane * step < count && units[first + lane * step] <= u;
    const int k = __popcll(__ballot(starts)) - 1;
    first += k * step;
    count = count - k * step < step ? count - k * step : step;
  }
  return __builtin_amdgcn_readfirstlane(first);
}

typedef const __attribute__((address_space(4))) mok_adamw_scalars* ScalarsPtr;

// The step's numbers, from the host or from device memory; false: nothing is
// done.  What depends on the step alone comes from the host where it knows it:
// in fp64 on the vector units it is 200 instructions of each wave.
__device__ __forceinline__ bool factors(const StepArg& h, float lr_scale, float weight_decay,
                                        uint32_t number, Factors& f, uint32_t& key) {
  f.b1 = h.b1; f.c1 = h.c1; f.b2 = h.b2; f.c2 = h.c2; f.eps = h.eps;
  double lr = h.lr, per_m = h.per_m;
  f.gs = h.grad_scale;
  f.inv_bc2 = h.inv_bc2;
  uint32_t step_key = h.step_key;
  if (h.scalars) {
    const ScalarsPtr sc = (ScalarsPtr)(uintptr_t)h.scalars;
    const int32_t step = sc->step;
    if (sc->skip != 0 || step < 1) return false;
    lr = sc->lr;
    f.gs = sc->grad_scale;
    per_m = static_cast<double>(sc->lr / static_cast<float>(1.0 - power(h.beta1, step)));
    f.inv_bc2 = 1.0f / sqrtf(static_cast<float>(1.0 - power(h.beta2, step)));
    step_key = hash32(h.seed + 0x9E3779B1u * static_cast<uint32_t>(step));
  }
  f.keep = static_cast<float>(1.0 - lr * static_cast<double>(lr_scale) * static_cast<double>(weight_decay));
  f.rate = static_cast<float>(per_m * static_cast<double>(lr_scale));
  key = hash32(step_key + number);
  return true;
}

template <bool MX>
__device__ __forceinline__ void unit(const TensorArg& t, const StepArg& h, int64_t u) {
  constexpr int kN = MX ? kMxGroups : 1;
  const int64_t i0 = u * (kGroup * kN) + 4 * static_cast<int64_t>(threadIdx.x);
  const bool wide = t.flags & kWide;
  const auto have = [&](int s) {
    const int64_t left = t.n - (i0 + s * kGroup);
    return left < 0 ? 0 : (left > 4 ? 4 : static_cast<int>(left));
  };
  Group<MX> o[kN];
#pragma unroll
  for (int s = 0; s < kN; ++s) load<MX>(t, i0 + s * kGroup, have(s), wide, o[s]);
  Factors f;
  uint32_t key;
  if (!factors(h, t.lr_scale, t.weight_decay, t.number, f, key)) return;   // while the loads are on their way
#pragma unroll
  for (int s = 0; s < kN; ++s) work<MX>(t, f, key, i0 + s * kGroup, have(s), wide, o[s]);
}

template <bool MX>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, MX ? kMxWaves : kF32Waves)))
void k_adamw(StepArg h) {
  int64_t u = blockIdx.x;
  if (!MX) {                                            // workgroups go round the XCDs: runs of units for each
    const uint32_t run = kXcds * kRun, block = blockIdx.x / run, in = blockIdx.x % run;
    if (block < gridDim.x / run) u = static_cast<int64_t>(block) * run + in % kXcds * kRun + in / kXcds;
  }
  const TablePtr p = (TablePtr)(uintptr_t)(h.tensors + tensor_of(h.units, h.n_tensors, u));
  TensorArg t;
  t.p = p->p; t.pb = p->pb; t.g = p->g; t.m = p->m; t.v = p->v; t.ms = p->ms; t.vs = p->vs;
  t.n = p->n; t.flags = p->flags; t.number = p->number; t.lr_scale = p->lr_scale;
  t.weight_decay = p->weight_decay; t.unit0 = p->unit0;
  unit<MX>(t, h, u - t.unit0);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

size_t adamw_table_bytes(int64_t n) { return descriptors_at(n) + static_cast<size_t>(n) * sizeof(TensorArg); }

int64_t adamw_units(int64_t n, bool mx) { return (n - 1) / (kGroup * (mx ? kMxGroups : 1)) + 1; }

hipError_t launch_adamw_table(const mok_adamw_tensor* tensors, int32_t n, void* table,
                              mok_adamw_plan& plan, hipStream_t s) {
  int64_t* units = static_cast<int64_t*>(table);
  TensorArg* out = reinterpret_cast<TensorArg*>(static_cast<uint8_t*>(table) + descriptors_at(n));
  TableArg a;
  a.first = a.count = 0;
  plan.list = n;
  for (int mx = 0; mx < 2; ++mx) {                      // the tensors of each format follow each other
    for (int32_t i = 0; i < n; ++i) {
      const mok_adamw_tensor& x = tensors[i];
      if (x.n == 0 || (x.state_format == MOK_STATE_MXFP8) != (mx == 1)) continue;
      const bool bf16 = x.grad_type == MOK_TYPE_BF16;
      const bool wide = aligned(x.p, 16) && (!x.p_bf16 || aligned(x.p_bf16, 8)) &&
                        aligned(x.grad, bf16 ? 8 : 16) && aligned(x.m, mx ? 4 : 16) &&
                        aligned(x.v, mx ? 4 : 16);
      a.t[a.count++] = TensorArg{x.p, static_cast<uint16_t*>(x.p_bf16), x.grad, x.m, x.v, x.m_scale,
                                 x.v_scale, x.n, (bf16 ? kBf16Grad : 0) | (wide ? kWide : 0),
                                 static_cast<uint32_t>(i), x.lr_scale, x.weight_decay, plan.n_units[mx]};
      plan.n_units[mx] += adamw_units(x.n, mx);
      ++plan.n_tensors[mx];
      if (a.count == kBatch) {
        hipLaunchKernelGGL(k_adamw_table, dim3(1), dim3(kWave), 0, s, a, units, out);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.first += a.count;
        a.count = 0;
      }
    }
  }
  if (a.count == 0) return hipSuccess;
  hipLaunchKernelGGL(k_adamw_table, dim3(1), dim3(kWave), 0, s, a, units, out);
  return hipGetLastError();
}

hipError_t launch_adamw(const void* table, const mok_adamw_plan& plan, const mok_adamw_hyper& h,
                        const mok_adamw_scalars* scalars, hipStream_t s) {
  const int64_t* units = static_cast<const int64_t*>(table);
  const TensorArg* t = reinterpret_cast<const TensorArg*>(static_cast<const uint8_t*>(table) + descriptors_at(plan.list));
  StepArg a{};
  a.lr = h.lr; a.beta1 = h.beta1; a.beta2 = h.beta2;
  a.b1 = static_cast<float>(h.beta1); a.c1 = static_cast<float>(1.0 - h.beta1);
  a.b2 = static_cast<float>(h.beta2); a.c2 = static_cast<float>(1.0 - h.beta2);
  a.eps = static_cast<float>(h.eps);
  a.seed = h.seed;
  a.scalars = scalars;
  if (!scalars) {
    a.grad_scale = static_cast<float>(h.grad_scale);
    a.per_m = h.lr / (1.0 - std::pow(h.beta1, h.step));
    a.inv_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h.beta2, h.step)));
    a.step_key = hash32(h.seed + 0x9E3779B1u * static_cast<uint32_t>(h.step));
  }
  a.units = units;
  a.tensors = t;
  a.n_tensors = plan.n_tensors[0];
  if (plan.n_units[0] > 0) {
    hipLaunchKernelGGL(k_adamw<false>, dim3(static_cast<uint32_t>(plan.n_units[0])), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (plan.n_units[1] == 0) return hipSuccess;
  a.units += plan.n_tensors[0];
  a.tensors += plan.n_tensors[0];
  a.n_tensors = plan.n_tensors[1];
  hipLaunchKernelGGL(k_adamw<true>, dim3(static_cast<uint32_t>(plan.n_units[1])), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace mok
