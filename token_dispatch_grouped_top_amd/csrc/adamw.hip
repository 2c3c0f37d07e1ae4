// adamw.hip -- one AdamW step over many tensors in one launch, states in fp32
// or in E4M3 codes with a scale per 32 elements.
//
// The tensors' pointers travel as a kernel argument (up to kMaxTensors per
// launch), so the call needs no device table.  A workgroup takes one unit of
// kUnit elements of one tensor: the unit's tensor is the last whose first unit
// is not behind it, found with one load per lane and a ballot.  A thread works
// on four consecutive elements at a time, so that every access of a wave is
// contiguous, and the 32 elements of an 8-bit block lie in eight lanes.
//
// The order of the fp32 operations is fixed (no contraction): the 8-bit codes
// follow from the bits of m and v.
#include "mok_internal.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;                         // groups of four per thread and unit
constexpr int kUnit = kThreads * 4 * kSteps;      // elements
constexpr int kMaxTensors = kAdamwMaxTensors;

struct TensorArg {
  float* p;
  uint16_t* pb;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  uint32_t flags;                                 // kBf16Grad, kMx, kWide
  uint32_t number;                                // of the tensor in the call
  float lr_scale, weight_decay;
};
constexpr uint32_t kBf16Grad = 1, kMx = 2, kWide = 4;

struct StepArg {
  double lr, beta1, beta2;
  float eps, grad_scale;
  int32_t step;
  uint32_t seed;
  const mok_adamw_scalars* scalars;
  int32_t n_tensors;
};

struct Args {
  StepArg h;
  uint32_t unit0[kMaxTensors];                    // first unit of each tensor
  TensorArg t[kMaxTensors];
};
static_assert(sizeof(Args) <= 4096, "kernel argument");

__device__ __forceinline__ uint32_t hash32(uint32_t x) {
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

__device__ __forceinline__ float unit_of(uint32_t b16) {
#pragma clang fp contract(off)
  return (static_cast<float>(b16) + 0.5f) * (1.0f / 65536.0f);
}

__device__ __forceinline__ uint32_t encode_m(float m, int E, uint32_t b16) {
#pragma clang fp contract(off)
  if (!finite(m)) return 0x7fu;
  const float a = __builtin_amdgcn_ldexpf(fabsf(m), -E);
  const uint32_t normal = ((__float_as_uint(a) + 16u * b16 + 8u) >> 20) - 960u;
  const uint32_t tiny = static_cast<uint32_t>(a * 512.0f + unit_of(b16));
  const uint32_t code = a >= 0.015625f ? normal : tiny;
  return m < 0.0f ? code | 0x80u : code;
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

struct Factors {
  float b1, c1, b2, c2, gs, keep, rate, inv_bc2, eps;
};

// One element: m, v (or r^2) and p updated; r = sqrt(v).
__device__ __forceinline__ void update(const Factors& f, float g, float& p, float& m, float& v,
                                       float& r) {
#pragma clang fp contract(off)
  g = g * f.gs;
  m = f.b1 * m + f.c1 * g;
  v = f.b2 * v + f.c2 * g * g;
  r = sqrtf(v);
  p = p * f.keep - f.rate * (m / (r * f.inv_bc2 + f.eps));
}

// Largest of the eight lanes that share a block of 32 elements.
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, __shfl_xor(v, 1));
  v = fmaxf(v, __shfl_xor(v, 2));
  return fmaxf(v, __shfl_xor(v, 4));
}

// Four elements from i0 on, of which `have` exist (0..4).  WIDE: 4, and every
// pointer is aligned for them.
template <bool MX, bool WIDE>
__device__ __forceinline__ void group4(const TensorArg& t, const Factors& f, uint32_t key,
                                       int64_t i0, int have) {
  float p[4] = {}, g[4] = {}, m[4] = {}, v[4] = {}, r[4] = {};
  const bool bf16 = t.flags & kBf16Grad;
  const uint16_t* gb = static_cast<const uint16_t*>(t.g);
  const float* gf = static_cast<const float*>(t.g);
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  float* mf = static_cast<float*>(t.m);
  float* vf = static_cast<float*>(t.v);
  uint32_t mw = 0, vw = 0;
  if (WIDE) {
    const float4 a = *reinterpret_cast<const float4*>(t.p + i0);
    p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
    if (bf16) {
      const uint2 b = *reinterpret_cast<const uint2*>(gb + i0);
      g[0] = __uint_as_float(b.x << 16); g[1] = __uint_as_float(b.x & 0xffff0000u);
      g[2] = __uint_as_float(b.y << 16); g[3] = __uint_as_float(b.y & 0xffff0000u);
    } else {
      const float4 b = *reinterpret_cast<const float4*>(gf + i0);
      g[0] = b.x; g[1] = b.y; g[2] = b.z; g[3] = b.w;
    }
    if (MX) {
      mw = *reinterpret_cast<const uint32_t*>(mc + i0);
      vw = *reinterpret_cast<const uint32_t*>(vc + i0);
    } else {
      const float4 b = *reinterpret_cast<const float4*>(mf + i0);
      const float4 c = *reinterpret_cast<const float4*>(vf + i0);
      m[0] = b.x; m[1] = b.y; m[2] = b.z; m[3] = b.w;
      v[0] = c.x; v[1] = c.y; v[2] = c.z; v[3] = c.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= have) break;
      p[j] = t.p[i0 + j];
      g[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(gb[i0 + j]) << 16) : gf[i0 + j];
      if (MX) {
        mw |= static_cast<uint32_t>(mc[i0 + j]) << (8 * j);
        vw |= static_cast<uint32_t>(vc[i0 + j]) << (8 * j);
      } else {
        m[j] = mf[i0 + j];
        v[j] = vf[i0 + j];
      }
    }
  }
  if (MX && have > 0) {
    const int em = t.ms[i0 >> 5] - 127, ev = t.vs[i0 >> 5] - 127;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = __builtin_amdgcn_ldexpf(e4m3_value((mw >> (8 * j)) & 0xffu), em);
      const float q = __builtin_amdgcn_ldexpf(e4m3_value((vw >> (8 * j)) & 0xffu), ev);
      v[j] = q * q;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (WIDE || j < have) update(f, g[j], p[j], m[j], v[j], r[j]);
  if (MX) {
    float am = 0.0f, ar = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (WIDE || j < have) {
        if (finite(m[j])) am = fmaxf(am, fabsf(m[j]));
        if (finite(r[j])) ar = fmaxf(ar, r[j]);
      }
    const int em = state_scale_exp(max8(am)), er = state_scale_exp(max8(ar));
    mw = vw = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t i = static_cast<uint64_t>(i0) + j;
      const uint32_t h = hash32(static_cast<uint32_t>(i) +
                                static_cast<uint32_t>(i >> 32) * 0x6A09E667u + key);
      mw |= encode_m(m[j], em, h & 0xffffu) << (8 * j);
      vw |= encode_r(r[j], er, h >> 16) << (8 * j);
    }
    if (have > 0 && (i0 & 31) == 0) {
      t.ms[i0 >> 5] = static_cast<uint8_t>(em + 127);
      t.vs[i0 >> 5] = static_cast<uint8_t>(er + 127);
    }
  }
  if (WIDE) {
    *reinterpret_cast<float4*>(t.p + i0) = make_float4(p[0], p[1], p[2], p[3]);
    if (MX) {
      *reinterpret_cast<uint32_t*>(mc + i0) = mw;
      *reinterpret_cast<uint32_t*>(vc + i0) = vw;
    } else {
      *reinterpret_cast<float4*>(mf + i0) = make_float4(m[0], m[1], m[2], m[3]);
      *reinterpret_cast<float4*>(vf + i0) = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (t.pb)
      *reinterpret_cast<uint2*>(t.pb + i0) =
          make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
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

template <bool MX>
__device__ __forceinline__ void unit_loop(const TensorArg& t, const Factors& f, uint32_t key,
                                          int64_t u0) {
  const bool whole = (t.flags & kWide) && u0 + kUnit <= t.n;
#pragma unroll 1
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i0 = u0 + s * (kThreads * 4) + 4 * static_cast<int64_t>(threadIdx.x);
    if (whole) {
      group4<MX, true>(t, f, key, i0, 4);
    } else {
      const int64_t left = t.n - i0;
      group4<MX, false>(t, f, key, i0, left < 0 ? 0 : (left > 4 ? 4 : static_cast<int>(left)));
    }
  }
}

__global__ __launch_bounds__(kThreads)
void k_adamw(const Args a) {
  const int lane = lane_id();
  const uint32_t u = blockIdx.x;
  const bool starts = lane < a.h.n_tensors && a.unit0[lane < kMaxTensors ? lane : 0] <= u;
  const int ti = __builtin_amdgcn_readfirstlane(__popcll(__ballot(starts)) - 1);
  const TensorArg& t = a.t[ti];
  double lr = a.h.lr;
  float gs = a.h.grad_scale;
  int32_t step = a.h.step;
  if (a.h.scalars) {
    const mok_adamw_scalars sc = *a.h.scalars;
    if (sc.skip != 0 || sc.step < 1) return;
    lr = sc.lr;
    gs = sc.grad_scale;
    step = sc.step;
  }
  Factors f;
  lr *= static_cast<double>(t.lr_scale);
  f.b1 = static_cast<float>(a.h.beta1);
  f.c1 = static_cast<float>(1.0 - a.h.beta1);
  f.b2 = static_cast<float>(a.h.beta2);
  f.c2 = static_cast<float>(1.0 - a.h.beta2);
  f.gs = gs;
  f.keep = static_cast<float>(1.0 - lr * static_cast<double>(t.weight_decay));
  f.rate = static_cast<float>(lr / (1.0 - power(a.h.beta1, step)));
  f.inv_bc2 = static_cast<float>(1.0 / sqrt(1.0 - power(a.h.beta2, step)));
  f.eps = a.h.eps;
  const uint32_t key = hash32(hash32(a.h.seed + 0x9E3779B1u * static_cast<uint32_t>(step)) + t.number);
  const int64_t u0 = static_cast<int64_t>(u - a.unit0[ti]) * kUnit;
  if (t.flags & kMx) unit_loop<true>(t, f, key, u0);
  else unit_loop<false>(t, f, key, u0);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

hipError_t launch_adamw(const mok_adamw_tensor* tensors, int32_t n_tensors,
                        const mok_adamw_hyper& h, const mok_adamw_scalars* scalars, hipStream_t s) {
  Args a;
  a.h = StepArg{h.lr, h.beta1, h.beta2, static_cast<float>(h.eps),
                static_cast<float>(h.grad_scale), h.step, h.seed, scalars, 0};
  uint32_t units = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const mok_adamw_tensor& x = tensors[i];
    if (x.n > 0) {
      const bool bf16 = x.grad_type == MOK_TYPE_BF16, mx = x.state_format == MOK_STATE_MXFP8;
      const bool wide = aligned(x.p, 16) && (!x.p_bf16 || aligned(x.p_bf16, 8)) &&
                        aligned(x.grad, bf16 ? 8 : 16) && aligned(x.m, mx ? 4 : 16) &&
                        aligned(x.v, mx ? 4 : 16);
      const int32_t at = a.h.n_tensors++;
      a.unit0[at] = units;
      a.t[at] = TensorArg{x.p, static_cast<uint16_t*>(x.p_bf16), x.grad, x.m, x.v, x.m_scale,
                          x.v_scale, x.n,
                          (bf16 ? kBf16Grad : 0) | (mx ? kMx : 0) | (wide ? kWide : 0),
                          static_cast<uint32_t>(i), x.lr_scale, x.weight_decay};
      units += static_cast<uint32_t>((x.n + kUnit - 1) / kUnit);
    }
    // a full argument, the last tensor, or a grid that the next one could push past 2^31
    const bool full = a.h.n_tensors == kMaxTensors ||
                      (i + 1 < n_tensors &&
                       units + static_cast<uint64_t>((tensors[i + 1].n + kUnit - 1) / kUnit) > 0x7fffffffull);
    if (a.h.n_tensors > 0 && (full || i + 1 == n_tensors)) {
      hipLaunchKernelGGL(k_adamw, dim3(units), dim3(kThreads), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      a.h.n_tensors = 0;
      units = 0;
    }
  }
  return hipSuccess;
}

int64_t adamw_max_elements() { return 0x7fffffffll * kUnit; }

}  // namespace mok
