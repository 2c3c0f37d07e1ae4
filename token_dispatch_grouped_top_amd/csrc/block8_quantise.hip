// block8_quantise.hip -- E4M3 codes with fp32 scales for blocks of 128: of
// token rows (optionally through SwiGLU or its backward), of the same rows
// transposed into slot blocks, and of weight matrices.
//
// scale = max(amax / 448, 2^-126), code = RNE(fl(value / scale)).  One
// workgroup takes 128 rows x 128 columns, reads them once into registers (4 x 8
// values a thread) and forms every scale that the tile has: of its rows, of
// its columns, of the whole.  The transposed codes go through LDS, so that both
// outputs are written in whole lines.  Bound: bytes, as long as a value costs
// few instructions (8192 x 7168 bf16 both ways: 55 us, 4.3 TB/s; with a test for
// NaN and IEEE divisions at each value it was 114): magnitudes are compared as
// whole numbers, in pairs where they are bf16, which shows what is not finite
// for nothing; a quotient is a product and one correction; and what is not
// finite then becomes NaN by itself.  Four rows a thread need 40 to 80 registers;
// eight need 64 to 150 and gain nothing (55 us; SwiGLU of 4095 x 2048 17.4 us
// instead of 16.3).  Through SwiGLU and its backward vector instructions bound
// it: they issue in 89 and 83 % of a CU's busy cycles (8192 rows of 8 experts,
// codes both ways: 2048 columns 25 us, the backward's 4096 65 us).
#include <algorithm>

#include "block8.h"

namespace mok {
namespace {

enum Mode { ROWS = 0, LINES = 1, BLOCKS = 2, WEIGHTS = 3 };

struct QuantArgs {
  const void* x; int64_t ld;
  const void* d; int64_t ldd;
  int32_t ring_rows;
  int32_t rows, W;
  const int32_t* offsets; int32_t n_local;
  uint8_t* codes; float* scales;
  uint8_t* codes_t; float* scales_t;
  int64_t S;                                   // places of a transposed row
  int32_t col_blocks;
};

// 8 values from an address of elements; VEC: 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (VEC) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
  } else {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (VEC) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
  }
}

// Eight values of a row in registers: as bf16 pairs where they come as such
// (half the registers, twice the waves), else in fp32.
template <bool PAIRS> struct Row8;
template <> struct Row8<true> {
  uint32_t w[4];
  __device__ __forceinline__ void set(uint4 u) { w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w; }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <> struct Row8<false> {
  float v[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};

// Magnitudes are compared as whole numbers, the values' bits without their
// sign: in that order infinity and NaN lie above every finite value, so a
// largest one says whether a block has any.
constexpr uint32_t kInf = 0x7f800000u;
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// Largest of the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#define MOK_ROT(n) m = umax(m, __builtin_amdgcn_update_dpp(0, m, 0x120 + (n), 0xf, 0xf, true))
  MOK_ROT(8); MOK_ROT(4); MOK_ROT(2); MOK_ROT(1);
#undef MOK_ROT
  return m;
}

// A block's scale s and 1 / s from its largest magnitude.  amax / 448 as fp32
// division rounds it: from the rounded reciprocal of 448 and one correction
// (scales below 2^-126 are not used).
struct Scale {
  float s, r;
  Scale() = default;
  __device__ __forceinline__ explicit Scale(uint32_t amax) {
    const float a = __uint_as_float(amax), q = a * (1.0f / 448.0f);
    s = fmaxf(__builtin_fmaf(__builtin_fmaf(-q, 448.0f, a), 1.0f / 448.0f, q), 0x1p-126f);
    r = __builtin_amdgcn_rcpf(s);
    r = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
  }
  // x / s as fp32 division rounds it, from the reciprocal and one correction
  // (subtracted in this way it leaves a zero its sign).  At most 448 + 2^-15,
  // which converts to 448.
  __device__ __forceinline__ float operator()(float x) const {
    const float q = x * r;
    return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
  }
};
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// e^-x for x >= 0, off by the rounding of x log2 e and a last place; the
// instruction gives zero for what is subnormal, so that is formed 2^64 larger.
__device__ __forceinline__ float exp_minus(float x) {
  const float t = x * -1.44269504f;
  const bool small = t < -126.0f;
  return __builtin_amdgcn_exp2f(small ? t + 64.0f : t) * (small ? 0x1p-64f : 1.0f);
}

constexpr int RP = 4, THREADS = 16 * kBlock / RP, WAVES = THREADS / kWave;   // rows of a thread
// grid: (column blocks x row blocks, matrices)
template <int OP, int MODE, bool BF16, bool VEC>
__global__ __launch_bounds__(THREADS) void k_block8_quantise(const QuantArgs a) {
  constexpr bool T = MODE != ROWS, PAIRS = OP == MOK_BLOCK8_COPY && BF16 && VEC;
  constexpr int PITCH = 128 + 8;
  __shared__ __attribute__((aligned(16))) uint8_t tile[T ? 128 * PITCH : 16];
  __shared__ uint32_t s_max[MODE == LINES ? WAVES : 1][128];
  __shared__ float2 s_scale[MODE == LINES ? 128 : 1];
  __shared__ uint32_t s_all[WAVES];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int c8 = tid & 15, rg = tid >> 4;
  const int cb = blockIdx.x % a.col_blocks, rb = blockIdx.x / a.col_blocks;
  const int col = cb * kBlock + 8 * c8;

  // ---- rows of the tile
  int64_t row0;
  int nrows;
  if (MODE == WEIGHTS) {
    row0 = static_cast<int64_t>(rb) * kBlock;
    nrows = a.rows - static_cast<int>(row0) < kBlock ? a.rows - static_cast<int>(row0) : kBlock;
  } else if (MODE == ROWS) {
    int32_t R = a.rows;
    if (a.offsets) {
      R = a.offsets[a.n_local];
      R = R < 0 ? 0 : R > a.rows ? a.rows : R;
    }
    row0 = static_cast<int64_t>(rb) * kBlock;
    if (row0 >= R) return;
    nrows = R - static_cast<int>(row0) < kBlock ? R - static_cast<int>(row0) : kBlock;
  } else {
    const ExpertRows ex(a.offsets, a.n_local, a.rows, lane);
    int units[4], e, before;
#pragma unroll
    for (int i = 0; i < 4; ++i) units[i] = (ex.count[i] + kBlock - 1) / kBlock;
    int32_t first, count;
    if (!ex.find(units, rb, lane, e, before, first, count)) return;
    const int j = (rb - before) * kBlock;
    row0 = static_cast<int64_t>(first) + j;
    nrows = count - j < kBlock ? count - j : kBlock;
  }
  const int64_t mat = MODE == WEIGHTS ? static_cast<int64_t>(blockIdx.y) * a.rows * a.W : 0;

  // ---- values: rows RP rg .. RP rg + RP - 1, columns 8 c8 .. 8 c8 + 7
  Row8<PAIRS> v[RP];
  const int half = a.W / 2;                     // MOK_BLOCK8_SWIGLU_BWD: I
#pragma unroll
  for (int p = 0; p < RP; ++p) {
    const int r = RP * rg + p;
    v[p].clear();
    if (r >= nrows || col >= a.W) continue;
    const int64_t row = row0 + r;
    if constexpr (OP == MOK_BLOCK8_COPY) {
      const int64_t at = MODE != WEIGHTS && a.ring_rows
                             ? colblk_byte(row % a.ring_rows, a.ring_rows, 2 * col) / 2
                             : mat + row * a.ld + col;
      if constexpr (PAIRS) v[p].set(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at));
      else load8<BF16, VEC>(a.x, at, v[p].v);
    } else {
      const int I = OP == MOK_BLOCK8_SWIGLU ? a.W : half;
      const bool up = OP == MOK_BLOCK8_SWIGLU_BWD && col >= I;   // the du half
      const int c = up ? col - I : col;
      float g[8], u[8], d[8];
      load8<BF16, VEC>(a.x, row * a.ld + c, g);
      if (!up) load8<BF16, VEC>(a.x, row * a.ld + I + c, u);
      if (OP == MOK_BLOCK8_SWIGLU_BWD) load8<BF16, VEC>(a.d, row * a.ldd + c, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // s and 1 - s from e^-|g|, which does not overflow: both keep their digits down to the subnormal
        const float e = exp_minus(fabsf(g[i])), one = 1.0f + e;
        float near1 = __builtin_amdgcn_rcpf(one);
        near1 = __builtin_fmaf(__builtin_fmaf(-one, near1, 1.0f), near1, near1);
        const float near0 = e * near1;
        const float s = g[i] < 0.0f ? near0 : near1, t = g[i] < 0.0f ? near1 : near0;
        if (OP == MOK_BLOCK8_SWIGLU) v[p].v[i] = g[i] * s * u[i];
        else v[p].v[i] = up ? d[i] * g[i] * s : d[i] * u[i] * s * (1.0f + g[i] * t);
      }
    }
  }

  // ---- largest magnitudes of the thread's rows and columns, of the tile (and
  // of its columns, in LDS).  If one is not finite they are formed once more
  // without such values.
  uint32_t row_max[RP], all = 0;
  auto maxima = [&](bool finite) {
    uint32_t col_max[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) col_max[i] = 0;
    if (PAIRS && finite) {
      if constexpr (PAIRS) {
        uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = v[p].w[i] & 0x7fff7fffu;
            cm[i] = max_pairs(cm[i], w[i]);
          }
          const uint32_t m = max_pairs(max_pairs(w[0], w[1]), max_pairs(w[2], w[3]));
          row_max[p] = umax(m << 16, m & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          col_max[2 * i] = cm[i] << 16;
          col_max[2 * i + 1] = cm[i] & 0xffff0000u;
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < RP; ++p) {
        row_max[p] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = v[p][i];
          if (!finite) asm volatile("" : "+v"(x));   // not kept from the first time: 64 registers
          uint32_t m = magnitude(x);
          if (!finite && m >= kInf) m = 0;
          row_max[p] = umax(row_max[p], m);
          col_max[i] = umax(col_max[i], m);
        }
      }
    }
    all = 0;
#pragma unroll
    for (int p = 0; p < RP; ++p) all = umax(all, row_max[p]);
    all = max16(all);
    all = umax(all, __shfl_xor(all, 16));
    all = umax(all, __shfl_xor(all, 32));
    if (lane == 0) s_all[wave] = all;
    if constexpr (MODE == LINES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = umax(col_max[i], __shfl_xor(col_max[i], 16));
        m = umax(m, __shfl_xor(m, 32));
        if (lane < 16) s_max[wave][8 * c8 + i] = m;
      }
    }
    __syncthreads();
    all = s_all[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) all = umax(all, s_all[w]);
  };
  maxima(true);
  if (__builtin_expect(all >= kInf, 0)) {
    __syncthreads();
    maxima(false);
  }
  // What is converted: NaN (of which the conversion makes 0xff) for a value that
  // is not finite: of infinity the correction makes it.
  auto quotient = [&](const Scale& s, int p, int i) { return s(v[p][i]); };

  // ---- the rows' codes
  const Scale whole(MODE == BLOCKS || MODE == WEIGHTS ? all : 0);
  if (MODE == WEIGHTS || a.codes) {
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const Scale s = MODE == WEIGHTS ? whole : Scale(max16(row_max[p]));
      const int row = RP * rg + p;
      if (row < nrows && col < a.W) {
        uint2 w;
        w.x = pack4(quotient(s, p, 0), quotient(s, p, 1), quotient(s, p, 2), quotient(s, p, 3));
        w.y = pack4(quotient(s, p, 4), quotient(s, p, 5), quotient(s, p, 6), quotient(s, p, 7));
        *reinterpret_cast<uint2*>(a.codes + mat + (row0 + row) * a.W + col) = w;
        if (MODE != WEIGHTS && c8 == 0) a.scales[static_cast<int64_t>(cb) * a.rows + row0 + row] = s.s;
      }
      if (PAIRS) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // ---- the transposed codes
  if constexpr (T) {
    if constexpr (PAIRS) {                      // not unpacked twice over: 64 registers
#pragma unroll
      for (int p = 0; p < RP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(v[p].w[i]));
    }
    __builtin_amdgcn_sched_barrier(0);
    if (MODE != WEIGHTS || a.codes_t) {
      if constexpr (MODE == LINES) {            // a column's scale once, for all of its threads
        if (tid < kBlock) {
          uint32_t m = s_max[0][tid];
#pragma unroll
          for (int w = 1; w < WAVES; ++w) m = umax(m, s_max[w][tid]);
          const Scale s(m);
          s_scale[tid] = make_float2(s.s, s.r);
          if (cb * kBlock + tid < a.W) a.scales_t[static_cast<int64_t>(rb) * a.W + cb * kBlock + tid] = s.s;
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 8 * c8 + i;
        Scale s = whole;
        if constexpr (MODE == LINES) {
          const float2 x = s_scale[c];
          s.s = x.x;
          s.r = x.y;
        }
        *reinterpret_cast<uint32_t*>(tile + c * PITCH + RP * rg) =
            pack4(quotient(s, 0, i), quotient(s, 1, i), quotient(s, 2, i), quotient(s, 3, i));
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      // columns of the tile: 8 lanes and 16 bytes each; a matrix's last block of rows may be half one
      const int64_t place = MODE == WEIGHTS ? row0 : static_cast<int64_t>(rb) * kBlock;
#pragma unroll
      for (int k = 0; k < 128 * 8 / THREADS; ++k) {
        const int c = THREADS / 8 * k + tid / 8, at = tid % 8 * 16;
        if (cb * kBlock + c < a.W && (MODE != WEIGHTS || at < nrows)) {
          const uint2 lo = *reinterpret_cast<const uint2*>(tile + c * PITCH + at);
          const uint2 hi = *reinterpret_cast<const uint2*>(tile + c * PITCH + at + 8);
          *reinterpret_cast<uint4*>(a.codes_t + mat + (static_cast<int64_t>(cb) * kBlock + c) * a.S + place + at) =
              make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
    if (MODE != LINES && tid == 0) {
      if (MODE == BLOCKS) {
        a.scales_t[cb * (a.S / kBlock) + rb] = whole.s;
      } else {
        const int64_t col_blocks = a.col_blocks, row_blocks = (a.rows + kBlock - 1) / kBlock, each = row_blocks * col_blocks;
        a.scales[blockIdx.y * each + rb * col_blocks + cb] = whole.s;
        if (a.codes_t) a.scales_t[blockIdx.y * each + cb * row_blocks + rb] = whole.s;
      }
    }
  }
}

template <int OP, int MODE, bool BF16>
hipError_t run(const QuantArgs& a, bool vec, dim3 grid, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((k_block8_quantise<OP, MODE, BF16, true>), grid, dim3(THREADS), 0, s, a);
  else hipLaunchKernelGGL((k_block8_quantise<OP, MODE, BF16, false>), grid, dim3(THREADS), 0, s, a);
  return hipGetLastError();
}
template <int OP, int MODE> hipError_t run(const QuantArgs& a, bool bf16, bool vec, dim3 grid, hipStream_t s) {
  return bf16 ? run<OP, MODE, true>(a, vec, grid, s) : run<OP, MODE, false>(a, vec, grid, s);
}
template <int MODE> hipError_t run(const QuantArgs& a, int op, bool bf16, bool vec, dim3 grid, hipStream_t s) {
  switch (op) {
    case MOK_BLOCK8_COPY: return run<MOK_BLOCK8_COPY, MODE>(a, bf16, vec, grid, s);
    case MOK_BLOCK8_SWIGLU: return run<MOK_BLOCK8_SWIGLU, MODE>(a, bf16, vec, grid, s);
    default: return run<MOK_BLOCK8_SWIGLU_BWD, MODE>(a, bf16, vec, grid, s);
  }
}

// Whether rows of `ld` elements of `size` bytes from p all begin at multiples of 16 bytes.
bool aligned(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

}  // namespace

hipError_t launch_block8_quantise(const mok_block8_source& src, int32_t rows, int32_t W,
                                  const int32_t* offsets, int32_t n_local, uint8_t* codes,
                                  float* scales, uint8_t* codes_t, float* scales_t, bool blocks,
                                  hipStream_t s) {
  if (rows == 0) return hipSuccess;
  QuantArgs a{};
  a.x = src.x; a.ld = src.ld; a.d = src.d; a.ldd = src.ldd;
  a.ring_rows = src.ring_rows;
  a.rows = rows; a.W = W; a.offsets = offsets; a.n_local = n_local;
  a.codes = codes; a.scales = scales; a.codes_t = codes_t; a.scales_t = scales_t;
  a.S = block8_slots(rows, n_local);
  a.col_blocks = (W + kBlock - 1) / kBlock;
  const bool bf16 = src.type == MOK_TYPE_BF16;
  const int size = bf16 ? 2 : 4;
  const bool vec = src.ring_rows ? reinterpret_cast<uintptr_t>(src.x) % 16 == 0
                                 : aligned(src.x, src.ld, size) &&
                                       (src.op != MOK_BLOCK8_SWIGLU_BWD || aligned(src.d, src.ldd, size));
  // without transposed codes the tiles go over the rows as they lie
  const int64_t row_blocks = codes_t ? a.S / kBlock : (static_cast<int64_t>(rows) + kBlock - 1) / kBlock;
  const dim3 grid(static_cast<unsigned>(row_blocks * a.col_blocks));
  if (!codes_t) return run<ROWS>(a, src.op, bf16, vec, grid, s);
  return blocks ? run<BLOCKS>(a, src.op, bf16, vec, grid, s) : run<LINES>(a, src.op, bf16, vec, grid, s);
}

hipError_t launch_block8_weights(const void* w, bool bf16, int32_t n, int32_t N, int32_t K,
                                 uint8_t* codes, float* scales, uint8_t* codes_t, float* scales_t,
                                 hipStream_t s) {
  if (n == 0) return hipSuccess;
  QuantArgs a{};
  a.x = w; a.ld = K; a.rows = N; a.W = K; a.n_local = 1;
  a.codes = codes; a.scales = scales; a.codes_t = codes_t; a.scales_t = scales_t;
  a.S = N;
  a.col_blocks = (K + kBlock - 1) / kBlock;
  const dim3 grid(static_cast<unsigned>(a.col_blocks * ((N + kBlock - 1) / kBlock)), static_cast<unsigned>(n));
  return run<MOK_BLOCK8_COPY, WEIGHTS>(a, bf16, aligned(w, K, bf16 ? 2 : 4), grid, s);
}

}  // namespace mok
