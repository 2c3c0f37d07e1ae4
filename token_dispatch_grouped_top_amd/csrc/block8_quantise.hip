// block8_quantise.hip -- E4M3 codes with fp32 scales for blocks of 128: of
// token rows (optionally through SwiGLU or its backward), of the same rows
// transposed into slot blocks, and of weight matrices.
//
// scale = max(amax / 448, 2^-126), code = RNE(fl(value / scale)).  One
// workgroup takes 128 rows x 128 columns, reads them once into registers (8 x 8
// values a thread) and forms every scale that the tile has: of its rows, of
// its columns, of the whole.  The transposed codes go through LDS, so that both
// outputs are written in whole lines.  Bound: bytes.
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

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// Largest of the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ float max16(float m) {
#define MOK_ROT(n)                                                                                  \
  m = fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), 0x120 + (n), 0xf, \
                                                           0xf, true)))
  MOK_ROT(8); MOK_ROT(4); MOK_ROT(2); MOK_ROT(1);
#undef MOK_ROT
  return m;
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / 448.0f, 0x1p-126f); }

// x / s rounded as fp32 division rounds it: a quotient from the reciprocal r
// of s (itself rounded correctly) and one correction, which would lose the
// sign of a zero.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);
}
// What is converted: at most 448 in magnitude, NaN (of which the conversion makes 0xff) for a value that is not finite.
__device__ __forceinline__ float to_code(float x, float s, float r) {
  return finite(x) ? __builtin_amdgcn_fmed3f(quotient(x, s, r), -448.0f, 448.0f) : __builtin_nanf("");
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// grid: (column blocks x row blocks, matrices)
template <int OP, int MODE, bool BF16, bool VEC>
__global__ __launch_bounds__(256) void k_block8_quantise(const QuantArgs a) {
  constexpr bool T = MODE != ROWS;
  constexpr int PITCH = 128 + 8;
  __shared__ __attribute__((aligned(16))) uint8_t tile[T ? 128 * PITCH : 16];
  __shared__ float s_max[4][128];
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

  // ---- values: rows 8 rg .. 8 rg + 7, columns 8 c8 .. 8 c8 + 7
  float v[8][8];
  const int half = a.W / 2;                     // MOK_BLOCK8_SWIGLU_BWD: I
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = 8 * rg + p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
    if (r >= nrows || col >= a.W) continue;
    const int64_t row = row0 + r;
    if constexpr (OP == MOK_BLOCK8_COPY) {
      if (MODE != WEIGHTS && a.ring_rows)
        load8<BF16, VEC>(a.x, colblk_byte(row % a.ring_rows, a.ring_rows, 2 * col) / 2, v[p]);
      else
        load8<BF16, VEC>(a.x, mat + row * a.ld + col, v[p]);
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
        const float e = expf(-fabsf(g[i])), near1 = 1.0f / (1.0f + e), near0 = e * near1;
        const float s = g[i] < 0.0f ? near0 : near1, t = g[i] < 0.0f ? near1 : near0;
        if (OP == MOK_BLOCK8_SWIGLU) v[p][i] = g[i] * s * u[i];
        else v[p][i] = up ? d[i] * g[i] * s : d[i] * u[i] * s * (1.0f + g[i] * t);
      }
    }
  }

  // ---- scales of the rows, and their codes
  float row_max[8], col_max[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) col_max[i] = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = finite(v[p][i]) ? fabsf(v[p][i]) : 0.0f;
      m = fmaxf(m, x);
      col_max[i] = fmaxf(col_max[i], x);
    }
    row_max[p] = m;
  }
  float block_scale = 0.0f, col_scale[8];
  if constexpr (T) {
    if constexpr (MODE == LINES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        col_max[i] = fmaxf(col_max[i], __shfl_xor(col_max[i], 16));
        col_max[i] = fmaxf(col_max[i], __shfl_xor(col_max[i], 32));
        if (lane < 16) s_max[wave][8 * c8 + i] = col_max[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 8 * c8 + i;
        col_scale[i] = scale_of(fmaxf(fmaxf(s_max[0][c], s_max[1][c]), fmaxf(s_max[2][c], s_max[3][c])));
      }
    } else {
      float m = row_max[0];
#pragma unroll
      for (int p = 1; p < 8; ++p) m = fmaxf(m, row_max[p]);
      m = max16(m);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      if (lane == 0) s_max[wave][0] = m;
      __syncthreads();
      block_scale = scale_of(fmaxf(fmaxf(s_max[0][0], s_max[1][0]), fmaxf(s_max[2][0], s_max[3][0])));
#pragma unroll
      for (int i = 0; i < 8; ++i) col_scale[i] = block_scale;
    }
  }
  if (MODE == WEIGHTS || a.codes) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float s = MODE == WEIGHTS ? block_scale : scale_of(max16(row_max[p]));
      const float r = 1.0f / s;
      const int row = 8 * rg + p;
      if (row < nrows && col < a.W) {
        uint2 w;
        w.x = pack4(to_code(v[p][0], s, r), to_code(v[p][1], s, r), to_code(v[p][2], s, r), to_code(v[p][3], s, r));
        w.y = pack4(to_code(v[p][4], s, r), to_code(v[p][5], s, r), to_code(v[p][6], s, r), to_code(v[p][7], s, r));
        *reinterpret_cast<uint2*>(a.codes + mat + (row0 + row) * a.W + col) = w;
        if (MODE != WEIGHTS && c8 == 0) a.scales[static_cast<int64_t>(cb) * a.rows + row0 + row] = s;
      }
    }
  }

  // ---- the transposed codes
  if constexpr (T) {
    if (MODE != WEIGHTS || a.codes_t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = col_scale[i], r = 1.0f / s;
        uint2 w;
        w.x = pack4(to_code(v[0][i], s, r), to_code(v[1][i], s, r), to_code(v[2][i], s, r), to_code(v[3][i], s, r));
        w.y = pack4(to_code(v[4][i], s, r), to_code(v[5][i], s, r), to_code(v[6][i], s, r), to_code(v[7][i], s, r));
        *reinterpret_cast<uint2*>(tile + (8 * c8 + i) * PITCH + 8 * rg) = w;
      }
      __syncthreads();
      // columns of the tile: 8 lanes and 16 bytes each; a matrix's last block of rows may be half one
      const int64_t place = MODE == WEIGHTS ? row0 : static_cast<int64_t>(rb) * kBlock;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = 32 * k + tid / 8, at = tid % 8 * 16;
        if (cb * kBlock + c < a.W && (MODE != WEIGHTS || at < nrows)) {
          const uint2 lo = *reinterpret_cast<const uint2*>(tile + c * PITCH + at);
          const uint2 hi = *reinterpret_cast<const uint2*>(tile + c * PITCH + at + 8);
          *reinterpret_cast<uint4*>(a.codes_t + mat + (static_cast<int64_t>(cb) * kBlock + c) * a.S + place + at) =
              make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
    const int64_t col_blocks = a.col_blocks;
    if (MODE == LINES) {
      if (tid < 16 && col < a.W) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a.scales_t[static_cast<int64_t>(rb) * a.W + col + i] = col_scale[i];
      }
    } else if (tid == 0) {
      if (MODE == BLOCKS) {
        a.scales_t[cb * (a.S / kBlock) + rb] = block_scale;
      } else {
        const int64_t row_blocks = (a.rows + kBlock - 1) / kBlock, each = row_blocks * col_blocks;
        a.scales[blockIdx.y * each + rb * col_blocks + cb] = block_scale;
        if (a.codes_t) a.scales_t[blockIdx.y * each + cb * row_blocks + rb] = block_scale;
      }
    }
  }
}

template <int OP, int MODE, bool BF16>
hipError_t run(const QuantArgs& a, bool vec, dim3 grid, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((k_block8_quantise<OP, MODE, BF16, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_block8_quantise<OP, MODE, BF16, false>), grid, dim3(256), 0, s, a);
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
