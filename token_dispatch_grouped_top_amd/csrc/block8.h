// block8.h -- launchers of the 8-bit block quantisers and products, and the
// expert lookup that their kernels share.
#pragma once

#include "mok_internal.h"

namespace mok {

constexpr int kBlock = 128;                    // values of a scale

// Places of a transposed operand's rows (0 rows: the empty experts' share of the formula).
inline int64_t block8_slots(int64_t rows, int64_t n_local) {
  return kBlock * ((rows + kBlock - 1) / kBlock + n_local - 1);
}

hipError_t launch_block8_quantise(const mok_block8_source& src, int32_t rows, int32_t W,
                                  const int32_t* offsets, int32_t n_local, uint8_t* codes,
                                  float* scales, uint8_t* codes_t, float* scales_t, bool blocks,
                                  hipStream_t s);
hipError_t launch_block8_weights(const void* w, bool bf16, int32_t n, int32_t N, int32_t K,
                                 uint8_t* codes, float* scales, uint8_t* codes_t, float* scales_t,
                                 hipStream_t s);

struct Block8Product {
  const uint8_t* t; const float* t_scales;     // token operand [t_rows][K or S]
  const uint8_t* w; const float* w_scales;     // weight operand
  const int32_t* offsets; int32_t n_local;
  int32_t rows;                                // routed rows (capacity)
  int32_t K, N;                                // forward: K contracted; N output columns
  int32_t M;                                   // gradient: output rows of an expert
  int32_t S;                                   // gradient: places of the operands' rows
  void* out;
  int32_t bf16, accumulate;
  int32_t n_cus;                               // of the device
};
hipError_t launch_block8_gemm(const Block8Product& p, hipStream_t s);
hipError_t launch_block8_wgrad(const Block8Product& p, hipStream_t s);

#ifdef __HIPCC__
// Rows of every expert, four experts to a lane: first[i] and count[i] of
// expert 4 * lane + i, within [0, rows) whatever the offsets hold.
struct ExpertRows {
  int32_t first[4], count[4];
  __device__ __forceinline__ ExpertRows(const int32_t* offsets, int32_t n_local, int32_t rows, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      int32_t a = 0, b = 0;
      if (e < n_local) {
        a = offsets ? offsets[e] : 0;
        b = offsets ? offsets[e + 1] : rows;
        a = a < 0 ? 0 : a > rows ? rows : a;
        b = b < a ? a : b > rows ? rows : b;
      }
      first[i] = a;
      count[i] = b - a;
    }
  }
  // The expert whose run of units[0..3] per lane holds unit t of all of them in
  // order; false past the last.  `before`: units of the experts before it;
  // `slots`: the places before it, each expert's count rounded up to a block.
  __device__ __forceinline__ bool find(const int (&units)[4], int t, int lane, int& e, int& before,
                                       int32_t& row0, int32_t& rows_e, int64_t* slots = nullptr) const {
    int sum = units[0] + units[1] + units[2] + units[3], upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(upto, d);
      if (lane >= d) upto += x;
    }
    const uint64_t past = __ballot(upto > t);
    if (past == 0) return false;
    const int l = __ffsll(static_cast<unsigned long long>(past)) - 1;
    int at = __shfl(upto - sum, l), i = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int u = __shfl(units[j], l);
      if (i == j && at + u <= t) { at += u; i = j + 1; }
    }
    e = __builtin_amdgcn_readfirstlane(4 * l + i);
    before = __builtin_amdgcn_readfirstlane(at);
    int32_t f = first[0], c = count[0];
#pragma unroll
    for (int j = 1; j < 4; ++j) {
      f = i == j ? first[j] : f;
      c = i == j ? count[j] : c;
    }
    row0 = __builtin_amdgcn_readfirstlane(__shfl(f, l));
    rows_e = __builtin_amdgcn_readfirstlane(__shfl(c, l));
    if (slots) {
      int blocks = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        blocks += 4 * lane + j < e ? (count[j] + kBlock - 1) / kBlock : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) blocks += __shfl_xor(blocks, d);
      *slots = static_cast<int64_t>(kBlock) * __builtin_amdgcn_readfirstlane(blocks);
    }
    return true;
  }
};
#endif

}  // namespace mok
