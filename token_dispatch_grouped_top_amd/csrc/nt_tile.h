// nt_tile.h -- parts of products of two operands whose rows lie along the
// contraction ("row-major, K contiguous"): what the 8-bit block products
// (block8_gemm.hip) and the fp16 products of the orthogonalised update
// (muon.hip) have in common -- types, the wait that ends a step, the order of a
// step's reads, loads and matrix instructions -- and the tile shape and loader
// of the former.  Each file has its own loop: the block products step by 128
// bytes of a row (128 codes: one cache line of HBM, 8 chunks of 16 bytes in
// LDS), the update by column blocks of 64 bytes (32 fp16 values).
//
// Roles: D[i][j] = sum_k W[i][k] T[j][k] with W the MFMA's first operand, so a
// lane holds, for one row j of T, runs of four consecutive i.  An output whose
// rows are j has i as its contiguous direction.
//
// Loads go straight to LDS (buffer loads with 16 bytes a lane, NS stages); a
// row or chunk outside an operand reads as zero through the buffer's extent.
// A chunk's place in its row depends on the row, which a lane realises by what
// it asks for, since the direct load puts lanes behind each other; for 128-byte
// rows chunk c of row r lies at place c ^ key(r).
#pragma once

#include "mok_internal.h"

namespace mok {
namespace nt {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kRow = 128;                      // bytes of a row in a stage
constexpr uint32_t kOutside = 0xfffffff0u;     // a buffer offset past every extent

// Place of logical chunk c of row r: eight rows behind each other hold one
// chunk at eight different places, and the next eight rows at the other four
// of each pair, so a fragment's 16-byte reads spread over the banks.
__device__ __forceinline__ int chunk_at(int r, int c) { return c ^ ((r & 7) ^ ((r >> 3) & 1)); }

template <int N> __device__ __forceinline__ void wait_vm_barrier() {
  static_assert(N >= 0 && N <= 63, "vmcnt range");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Asks the scheduler to put one of A LDS reads behind each of the first of M
// matrix instructions, and B loads from memory evenly behind the others.  (Reads
// come first in the program, too: a load to LDS does not pass a read.)
template <int M, int A, int B, int m = 0> __device__ __forceinline__ void interleave() {
  if constexpr (m < M) {
    constexpr int per = A >= M ? (A + M - 1) / M : 1, from = A >= M ? M - 1 : A;
    constexpr int reads = m * per < A ? (A - m * per < per ? A - m * per : per) : 0;
    constexpr int loads = m < from ? 0 : B * (m + 1 - from) / (M - from) - B * (m - from) / (M - from);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
    interleave<M, A, B, m + 1>();
  }
}

// TT x TW: rows of T and of W in a workgroup's tile; WT x WW waves; NS stages,
// each with a 4-byte slot for a scale a thread.
template <int TT_, int TW_, int WT_, int WW_, int NS_> struct Geo {
  static constexpr int TT = TT_, TW = TW_, WT = WT_, WW = WW_, NS = NS_;
  static constexpr int WAVES = WT * WW, THREADS = 64 * WAVES;
  static constexpr int FT = TT / WT / 32, FW = TW / WW / 32;       // 32-row fragments of a wave
  static constexpr int LT = TT * kRow / 1024 / WAVES, LW = TW * kRow / 1024 / WAVES;   // loads of a wave
  static constexpr int LPS = LT + LW + 1;
  static constexpr int STAGE = (TT + TW) * kRow + THREADS * 4;
  static constexpr int EPI = WAVES * 32 * (32 * FW + 4) * 4;       // a wave's 32 rows of fp32 results
  static constexpr int LDS = NS * STAGE > EPI ? NS * STAGE : EPI;
  static_assert(FT >= 1 && FW >= 1 && LT >= 1 && LW >= 1, "every wave loads and multiplies");
  static_assert(TT + TW / 128 + 1 <= THREADS, "a thread for each scale");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

// One operand of a tile: `base` at the tile's first row and first K-step.
struct Operand {
  const uint8_t* base;
  int64_t stride;              // bytes between rows
  int64_t extent;              // bytes from base on that may be read
};

// Loads of an operand's rows, eight rows (1 KiB) an instruction: wave `wave` of
// WAVES takes KiB j * WAVES + wave of a stage.  A lane's row and chunk in the
// first of its KiB are one offset; the others lie whole rows further on (the
// chunk's place is the same: WAVES is even).  Rows past the operand's last lie
// past its extent.
template <int WAVES> struct Loader {
  static_assert(WAVES % 2 == 0, "a lane's chunk is the same in all of its KiB");
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t at;                 // offset of step 0
  uint32_t next;               // bytes to the next KiB's rows
  bool far;                    // a chunk that a half step does not have
  __device__ __forceinline__ Loader(const Operand& o, int wave, int lane) {
    const int64_t e = o.extent < 0xfffffff0ll ? o.extent : 0xfffffff0ll;
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.base), 0, static_cast<int32_t>(e),
                                             0x00020000);
    const int r = wave * 8 + lane / 8, c = chunk_at(r, lane % 8);
    at = static_cast<uint32_t>(r * o.stride + c * 16);
    far = c >= 4;
    next = static_cast<uint32_t>(WAVES * 8 * o.stride);
  }
  template <int J> __device__ __forceinline__ void load(uint8_t* stage, int wave, uint32_t step, bool half) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(stage + (J * WAVES + wave) * 1024), 16, half && far ? kOutside : at,
                                             step * kRow + J * next, 0, 0);
  }
};

// LDS address of a fragment chunk: rows 32 f + lane % 32 of a wave's block,
// whose first row is a multiple of 32; the place of a chunk depends on the
// lane alone.
__device__ __forceinline__ u32x4_t chunk16(const uint8_t* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}

}  // namespace nt
}  // namespace mok
