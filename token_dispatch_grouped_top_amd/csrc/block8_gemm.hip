// block8_gemm.hip -- products of E4M3 operands with fp32 scales: one for 128
// values of a token row, one for 128 x 128 values of a weight matrix.
//
//   out[j][i] = sum_b t_scale[b][j] w_scale[i / 128][b] P_b[i][j],
//   P_b[i][j] = sum_{k in block b} w[i][k] t[j][k]
//
// P_b is two v_mfma_f32_32x32x64_f8f6f4 that start from zero; the scales enter
// when it is added to the accumulator: one fma a value, with a factor that is
// the same for all of a lane's values of a fragment, because a lane's values
// share the row j and a wave's columns lie within one block of 128.  (Feeding
// the weights as the first operand is what puts j on the lanes.)  16 values a
// lane and 64 cycles of fma stand against 128 cycles of matrix instructions, a
// SIMD has two waves, and each of them has the fma of one block behind the
// matrix instructions of the next.  That hides the fma in part: of a CU's busy
// cycles the matrix units work in 46 % and vector instructions issue in 38 %,
// LDS reads in 24 % (8192 rows of 8 experts, 7168 -> 4096: 280 us).
//
// gfx950's 8-bit matrix instructions add up a group of products aligned to the
// largest of them and drop what lies below 2^-13 of it (whole products below
// 2^-13 vanish; at random codes a sum is off by 1e-5 to 5e-5 of its size).
// That is far below a result in bf16 (where one product of the 64 is much larger
// than their sum it can reach 63 x 2^-13 of that one, a step of bf16), but not
// what a result in fp32 is asked for: such a one (EXACT) is formed by v_mfma_f32_32x32x16_f16 from the codes
// converted to fp16, which holds them all, at half the rate, with sums as exact
// as fp32's.
//
// The gradient of the weights is the same product over slot blocks: dy_t takes
// the tokens' place (a scale for 128 slots of a column), x_t the weights'.
#include <type_traits>

#include "block8.h"
#include "nt_tile.h"

namespace mok {
namespace {

using namespace nt;

// The two 64-byte halves of a 128-byte row as MFMA operands: lane half h takes
// chunks h and 2 + h of each half; any split will do that both operands share.
__device__ __forceinline__ i32x8_t frag(const uint8_t* rows, int lane, int half) {
  const int r = lane & 31, h = lane >> 5;
  const u32x4_t lo = chunk16(rows + r * kRow + chunk_at(r, 4 * half + h) * 16);
  const u32x4_t hi = chunk16(rows + r * kRow + chunk_at(r, 4 * half + 2 + h) * 16);
  return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Codes 8 g .. 8 g + 7 of a chunk in fp16.
__device__ __forceinline__ f16x8_t to_f16(u32x4_t c, int g) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const uint32_t a = c[2 * g], b = c[2 * g + 1];
  const auto p = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false));
  const auto q = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true));
  const auto r = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
  const auto s = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
  return f16x8_t{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}

// One step of a wave: acc += scales * (block product), with the codes of its
// rows of the two stages.
template <class G, bool EXACT>
__device__ __forceinline__ void block8_step(f32x16_t (&acc)[G::FW][G::FT], const uint8_t* T, const uint8_t* W,
                                            const float* t_scale, float sw, int lane) {
  const int r = lane & 31, h = lane >> 5;
  if constexpr (EXACT) {
    // lane half h takes chunks 2 k + h: codes 8 g .. 8 g + 7 of both operands meet
    u32x4_t wq[G::FW][4];
#pragma unroll
    for (int i = 0; i < G::FW; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) wq[i][k] = chunk16(W + (32 * i + r) * kRow + chunk_at(r, 2 * k + h) * 16);
#pragma unroll
    for (int j = 0; j < G::FT; ++j) {
      f16x8_t tq[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u32x4_t c = chunk16(T + (32 * j + r) * kRow + chunk_at(r, 2 * k + h) * 16);
#pragma unroll
        for (int g = 0; g < 2; ++g) tq[k][g] = to_f16(c, g);
      }
      const float f = sw * t_scale[32 * j + r];
#pragma unroll
      for (int i = 0; i < G::FW; ++i) {
        f32x16_t part;
#pragma unroll
        for (int k = 0; k < 16; ++k) part[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int g = 0; g < 2; ++g)
            part = __builtin_amdgcn_mfma_f32_32x32x16_f16(to_f16(wq[i][k], g), tq[k][g], part, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][j][k] = __builtin_fmaf(part[k], f, acc[i][j][k]);
      }
    }
  } else {
    i32x8_t wf[G::FW][2];
#pragma unroll
    for (int i = 0; i < G::FW; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) wf[i][k] = frag(W + 32 * i * kRow, lane, k);
#pragma unroll
    for (int j = 0; j < G::FT; ++j) {
      const i32x8_t t0 = frag(T + 32 * j * kRow, lane, 0), t1 = frag(T + 32 * j * kRow, lane, 1);
      const float f = sw * t_scale[32 * j + r];
#pragma unroll
      for (int i = 0; i < G::FW; ++i) {
        f32x16_t part;
#pragma unroll
        for (int k = 0; k < 16; ++k) part[k] = 0.0f;
        part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i][0], t0, part, 0, 0, 0, 0, 0, 0);
        part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i][1], t1, part, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][j][k] = __builtin_fmaf(part[k], f, acc[i][j][k]);
      }
    }
  }
}

// What a workgroup computes: the G::TT x G::TW results of expert e from row t0
// (of its t_all) and column i0 on.
struct Job {
  int e, t0, i0, t_all;
  int32_t row0, count;         // the expert's rows
  int64_t slots;               // its first place
};

template <class G, bool WGRAD, bool EXACT>
__device__ __forceinline__ void block8_tile(const Block8Product& p, const Job& job, uint8_t* __restrict__ lds) {
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int e = job.e, t0 = job.t0, i0 = job.i0, t_all = job.t_all;
  const int32_t row0 = job.row0, count = job.count;
  const int64_t slots = job.slots;

  // ---- operands
  const int t_rows = t_all - t0 < G::TT ? t_all - t0 : G::TT;
  const int w_rows = p.N - i0 < G::TW ? p.N - i0 : G::TW;
  const int steps = WGRAD ? (count + kBlock - 1) / kBlock : (p.K + kBlock - 1) / kBlock;
  const bool half = !WGRAD && p.K % kBlock != 0;           // the last step has 64 codes of a row
  Operand ot, ow;
  const float *ts, *ws;                                    // scales of row j, of row i, at block 0
  int64_t ts_step;                                         // elements between blocks (of ws: 1)
  if (WGRAD) {
    ot.stride = ow.stride = p.S;
    ot.base = p.t + static_cast<int64_t>(t0) * p.S + slots;
    ow.base = p.w + static_cast<int64_t>(i0) * p.S + slots;
    ot.extent = static_cast<int64_t>(p.M - t0) * p.S - slots;
    ow.extent = static_cast<int64_t>(p.N - i0) * p.S - slots;
    ts_step = p.M;
    ts = p.t_scales + slots / kBlock * ts_step + t0;
    ws = p.w_scales + static_cast<int64_t>(i0 / kBlock) * (p.S / kBlock) + slots / kBlock;
  } else {
    ot.stride = ow.stride = p.K;
    ot.base = p.t + (static_cast<int64_t>(row0) + t0) * p.K;
    ow.base = p.w + (static_cast<int64_t>(e) * p.N + i0) * p.K;
    ot.extent = static_cast<int64_t>(t_rows) * p.K;
    ow.extent = static_cast<int64_t>(w_rows) * p.K;
    ts_step = p.rows;
    ts = p.t_scales + row0 + t0;
    ws = p.w_scales + (static_cast<int64_t>(e) * ((p.N + kBlock - 1) / kBlock) + i0 / kBlock) * steps;
  }
  const int64_t ws_row = WGRAD ? p.S / kBlock : steps;
  const Loader<G::WAVES> lt(ot, wave, lane), lw(ow, wave, lane);
  // A thread's scale of a step: of row tid of the tokens; of one of the tile's
  // blocks of weight rows from the first wave behind those on.
  static_assert(G::TT % 64 == 0, "a wave's scales are of one kind");
  const bool t_wave = wave < G::TT / 64;
  const int blocks = (w_rows + kBlock - 1) / kBlock;
  const float* scale_at = t_wave ? ts : ws;                // advanced by the steps' number times
  const int64_t scale_step = t_wave ? ts_step : 1;
  const uint32_t my_scale = t_wave ? (tid < t_rows ? tid : t_rows - 1) * 4u
                                   : static_cast<uint32_t>((lane < blocks ? lane : blocks - 1) * ws_row * 4);
  // (all stages of an operand behind each other: 64 KiB, what an offset in an instruction reaches)
  auto stage_t = [&](int b) { return lds + b * (G::TT * kRow); };
  auto stage_w = [&](int b) { return lds + G::NS * G::TT * kRow + b * (G::TW * kRow); };
  auto stage_s = [&](int b) { return lds + G::NS * (G::TT + G::TW) * kRow + b * (G::THREADS * 4); };
  // A stage's loads: tokens and scales, or weights.  Past the last step they are
  // of the last one, and nobody reads them.
  auto issue_t = [&](int step, int b) {
    step = step < steps ? step : steps - 1;
    const bool cut = half && step == steps - 1;
    static_assert(G::LT <= 4 && G::LW <= 4 && G::LT != 3 && G::LW != 3, "loads of a stage");
    lt.template load<0>(stage_t(b), wave, step, cut);
    if constexpr (G::LT > 1) lt.template load<1>(stage_t(b), wave, step, cut);
    if constexpr (G::LT > 2) { lt.template load<2>(stage_t(b), wave, step, cut); lt.template load<3>(stage_t(b), wave, step, cut); }
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(scale_at + step * scale_step), 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(stage_s(b) + wave * 256), 4, my_scale, 0, 0, 0);
  };
  auto issue_w = [&](int step, int b) {
    step = step < steps ? step : steps - 1;
    const bool cut = half && step == steps - 1;
    lw.template load<0>(stage_w(b), wave, step, cut);
    if constexpr (G::LW > 1) lw.template load<1>(stage_w(b), wave, step, cut);
    if constexpr (G::LW > 2) { lw.template load<2>(stage_w(b), wave, step, cut); lw.template load<3>(stage_w(b), wave, step, cut); }
  };

  // ---- main loop
  const int wt = wave % G::WT * (G::TT / G::WT), ww = wave / G::WT * (G::TW / G::WW);
  f32x16_t acc[G::FW][G::FT];
#pragma unroll
  for (int i = 0; i < G::FW; ++i)
#pragma unroll
    for (int j = 0; j < G::FT; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  if constexpr (!EXACT && G::FW == 2 && G::NS == 2) {
    if (steps > 0) {
      // Two stages, one block of 32 x 32 after another.  Of a step's eight blocks
      // the last one's operands are in registers when the others are done: behind
      // it stands the barrier that says that this stage is read and the next one
      // has landed, and while it is multiplied the next step's first operands are
      // read.  (A burst of reads at the start of a step, by all waves at once, left
      // the matrix units idle for as long as it took.)  The blocks go up and down
      // so that the half of the weights' fragments that the next step begins with
      // is the one that is free first; that is the other one in every second step
      // (with one row group the same in all of them).
      // The fma of a block stand behind the matrix instructions of the next.
      i32x8_t wf[2][2], tf[2][2];
      f32x16_t part[2];
      float f[G::FT], last = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) part[1][k] = 0.0f;
      // A lane's first chunk of the first row group; the other three of a row lie at
      // that address with bits 5 and 6 turned over.  They are formed where they
      // are read: kept, they would be a dozen registers of 256.
      typedef const __attribute__((address_space(3))) u32x4_t* lds_chunk_t;
      typedef const __attribute__((address_space(3))) float* lds_float_t;
      const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr_t)lds));
      const uint32_t t_at = lds0 + (wt + (lane & 31)) * kRow + chunk_at(lane & 31, lane >> 5) * 16;
      const uint32_t w_off = G::NS * G::TT * kRow + (ww - wt) * kRow;       // from there to the weights' first
      const uint32_t s_at = lds0 + G::NS * (G::TT + G::TW) * kRow + (wt + (lane & 31)) * 4;
      const uint32_t s_w = lds0 + G::NS * (G::TT + G::TW) * kRow + (G::TT + ww / kBlock) * 4;
      auto rows_at = [](uint32_t at, i32x8_t (&to)[2]) {
        u32x4_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<lds_chunk_t>(static_cast<uintptr_t>(at ^ (32u * k)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          to[h] = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(c[2 * h], c[2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7));
      };
      static_assert(G::FT == 1 || G::FT % 2 == 0, "how the blocks of a step end");
      constexpr bool ONE = G::FT == 1;                     // one row group: its fragments change places with every step
      auto read_t = [&](int b, int j, int slot) {
        uint32_t at = t_at, sc = s_at, sw = s_w;
        asm volatile("" : "+v"(at), "+v"(sc), "+s"(sw));
        rows_at(at + (b * G::TT + 32 * j) * kRow, tf[slot]);
        return *reinterpret_cast<lds_float_t>(static_cast<uintptr_t>(sc + b * G::THREADS * 4 + 128 * j)) *
               *reinterpret_cast<lds_float_t>(static_cast<uintptr_t>(sw + b * G::THREADS * 4));
      };
      auto read_w = [&](int b, int i) {
        uint32_t at = t_at;
        asm volatile("" : "+v"(at));
        rows_at(at + w_off + (b * G::TW + 32 * i) * kRow, wf[i]);
      };
      auto step = [&](int s, auto parity) {
        constexpr int P = decltype(parity)::value, B = 2 * G::FT;
        constexpr int FIRST = ONE ? 0 : P, THEN = ONE ? 0 : 1 - P;   // the halves that this step and the next begin with
        const auto column = [](int k) { return ((k + 1) / 2 + FIRST) & 1; };
        float f0 = f[0];
#pragma unroll
        for (int k = 0; k < B; ++k) {
          const int i = column(k), j = k / 2;
          if (k == B - 1) {
            wait_vm_barrier<0>();
            read_w(1 - P, THEN);
            f[0] = read_t(1 - P, 0, ONE ? 1 - P : 0);
            issue_t(s + 2, P);
          }
          if (k == 0) {
            read_w(P, 1 - FIRST);
            issue_w(s + 1, 1 - P);
          }
          if (k % 2 == 1 && k < B - 1) f[j + 1] = read_t(P, j + 1, (j + 1) & 1);
          const int slot = ONE ? P : j & 1;
          f32x16_t& p = part[k & 1];
#pragma unroll
          for (int q = 0; q < 16; ++q) p[q] = 0.0f;
          p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i][0], tf[slot][0], p, 0, 0, 0, 0, 0, 0);
          p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i][1], tf[slot][1], p, 0, 0, 0, 0, 0, 0);
          const int ii = k == 0 ? 1 - FIRST : column(k - 1), jj = k == 0 ? G::FT - 1 : (k - 1) / 2;
          const float factor = k == 0 ? last : jj == 0 ? f0 : f[jj];
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[ii][jj][q] = __builtin_fmaf(part[1 - (k & 1)][q], factor, acc[ii][jj][q]);
          __builtin_amdgcn_sched_barrier(0);
        }
        last = ONE ? f0 : f[G::FT - 1];
      };
      issue_t(0, 0);
      issue_w(0, 0);
      issue_t(1, 1);
      wait_vm_barrier<G::LT + 1>();
      read_w(0, 0);
      f[0] = read_t(0, 0, 0);
      int s = 0;
      for (; s + 1 < steps; s += 2) {
        step(s, std::integral_constant<int, 0>());
        step(s + 1, std::integral_constant<int, 1>());
      }
      if (s < steps) step(s, std::integral_constant<int, 0>());
      if (!ONE && s < steps) {
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[0][G::FT - 1][q] = __builtin_fmaf(part[1][q], last, acc[0][G::FT - 1][q]);
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[1][G::FT - 1][q] = __builtin_fmaf(part[1][q], last, acc[1][G::FT - 1][q]);
      }
    }
  } else {
    if (steps > 0) {
#pragma unroll
      for (int s = 0; s < G::NS - 1; ++s) {
        issue_t(s, s);
        issue_w(s, s);
      }
    }
    int buf = 0;
    for (int s = 0; s < steps; ++s) {
      wait_vm_barrier<(G::NS - 2) * G::LPS>();
      const int to = buf == 0 ? G::NS - 1 : buf - 1;
      issue_t(s + G::NS - 1, to);
      issue_w(s + G::NS - 1, to);
      const float* sc = reinterpret_cast<const float*>(stage_s(buf));
      block8_step<G, EXACT>(acc, stage_t(buf) + wt * kRow, stage_w(buf) + ww * kRow, sc + wt, sc[G::TT + ww / kBlock], lane);
      buf = buf + 1 == G::NS ? 0 : buf + 1;
    }
  }
  wait_vm_barrier<0>();

  // ---- results: 32 rows at a time through the wave's own part of LDS, so that
  // a row's columns are stored behind each other.  What they are added to is
  // loaded a group ahead: a load does not pass the stores.
  constexpr int CW = 32 * G::FW, PITCH = CW + 4, LPR = CW / 4, NK = 32 * LPR / 64;   // LPR: lanes of a row
  float* own = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  const int64_t out0 = WGRAD ? static_cast<int64_t>(e) * p.M + t0 : static_cast<int64_t>(row0) + t0;
  const bool add = WGRAD && EXACT && p.accumulate;
  float4 old[2][NK];
  auto place = [&](int j, int k, int64_t& o) {
    const int tr = wt + 32 * j + (k * 64 + lane) / LPR, col = i0 + ww + (k * 64 + lane) % LPR * 4;
    o = (out0 + tr) * p.N + col;
    return tr < t_rows && col < p.N && col < i0 + G::TW;
  };
  auto fetch = [&](int j) {
    if constexpr (WGRAD && EXACT) {
      int64_t o;
#pragma unroll
      for (int k = 0; k < NK; ++k)
        if (add && place(j, k, o)) old[j & 1][k] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.out) + o);
    }
  };
  fetch(0);
#pragma unroll
  for (int j = 0; j < G::FT; ++j) {
    if (j + 1 < G::FT) fetch(j + 1);
#pragma unroll
    for (int i = 0; i < G::FW; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(own + (lane & 31) * PITCH + 32 * i + 8 * g + 4 * (lane >> 5)) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // lanes read others' values
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      float4 v = *reinterpret_cast<const float4*>(own + (k * 64 + lane) / LPR * PITCH + (k * 64 + lane) % LPR * 4);
      int64_t o;
      if (!place(j, k, o)) continue;
      if constexpr (!EXACT) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      } else {
        if (add) {
          const float4 w = old[j & 1][k];
          v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = v;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // read before the next rows are written
  }
}

// Workgroup -> tile: expert by expert, columns outside, rows inside, each XCD a
// contiguous eighth of them (workgroup ids go round the XCDs); of gradients an
// eighth of each expert's, and what eight does not divide in turn, since an
// expert's tiles are as long as its slots are many (8192 slots of 8 experts, 7168 x
// 2048: half of them one expert's 210 us, 416 with an eighth of all; uneven by
// 30 % 192 / 208; even 182 / 182; smaller even ones lose up to a tenth: 4096 of 8,
// 2048 x 2048 41 / 38).  The tiles that
// would make a last round of their own, with most of the XCD's CUs idle, are
// cut into two or four by columns where there are CUs for that (SPLIT); a tile
// with few rows is one of half the rows.
template <class G, bool WGRAD, bool EXACT, bool SPLIT>
__device__ __forceinline__ void block8_job(const Block8Product& p, int n_wt, uint8_t* __restrict__ lds) {
  const int lane = lane_id();
  const ExpertRows ex(p.offsets, p.n_local, p.rows, lane);
  int units[4], total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    units[i] = WGRAD ? (4 * lane + i < p.n_local ? (p.M + G::TT - 1) / G::TT * n_wt : 0)
                     : (ex.count[i] + G::TT - 1) / G::TT * n_wt;
    total += units[i];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  total = __builtin_amdgcn_readfirstlane(total);
  const int q = total / 8, rest = total % 8, x = blockIdx.x % 8;
  // gradients: tiles of an expert, XCD x's tiles of the first k experts
  const int n = WGRAD ? (p.M + G::TT - 1) / G::TT * n_wt : 0, left = n % 8;
  auto upto = [&](int k) { return k * (n / 8) + (k * left + 7 - x) / 8; };
  const int c = WGRAD ? upto(p.n_local) : q + (x < rest);
  int at = blockIdx.x / 8, piece = 0, pieces = 1;
  if constexpr (SPLIT) {
    const int P = p.n_cus / 8, last = P > 0 ? c % P : 0;
    pieces = last == 0 ? 1 : 4 * last <= P ? 4 : 2 * last <= P ? 2 : 1;
    if (at >= c - last) {
      const int u = at - (c - last);
      piece = u % pieces;
      at = c - last + u / pieces;
    } else {
      pieces = 1;
    }
  }
  if (at >= c) return;
  int t = x * q + (x < rest ? x : rest) + at;
  if constexpr (WGRAD) {
    int k = 0;                                   // the first expert of four whose tiles reach past `at`
#pragma unroll
    for (int i = 0; i < 4; ++i) k += __popcll(__ballot(4 * lane + i < p.n_local && upto(4 * lane + i + 1) <= at));
    at -= upto(k);
    t = k * n + (at < n / 8 ? x * (n / 8) + at : n - left + ((x - k * left) & 7));
  }
  Job job;
  int before;
  job.slots = 0;
  if (!ex.find(units, t, lane, job.e, before, job.row0, job.count, WGRAD ? &job.slots : nullptr)) return;
  if (WGRAD && job.count > p.S - job.slots) {    // runs of rows that overlap: nothing past the operands' places
    job.count = job.slots < p.S ? static_cast<int32_t>(p.S - job.slots) : 0;
    job.slots = job.count ? job.slots : 0;
  }
  job.t_all = WGRAD ? p.M : job.count;
  const int t_tiles = (job.t_all + G::TT - 1) / G::TT;
  job.t0 = (t - before) % t_tiles * G::TT;
  job.i0 = (t - before) / t_tiles * G::TW;
  if constexpr (SPLIT) {
    static_assert(G::TT == 256 && G::TW == 256 && G::WAVES == 8, "the parts of this tile");
    job.i0 += piece * (G::TW / pieces);
    if (job.i0 >= p.N) return;
    if (pieces == 4) return block8_tile<Geo<256, 64, 8, 1, 2>, WGRAD, EXACT>(p, job, lds);
    if (pieces == 2) return block8_tile<Geo<256, 128, 4, 2, 2>, WGRAD, EXACT>(p, job, lds);
    if (job.t_all - job.t0 <= 128) return block8_tile<Geo<128, 256, 2, 4, 2>, WGRAD, EXACT>(p, job, lds);
  }
  block8_tile<G, WGRAD, EXACT>(p, job, lds);
}

template <class G, bool WGRAD, bool EXACT, bool SPLIT>
__global__ __launch_bounds__(G::THREADS) void k_block8(const Block8Product p, int n_wt) {
  __shared__ __attribute__((aligned(kRow))) uint8_t lds[G::LDS];   // chunks of a row are told apart by address bits
  block8_job<G, WGRAD, EXACT, SPLIT>(p, n_wt, lds);
}

template <class G, bool WGRAD, bool EXACT> hipError_t run(const Block8Product& p, hipStream_t s) {
  constexpr bool SPLIT = G::TT == 256 && G::TW == 256;
  const int64_t n_wt = (p.N + G::TW - 1) / G::TW;
  int64_t tt;
  if (WGRAD) {
    tt = static_cast<int64_t>(p.n_local) * ((p.M + G::TT - 1) / G::TT);
  } else {
    tt = (static_cast<int64_t>(p.rows) + G::TT - 1) / G::TT + p.n_local - 1;
    if (tt > p.rows) tt = p.rows;
  }
  if (tt == 0) return hipSuccess;
  // an XCD's pieces are at most as many as its CUs
  const int64_t grid = tt * n_wt + (SPLIT ? p.n_cus : 0);
  hipLaunchKernelGGL((k_block8<G, WGRAD, EXACT, SPLIT>), dim3(static_cast<unsigned>(grid)), dim3(G::THREADS), 0, s, p,
                     static_cast<int>(n_wt));
  return hipGetLastError();
}

// A 32 x 32 tile whose waves each take every eighth block of K, from registers:
// for products of few tiles, which wait in every step of a loop that all waves
// run together (for its barrier, the reads behind it, two matrix instructions
// and what they are added to: 0.55 us, however far ahead the loads go).  The
// waves' sums are added in their order.
constexpr int kThin = 32, kThinWaves = 8;
template <bool EXACT>
__device__ __forceinline__ void block8_thin(const Block8Product& p, uint8_t* __restrict__ lds) {
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = lane & 31, h = lane >> 5;
  const int n_wt = (p.N + kThin - 1) / kThin;
  const ExpertRows ex(p.offsets, p.n_local, p.rows, lane);
  int units[4], e, before;
#pragma unroll
  for (int i = 0; i < 4; ++i) units[i] = (ex.count[i] + kThin - 1) / kThin * n_wt;
  int32_t row0, count;
  if (!ex.find(units, blockIdx.x, lane, e, before, row0, count)) return;
  const int t_tiles = (count + kThin - 1) / kThin, at = blockIdx.x - before;
  const int t0 = at % t_tiles * kThin, i0 = at / t_tiles * kThin;
  const int t_rows = count - t0 < kThin ? count - t0 : kThin, w_rows = p.N - i0 < kThin ? p.N - i0 : kThin;
  const int steps = (p.K + kBlock - 1) / kBlock;
  auto rsrc = [&](const uint8_t* base, int rows) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, rows * p.K, 0x00020000);   // below 2^26
  };
  const __amdgpu_buffer_rsrc_t rt = rsrc(p.t + (static_cast<int64_t>(row0) + t0) * p.K, t_rows);
  const __amdgpu_buffer_rsrc_t rw = rsrc(p.w + (static_cast<int64_t>(e) * p.N + i0) * p.K, w_rows);
  const float* ts = p.t_scales + row0 + t0 + (r < t_rows ? r : t_rows - 1);
  const float* ws = p.w_scales + (static_cast<int64_t>(e) * ((p.N + kBlock - 1) / kBlock) + i0 / kBlock) * steps;
  const int row_at = r * p.K;
  struct Step { u32x4_t t[4], w[4]; float f; };
  // chunks h, 2 + h, 4 + h, 6 + h of the lane's rows; what a half block does not have reads as zero
  auto load = [&](int s, Step& x) {
    if (s >= steps) return;
    const bool cut = p.K % kBlock != 0 && s == steps - 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int off = cut && k >= 2 ? 0x7ffffff0 : row_at + (2 * k + h) * 16;
      x.t[k] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rt, off, s * kBlock, 0));
      x.w[k] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, off, s * kBlock, 0));
    }
    x.f = ts[static_cast<int64_t>(s) * p.rows] * ws[s];
  };
  f32x16_t acc;
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.0f;
  auto add = [&](const Step& x) {
    f32x16_t part;
#pragma unroll
    for (int k = 0; k < 16; ++k) part[k] = 0.0f;
    if constexpr (EXACT) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int g = 0; g < 2; ++g)
          part = __builtin_amdgcn_mfma_f32_32x32x16_f16(to_f16(x.w[k], g), to_f16(x.t[k], g), part, 0, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            __builtin_bit_cast(i32x8_t, __builtin_shufflevector(x.w[2 * k], x.w[2 * k + 1], 0, 1, 2, 3, 4, 5, 6, 7)),
            __builtin_bit_cast(i32x8_t, __builtin_shufflevector(x.t[2 * k], x.t[2 * k + 1], 0, 1, 2, 3, 4, 5, 6, 7)),
            part, 0, 0, 0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = __builtin_fmaf(part[k], x.f, acc[k]);
  };
  Step a, b;
  load(wave, a);
  for (int s = wave; s < steps; s += 2 * kThinWaves) {
    load(s + kThinWaves, b);
    add(a);
    if (s + kThinWaves >= steps) break;
    load(s + 2 * kThinWaves, a);
    add(b);
  }
  constexpr int PITCH = kThin + 4;
  float* own = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<float4*>(own + (wave * kThin + r) * PITCH + 8 * g + 4 * h) =
        make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
  __syncthreads();
  const int tr = tid / 16, c = tid % 16 * 2;
  float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kThinWaves; ++w) {
    const float2 x = *reinterpret_cast<const float2*>(own + (w * kThin + tr) * PITCH + c);
    v.x += x.x;
    v.y += x.y;
  }
  if (tr < t_rows && c < w_rows) {
    const int64_t o = (static_cast<int64_t>(row0) + t0 + tr) * p.N + i0 + c;
    if constexpr (EXACT) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) = v;
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o) = pack_bf16x2(v.x, v.y);
  }
}

template <bool EXACT>
__global__ __launch_bounds__(kThinWaves * kWave) void k_block8_thin(const Block8Product p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kThinWaves * kThin * (kThin + 4) * 4];
  block8_thin<EXACT>(p, lds);
}

hipError_t run_thin(const Block8Product& p, hipStream_t s) {
  int64_t tt = (static_cast<int64_t>(p.rows) + kThin - 1) / kThin + p.n_local - 1;
  if (tt > p.rows) tt = p.rows;
  if (tt == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(tt * ((p.N + kThin - 1) / kThin)));
  if (p.bf16) hipLaunchKernelGGL(k_block8_thin<false>, grid, dim3(kThinWaves * kWave), 0, s, p);
  else hipLaunchKernelGGL(k_block8_thin<true>, grid, dim3(kThinWaves * kWave), 0, s, p);
  return hipGetLastError();
}

using Big = Geo<256, 256, 2, 4, 2>;
using Mid = Geo<64, 128, 1, 4, 3>;       // two to a CU
using Mid16 = Geo<64, 128, 1, 4, 2>;     // fp16's products: three to a CU (85 us with two, 76 with three)
using Out = Geo<128, 128, 2, 2, 2>;      // gradients: two to a CU, stores under other tiles' loads

// Tiles of an even split of the rows.
template <class G> int64_t even_tiles(const Block8Product& p) {
  const int64_t each = (static_cast<int64_t>(p.rows) + p.n_local - 1) / p.n_local;
  return (each + G::TT - 1) / G::TT * p.n_local * ((p.N + G::TW - 1) / G::TW);
}

}  // namespace

// Measured, in us, 256 x 256 tiles against 64 x 128: 8192 rows of 8 experts,
// 7168 -> 4096 (512 large tiles) 277 / 430; 4096 of 8, 2048 -> 7168 (448) 72 /
// 108; 4096 of 32, 2048 -> 1408 (192) 26 / 29; 640 of 8, 7168 -> 4096 (128) 64 /
// 46; 2048 of 16, 2048 -> 1024 (64) 20 / 14.  fp16's products gain nothing from
// large tiles (151 / 153, 37 / 34).  32 x 32 against 64 x 128: 4 rows, 7168 ->
// 1408 (44 small tiles) 11 / 30; 512 rows, 7168 -> 512 (256) 17 / 31; 16 rows of
// 8 experts, 7168 -> 2048 (512) 22 / 32; 256 rows, 2048 -> 2048 (512) 12 / 12;
// 1024 rows, 4096 -> 1024 (1024) 33 / 20; fp32 results 11 / 42, 18 / 43, 23 / 44,
// 12 / 16, 34 / 28.
hipError_t launch_block8_gemm(const Block8Product& p, hipStream_t s) {
  if (p.bf16 && p.rows / p.n_local >= 128 && even_tiles<Big>(p) >= 160) return run<Big, false, false>(p, s);
  const int64_t each = (static_cast<int64_t>(p.rows) + p.n_local - 1) / p.n_local;
  if ((each + kThin - 1) / kThin * p.n_local * ((p.N + kThin - 1) / kThin) <= 2 * p.n_cus) return run_thin(p, s);
  return p.bf16 ? run<Mid, false, false>(p, s) : run<Mid16, false, true>(p, s);
}

// Measured, in us, 256 x 256 tiles against 128 x 128: 4096 slots of 32 experts,
// 1408 x 2048: 65 / 72; 4096 of one, 1024 x 1024: 23 / 30; with fp32 results
// the smaller tile is as good or better (104 / 93, 54 / 41).
hipError_t launch_block8_wgrad(const Block8Product& p, hipStream_t s) {
  if (!p.bf16) return run<Out, true, true>(p, s);
  if (p.rows / p.n_local < 128 || p.M < 256 || p.N < 256) return run<Out, true, false>(p, s);
  return run<Big, true, false>(p, s);
}

}  // namespace mok
