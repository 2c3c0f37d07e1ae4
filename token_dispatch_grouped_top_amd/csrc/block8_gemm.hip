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
// lane and 64 cycles of fma stand against 128 cycles of matrix instructions,
// which another wave of the same SIMD fills.
//
// gfx950's 8-bit matrix instructions add up a group of products aligned to the
// largest of them and drop what lies below 2^-13 of it (whole products below
// 2^-13 vanish; at random codes a sum is off by 1e-5 to 5e-5 of its size).
// That is far below a result in bf16, but not what a result in fp32 is asked
// for: such a one (EXACT) is formed by v_mfma_f32_32x32x16_f16 from the codes
// converted to fp16, which holds them all, at half the rate, with sums as exact
// as fp32's.
//
// The gradient of the weights is the same product over slot blocks: dy_t takes
// the tokens' place (a scale for 128 slots of a column), x_t the weights'.
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

template <class G, bool WGRAD, bool EXACT>
__device__ __forceinline__ void block8_tile(const Block8Product& p, int n_wt, uint8_t* __restrict__ lds) {
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);

  // ---- which tile: expert by expert, columns outside, rows inside, each XCD
  // a contiguous eighth of them (workgroup ids go round the XCDs)
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
  const int q = total / 8, rest = total % 8, x = blockIdx.x % 8, at = blockIdx.x / 8;
  if (at >= q + (x < rest)) return;
  const int t = x * q + (x < rest ? x : rest) + at;
  int e, before;
  int32_t row0, count;
  int64_t slots = 0;
  if (!ex.find(units, t, lane, e, before, row0, count, WGRAD ? &slots : nullptr)) return;
  const int t_all = WGRAD ? p.M : count, t_tiles = (t_all + G::TT - 1) / G::TT;
  const int t0 = (t - before) % t_tiles * G::TT, i0 = (t - before) / t_tiles * G::TW;

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
  const Loader<G::LT> lt(ot, t_rows, wave, G::WAVES, lane);
  const Loader<G::LW> lw(ow, w_rows, wave, G::WAVES, lane);
  // a thread's scale: of row tid of the tokens, or of one of the tile's blocks of weight rows
  const float* my_scale;
  int64_t my_step;
  if (tid < G::TT) {
    my_scale = ts + (tid < t_rows ? tid : t_rows - 1);
    my_step = ts_step;
  } else {
    int b = tid - G::TT;
    const int blocks = (w_rows + kBlock - 1) / kBlock;
    my_scale = ws + (b < blocks ? b : blocks - 1) * ws_row;
    my_step = 1;
  }
  auto stage_t = [&](int b) { return lds + b * G::STAGE; };
  auto stage_w = [&](int b) { return lds + b * G::STAGE + G::TT * kRow; };
  auto stage_s = [&](int b) { return lds + b * G::STAGE + (G::TT + G::TW) * kRow; };
  auto issue = [&](int step, int b) {
    step = step < steps ? step : steps - 1;                // past the end: loads that nobody reads
    const bool cut = half && step == steps - 1;
    const uint32_t off = static_cast<uint32_t>(step) * kRow;
#pragma unroll
    for (int j = 0; j < G::LT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lt.rsrc, (lds_ptr_t)(stage_t(b) + (j * G::WAVES + wave) * 1024),
                                               16, cut ? lt.tail[j] : lt.at[j], off, 0, 0);
#pragma unroll
    for (int j = 0; j < G::LW; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lw.rsrc, (lds_ptr_t)(stage_w(b) + (j * G::WAVES + wave) * 1024),
                                               16, cut ? lw.tail[j] : lw.at[j], off, 0, 0);
    __builtin_amdgcn_global_load_lds((glb_ptr_t)(my_scale + step * my_step),
                                     (lds_ptr_t)(stage_s(b) + wave * 256), 4, 0, 0);
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
  if (steps > 0) {
#pragma unroll
    for (int s = 0; s < G::NS - 1; ++s) issue(s, s);
  }
  int buf = 0;
  for (int s = 0; s < steps; ++s) {
    wait_vm_barrier<(G::NS - 2) * G::LPS>();
    issue(s + G::NS - 1, buf == 0 ? G::NS - 1 : buf - 1);
    const float* sc = reinterpret_cast<const float*>(stage_s(buf));
    block8_step<G, EXACT>(acc, stage_t(buf) + wt * kRow, stage_w(buf) + ww * kRow, sc + wt,
                          sc[G::TT + ww / kBlock], lane);
    buf = buf + 1 == G::NS ? 0 : buf + 1;
  }
  wait_vm_barrier<0>();

  // ---- results: 32 rows at a time through the wave's own part of LDS, so that
  // a row's columns are stored behind each other
  constexpr int CW = 32 * G::FW, PITCH = CW + 4, LPR = CW / 4;   // lanes of a row
  float* own = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  const int64_t out0 = WGRAD ? static_cast<int64_t>(e) * p.M + t0 : static_cast<int64_t>(row0) + t0;
#pragma unroll
  for (int j = 0; j < G::FT; ++j) {
#pragma unroll
    for (int i = 0; i < G::FW; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(own + (lane & 31) * PITCH + 32 * i + 8 * g + 4 * (lane >> 5)) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
#pragma unroll
    for (int k = 0; k < 32 * LPR / 64; ++k) {
      const int r = (k * 64 + lane) / LPR, c = (k * 64 + lane) % LPR * 4;
      float4 v = *reinterpret_cast<const float4*>(own + r * PITCH + c);
      const int tr = wt + 32 * j + r, col = i0 + ww + c;
      if (tr < t_rows && col < p.N) {
        const int64_t o = (out0 + tr) * p.N + col;
        if constexpr (!EXACT) {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        } else {
          float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
          if (p.accumulate) {
            const float4 w = *to;
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
          }
          *to = v;
        }
      }
    }
  }
}

template <class G, bool WGRAD, bool EXACT>
__global__ __launch_bounds__(G::THREADS) void k_block8(const Block8Product p, int n_wt) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::LDS];
  block8_tile<G, WGRAD, EXACT>(p, n_wt, lds);
}

template <class G, bool WGRAD> hipError_t run(const Block8Product& p, hipStream_t s) {
  const int64_t n_wt = (p.N + G::TW - 1) / G::TW;
  int64_t tt;
  if (WGRAD) {
    tt = static_cast<int64_t>(p.n_local) * ((p.M + G::TT - 1) / G::TT);
  } else {
    tt = (static_cast<int64_t>(p.rows) + G::TT - 1) / G::TT + p.n_local - 1;
    if (tt > p.rows) tt = p.rows;
  }
  if (tt * n_wt == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(tt * n_wt));
  if (p.bf16) hipLaunchKernelGGL((k_block8<G, WGRAD, false>), grid, dim3(G::THREADS), 0, s, p, static_cast<int>(n_wt));
  else hipLaunchKernelGGL((k_block8<G, WGRAD, true>), grid, dim3(G::THREADS), 0, s, p, static_cast<int>(n_wt));
  return hipGetLastError();
}

using Big = Geo<256, 256, 2, 4, 2, true>;
using Mid = Geo<64, 128, 1, 4, 3, true>;

}  // namespace

hipError_t launch_block8_gemm(const Block8Product& p, hipStream_t s) {
  return p.rows / p.n_local >= 128 ? run<Big, false>(p, s) : run<Mid, false>(p, s);
}

hipError_t launch_block8_wgrad(const Block8Product& p, hipStream_t s) {
  return p.M >= 256 && p.N >= 256 ? run<Big, true>(p, s) : run<Mid, true>(p, s);
}

}  // namespace mok
