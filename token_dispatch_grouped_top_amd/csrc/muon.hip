// muon.hip -- orthogonalised updates of matrices by Newton-Schulz products,
// alone or as the step of an optimizer with momentum.
//
//   X = v / |v|_F;  G = X X^T,  B = b G + c G^2,  X = a X + B X  (`steps` times)
//
// on the smaller side m of the matrix (m <= n), so G and B are m x m and
// symmetric: of X X^T and G^2 only the tiles on and above the diagonal are
// computed, and stored twice.  Every product then has two operands whose rows
// lie along the contraction, given X and its transpose: G takes X, G^2 takes G,
// B X takes B and X^T.  The last one's epilogue adds a X and writes X and X^T.
//
// X, G and B are held in fp16: their values are at most about 1.3, 1.7 and 12
// in magnitude and get a factor 2^8 (exact), with which they keep 11 bits down
// to 2^-22; bf16, at the same rate, would keep 8, and the errors of five steps
// would show in an update of 8 bits.  Near the end G and B are close to multiples
// of the identity, whose rounding all rows would share and every step would
// carry on (4e-3 of the result where all singular values are equal); what the
// rounding takes from their diagonals is therefore kept beside them in fp32 and
// enters by the epilogues:  with G = H + D (H rounded, D diagonal),
//   G^2 = H H + D H + H D (+ D^2, below 2^-22),   B X = fp16(B) X + rest of B's diagonal * X.
// Sums are fp32, the norm fp64.
#include "muon.h"
#include "nt_tile.h"

namespace mok {
namespace {

using namespace nt;

constexpr float kIn = 256.0f, kBack = 1.0f / 256.0f;   // factor of what is held in fp16
constexpr int kChunks = 512;                            // partial sums of a matrix's norm

struct Shape {
  int32_t rows, cols, m, n, mp, np, tall, chunks;       // m <= n; mp, np: to whole K-steps
  int64_t size;
};
Shape shape_of(int32_t rows, int32_t cols) {
  Shape s{};
  s.rows = rows; s.cols = cols; s.tall = rows > cols;
  s.m = s.tall ? cols : rows; s.n = s.tall ? rows : cols;
  s.mp = (s.m + 63) / 64 * 64; s.np = (s.n + 63) / 64 * 64;
  s.size = static_cast<int64_t>(rows) * cols;
  const int64_t c = (s.size + 4095) / 4096;
  s.chunks = static_cast<int32_t>(c < kChunks ? c : kChunks);
  return s;
}

struct Work {
  double* norms;                // [n][chunks] sums of squares
  _Float16 *x, *xt[2], *g, *b;  // [n][mp][np], [n][np][mp], [n][mp][mp]
  float *g_rest, *b_rest;       // [n][mp]: what rounding took from the diagonals of g and b
};
size_t carve(const Shape& s, int32_t n, void* ws, Work* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(ws) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t mats = static_cast<size_t>(n), xn = mats * s.mp * s.np * 2, gn = mats * s.mp * s.mp * 2;
  Work k{};
  k.norms = reinterpret_cast<double*>(take(mats * s.chunks * 8));
  k.x = reinterpret_cast<_Float16*>(take(xn));
  k.xt[0] = reinterpret_cast<_Float16*>(take(xn));
  k.xt[1] = reinterpret_cast<_Float16*>(take(xn));
  k.g = reinterpret_cast<_Float16*>(take(gn));
  k.b = reinterpret_cast<_Float16*>(take(gn));
  k.g_rest = reinterpret_cast<float*>(take(mats * s.mp * 4));
  k.b_rest = reinterpret_cast<float*>(take(mats * s.mp * 4));
  if (w) *w = k;
  return at;
}

// ------------------------------------------------------------- momentum, norm
struct Input {
  const void* x; int32_t bf16;
  float* m;                     // null: v = x
  float momentum, grad_scale;
  int32_t nesterov;
  const mok_adamw_scalars* scalars;
};
__device__ __forceinline__ float value(const Input& in, int64_t i) {
  return in.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(in.x)[i]) << 16)
                 : static_cast<const float*>(in.x)[i];
}
__device__ __forceinline__ float factor(const Input& in) {
  return in.scalars ? in.scalars->grad_scale : in.grad_scale;
}
__device__ __forceinline__ bool skipped(const mok_adamw_scalars* s) { return s && s->skip != 0; }

// m = momentum m + g, and the sum of the squares of v over a chunk of a matrix.
__global__ __launch_bounds__(256) void k_muon_norm(const Input in, const Shape s, double* norms) {
  if (skipped(in.scalars)) return;
  __shared__ double part[4];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * s.size;
  const int64_t each = (s.size + s.chunks - 1) / s.chunks;
  const int64_t i0 = blockIdx.x * each, i1 = i0 + each < s.size ? i0 + each : s.size;
  const float f = factor(in);
  double sum = 0.0;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
    float v = value(in, base + i);
    if (in.m) {
      const float g = v * f;
      const float m = __builtin_fmaf(in.momentum, in.m[base + i], g);
      in.m[base + i] = m;
      v = in.nesterov ? __builtin_fmaf(in.momentum, m, g) : m;
    }
    sum += static_cast<double>(v) * v;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) part[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    norms[static_cast<int64_t>(blockIdx.y) * s.chunks + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and X^T, scaled, in fp16, zero in the padding: 64 x 64 values of v a
// workgroup, through LDS for the transposed one.
__global__ __launch_bounds__(256) void k_muon_convert(const Input in, const Shape s, const double* norms,
                                                      _Float16* x, _Float16* xt) {
  if (skipped(in.scalars)) return;
  __shared__ _Float16 tile[64][66];
  __shared__ double part[4];
  const int tid = threadIdx.x;
  const int rp = s.tall ? s.np : s.mp, cp = s.tall ? s.mp : s.np;    // padded rows, columns of v
  const int c0 = blockIdx.x % (cp / 64) * 64, r0 = blockIdx.x / (cp / 64) * 64;
  double sum = 0.0;
  for (int i = tid; i < s.chunks; i += 256) sum += norms[static_cast<int64_t>(blockIdx.y) * s.chunks + i];
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) part[tid / kWave] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  const double scale = sum > 0.0 || sum != sum ? kIn / sqrt(sum) : 0.0;
  const float f = factor(in);
  const int64_t base = static_cast<int64_t>(blockIdx.y) * s.size;
  _Float16* straight = (s.tall ? xt : x) + static_cast<int64_t>(blockIdx.y) * rp * cp;
  _Float16* turned = (s.tall ? x : xt) + static_cast<int64_t>(blockIdx.y) * rp * cp;
  for (int k = 0; k < 16; ++k) {
    const int r = 4 * k + tid / 64, c = tid % 64;
    float v = 0.0f;
    if (r0 + r < s.rows && c0 + c < s.cols) {
      const int64_t i = base + static_cast<int64_t>(r0 + r) * s.cols + c0 + c;
      if (in.m) {
        v = in.m[i];
        if (in.nesterov) v = __builtin_fmaf(in.momentum, v, value(in, i) * f);
      } else {
        v = value(in, i);
      }
      v = static_cast<float>(v * scale);
    }
    tile[r][c] = static_cast<_Float16>(v);
    straight[static_cast<int64_t>(r0 + r) * cp + c0 + c] = tile[r][c];
  }
  __syncthreads();
  for (int k = 0; k < 16; ++k) {
    const int c = 4 * k + tid / 64, r = tid % 64;
    turned[static_cast<int64_t>(c0 + c) * rp + r0 + r] = tile[r][c];
  }
}

// ------------------------------------------------------------------- products
enum Epi { GRAM = 0, POLY = 1, UPDATE = 2, LAST_OUT = 3, LAST_STEP = 4 };

struct Product {
  const _Float16 *t, *w;        // operands [rows][K] of each matrix
  int32_t t_rows, w_rows, K;
  int64_t t_mat, w_mat;         // values of a matrix's operand
  const _Float16* add;          // [t_rows][w_rows]: G (POLY), X (UPDATE, LAST)
  _Float16* out;                // [t_rows][w_rows]
  _Float16* out_t;              // [w_rows][t_rows]
  float c_add, c_acc;           // out = c_add * add + c_acc * sum
  const float* rest_in;         // POLY: G's; UPDATE, LAST: B's
  float* rest_out;              // GRAM: G's; POLY: B's
  int32_t rest_cols;            // UPDATE, LAST: B's rows are the output's columns
  int32_t mats;
  // LAST: the true size of out and what is done with it
  int32_t rows, cols;
  uint16_t* o;
  float* p; uint16_t* p_bf16;
  double lr, weight_decay, scale;
  const mok_adamw_scalars* scalars;
};

template <class G, int EPI>
__device__ __forceinline__ void muon_tile(const Product& p, uint8_t* __restrict__ lds) {
  constexpr bool SYM = EPI == GRAM || EPI == POLY;
  if (skipped(p.scalars)) return;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // ---- which tile: each XCD a contiguous eighth of them
  const int nt = (p.t_rows + G::TT - 1) / G::TT, nw = (p.w_rows + G::TW - 1) / G::TW;
  const int per = SYM ? nt * (nt + 1) / 2 : nt * nw, total = per * p.mats;
  const int q = total / 8, rest = total % 8, x = blockIdx.x % 8;
  const int t = x * q + (x < rest ? x : rest) + blockIdx.x / 8;
  if (static_cast<int>(blockIdx.x / 8) >= q + (x < rest)) return;
  const int mat = t / per;
  int tt = t % per, tw;
  if (SYM) {                                    // row tt of the triangle has its tiles tw >= tt
    int row = 0;
    while (tt >= nt - row) { tt -= nt - row; ++row; }
    tw = row + tt;
    tt = row;
  } else {
    tw = tt / nt;
    tt = tt % nt;
  }
  const int t0 = tt * G::TT, w0 = tw * G::TW;
  const int t_rows = p.t_rows - t0 < G::TT ? p.t_rows - t0 : G::TT;
  const int w_rows = p.w_rows - w0 < G::TW ? p.w_rows - w0 : G::TW;
  const int64_t stride = static_cast<int64_t>(p.K) * 2;
  Operand ot, ow;
  ot.base = reinterpret_cast<const uint8_t*>(p.t + mat * p.t_mat) + t0 * stride;
  ow.base = reinterpret_cast<const uint8_t*>(p.w + mat * p.w_mat) + w0 * stride;
  ot.stride = ow.stride = stride;
  ot.extent = t_rows * stride;
  ow.extent = w_rows * stride;
  const Loader<G::LT> lt(ot, t_rows, wave, G::WAVES, lane);
  const Loader<G::LW> lw(ow, w_rows, wave, G::WAVES, lane);
  const int steps = p.K / 64;
  auto stage_t = [&](int b) { return lds + b * G::STAGE; };
  auto stage_w = [&](int b) { return lds + b * G::STAGE + G::TT * kRow; };
  auto issue = [&](int step, int b) {
    step = step < steps ? step : steps - 1;
    const uint32_t off = static_cast<uint32_t>(step) * kRow;
#pragma unroll
    for (int j = 0; j < G::LT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lt.rsrc, (lds_ptr_t)(stage_t(b) + (j * G::WAVES + wave) * 1024),
                                               16, lt.at[j], off, 0, 0);
#pragma unroll
    for (int j = 0; j < G::LW; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lw.rsrc, (lds_ptr_t)(stage_w(b) + (j * G::WAVES + wave) * 1024),
                                               16, lw.at[j], off, 0, 0);
  };
  const int wt = wave % G::WT * (G::TT / G::WT), ww = wave / G::WT * (G::TW / G::WW);
  f32x16_t acc[G::FW][G::FT];
#pragma unroll
  for (int i = 0; i < G::FW; ++i)
#pragma unroll
    for (int j = 0; j < G::FT; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
#pragma unroll
  for (int s = 0; s < G::NS - 1; ++s) issue(s, s);
  int buf = 0;
  for (int s = 0; s < steps; ++s) {
    wait_vm_barrier<(G::NS - 2) * G::LPS>();
    issue(s + G::NS - 1, buf == 0 ? G::NS - 1 : buf - 1);
    const uint8_t* T = stage_t(buf) + wt * kRow;
    const uint8_t* W = stage_w(buf) + ww * kRow;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int r = lane & 31, at = r * kRow + chunk_at(r, 2 * kk + (lane >> 5)) * 16;
      f16x8_t wf[G::FW], tf[G::FT];
#pragma unroll
      for (int i = 0; i < G::FW; ++i) wf[i] = __builtin_bit_cast(f16x8_t, chunk16(W + 32 * i * kRow + at));
#pragma unroll
      for (int j = 0; j < G::FT; ++j) tf[j] = __builtin_bit_cast(f16x8_t, chunk16(T + 32 * j * kRow + at));
#pragma unroll
      for (int j = 0; j < G::FT; ++j)
#pragma unroll
        for (int i = 0; i < G::FW; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wf[i], tf[j], acc[i][j], 0, 0, 0);
    }
    buf = buf + 1 == G::NS ? 0 : buf + 1;
  }
  wait_vm_barrier<0>();

  // ---- results: 32 rows at a time through the wave's own part of LDS
  constexpr int CW = 32 * G::FW, PITCH = CW + 4, LPR = CW / 4;
  float* own = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  const int64_t o_mat = static_cast<int64_t>(mat) * p.t_rows * p.w_rows;
  float keep = 1.0f, step = 0.0f;               // LAST_STEP
  if (EPI == LAST_STEP) {
    const double lr = p.scalars ? static_cast<double>(p.scalars->lr) : p.lr;
    keep = static_cast<float>(1.0 - lr * p.weight_decay);
    step = static_cast<float>(-lr * p.scale * kBack);
  }
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
      float* f = reinterpret_cast<float*>(&v);
      const int row = t0 + wt + 32 * j + r, col = w0 + ww + c;
      const bool in = row < p.t_rows && col < p.w_rows;
      const int64_t o = o_mat + static_cast<int64_t>(row) * p.w_rows + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] *= p.c_acc;
      if (EPI != GRAM && in) {
        const uint2 w = *reinterpret_cast<const uint2*>(p.add + o);
        const uint32_t h[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
        const float* rest = p.rest_in + static_cast<int64_t>(mat) * (EPI == POLY || !p.rest_cols ? p.t_rows : p.w_rows);
        const float4 rc = EPI == POLY || p.rest_cols ? *reinterpret_cast<const float4*>(rest + col)
                                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float rr = EPI == POLY || !p.rest_cols ? rest[row] : 0.0f;
        const float rest4[4] = {rc.x + rr, rc.y + rr, rc.z + rr, rc.w + rr};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h[i])));
          if (EPI == POLY) {          // b (G + D) + c (H H + D H + H D)
            f[i] = __builtin_fmaf(p.c_add, a + (row == col + i ? rr : 0.0f), __builtin_fmaf(p.c_acc * rest4[i], a, f[i]));
          } else {                    // (a + rest) X + B X
            f[i] = __builtin_fmaf(__builtin_fmaf(rest4[i], kBack, p.c_add), a, f[i]);
          }
        }
      }
      if (EPI <= UPDATE) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f[i]));
        if (in) *reinterpret_cast<uint2*>(p.out + o) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        if (SYM && in && static_cast<uint32_t>(row - col) < 4u) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row == col + i)
              p.rest_out[static_cast<int64_t>(mat) * p.t_rows + row] =
                  f[i] - static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h[i])));
        }
        *reinterpret_cast<float4*>(own + r * PITCH + c) = v;
      } else {
        const int64_t to = static_cast<int64_t>(mat) * p.rows * p.cols + static_cast<int64_t>(row) * p.cols + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (row >= p.rows || col + i >= p.cols) continue;
          if (EPI == LAST_OUT) {
            p.o[to + i] = f32_to_bf16(f[i] * kBack);
          } else {
            const float n = __builtin_fmaf(step, f[i], p.p[to + i] * keep);
            p.p[to + i] = n;
            if (p.p_bf16) p.p_bf16[to + i] = f32_to_bf16(n);
          }
        }
      }
    }
    if (EPI <= UPDATE && !(SYM && tt == tw)) {
#pragma unroll
      for (int k = 0; k < CW * 8 / 64; ++k) {
        const int c = (k * 64 + lane) / 8, r = (k * 64 + lane) % 8 * 4;
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(own[(r + i) * PITCH + c]));
        const int row = t0 + wt + 32 * j + r, col = w0 + ww + c;
        if (row < p.t_rows && col < p.w_rows)
          *reinterpret_cast<uint2*>(p.out_t + o_mat + static_cast<int64_t>(col) * p.t_rows + row) =
              make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      }
    }
  }
}

template <class G, int EPI>
__global__ __launch_bounds__(G::THREADS) void k_muon_product(const Product p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::LDS];
  muon_tile<G, EPI>(p, lds);
}

using Big = Geo<256, 256, 2, 4, 2, false>;
using Small = Geo<64, 64, 2, 2, 4, false>;

template <class G, int EPI> hipError_t run(const Product& p, hipStream_t s) {
  const int64_t nt = (p.t_rows + G::TT - 1) / G::TT, nw = (p.w_rows + G::TW - 1) / G::TW;
  const int64_t tiles = (EPI <= POLY ? nt * (nt + 1) / 2 : nt * nw) * p.mats;
  hipLaunchKernelGGL((k_muon_product<G, EPI>), dim3(static_cast<unsigned>(tiles)), dim3(G::THREADS), 0, s, p);
  return hipGetLastError();
}
template <int EPI> hipError_t run(const Product& p, hipStream_t s) {
  const int64_t nt = (p.t_rows + 255) / 256, nw = (p.w_rows + 255) / 256;
  return (EPI <= POLY ? nt * (nt + 1) / 2 : nt * nw) * p.mats >= 128 ? run<Big, EPI>(p, s) : run<Small, EPI>(p, s);
}

}  // namespace

size_t muon_ws_bytes(int32_t n, int32_t rows, int32_t cols) {
  return carve(shape_of(rows, cols), n, nullptr, nullptr);
}

hipError_t launch_muon(const MuonArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const Shape sh = shape_of(a.rows, a.cols);
  Work w;
  carve(sh, a.n, a.ws, &w);
  Input in{};
  in.x = a.x; in.bf16 = a.x_bf16; in.m = a.p ? a.m : nullptr;
  in.momentum = static_cast<float>(a.momentum); in.grad_scale = static_cast<float>(a.grad_scale);
  in.nesterov = a.nesterov; in.scalars = a.scalars;
  const unsigned n = static_cast<unsigned>(a.n);
  hipLaunchKernelGGL(k_muon_norm, dim3(sh.chunks, n), dim3(256), 0, s, in, sh, w.norms);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_muon_convert, dim3(sh.mp / 64 * (sh.np / 64), n), dim3(256), 0, s, in, sh, w.norms, w.x,
                     w.xt[0]);
  e = hipGetLastError();
  for (int i = 0; i < a.ns.steps && e == hipSuccess; ++i) {
    const int64_t xm = static_cast<int64_t>(sh.mp) * sh.np, gm = static_cast<int64_t>(sh.mp) * sh.mp;
    Product g{};
    g.mats = a.n; g.scalars = a.scalars;
    g.t = g.w = w.x; g.t_rows = g.w_rows = sh.mp; g.K = sh.np; g.t_mat = g.w_mat = xm;
    g.out = g.out_t = w.g; g.c_acc = kBack; g.rest_out = w.g_rest;
    e = run<GRAM>(g, s);
    if (e != hipSuccess) break;
    Product b = g;
    b.t = b.w = w.g; b.K = sh.mp; b.t_mat = b.w_mat = gm;
    b.add = w.g; b.out = b.out_t = w.b; b.c_add = a.ns.b; b.c_acc = a.ns.c * kBack;
    b.rest_in = w.g_rest; b.rest_out = w.b_rest;
    e = run<POLY>(b, s);
    if (e != hipSuccess) break;
    // rows of the output: v's rows, so that the last one is v's layout
    const _Float16* xt = w.xt[i & 1];
    Product u{};
    u.mats = a.n; u.scalars = a.scalars; u.K = sh.mp; u.c_add = a.ns.a; u.c_acc = kBack;
    u.rest_in = w.b_rest; u.rest_cols = sh.tall;
    if (sh.tall) {
      u.t = xt; u.t_rows = sh.np; u.t_mat = xm; u.w = w.b; u.w_rows = sh.mp; u.w_mat = gm;
      u.add = xt; u.out = w.xt[1 - (i & 1)]; u.out_t = w.x;
    } else {
      u.t = w.b; u.t_rows = sh.mp; u.t_mat = gm; u.w = xt; u.w_rows = sh.np; u.w_mat = xm;
      u.add = u.out = w.x; u.out_t = w.xt[1 - (i & 1)];
    }
    if (i + 1 < a.ns.steps) {
      e = run<UPDATE>(u, s);
    } else {
      u.rows = a.rows; u.cols = a.cols; u.o = static_cast<uint16_t*>(a.out);
      u.p = a.p; u.p_bf16 = static_cast<uint16_t*>(a.p_bf16);
      u.lr = a.lr; u.weight_decay = a.weight_decay; u.scale = a.scale;
      e = a.p ? run<LAST_STEP>(u, s) : run<LAST_OUT>(u, s);
    }
  }
  return e;
}

}  // namespace mok
