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

// Operands of the products are column-blocked: value (r, k) of R rows at
// ((k / 32) * R + r) * 32 + k % 32, so a K-step of 32 of a tile's rows is
// contiguous memory, read in whole lines, and so is a 32 x 32 block that is
// written, either way round.
__device__ __forceinline__ int64_t blocked(int64_t r, int64_t k, int64_t R) {
  return ((k >> 5) * R + r) * 32 + (k & 31);
}

// Few tiles with a long K leave most CUs idle: K is cut into pieces of at least
// four steps, as many as fill the chip once.
constexpr int kPieces = 16, kSmallTile = 64, kCut = 128;
int gram_pieces(int64_t tiles, int32_t K) {
  int64_t n = tiles > 0 ? 256 / tiles : 1;
  n = n < K / 256 ? n : K / 256;
  n = n < kPieces ? n : kPieces;
  return n < 2 ? 1 : static_cast<int>(n);
}
int64_t gram_tiles(const Shape& s, int32_t n) {
  const int64_t t = (s.mp + kSmallTile - 1) / kSmallTile;
  return t * (t + 1) / 2 * n;
}

struct Work {
  double* norms;                // [n][chunks] sums of squares
  _Float16 *x, *xt[2], *g, *b;  // [n][mp][np], [n][np][mp], [n][mp][mp]
  float *g_rest, *b_rest;       // [n][mp]: what rounding took from the diagonals of g and b
  float* parts;                 // fp32 sums of the pieces of X X^T
  int32_t* arrived;             // [kCut]: pieces that are there (of two at least each, of 256 together)
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
  const int64_t tiles = gram_tiles(s, n);
  const int pieces = gram_pieces(tiles, s.np);
  k.parts = reinterpret_cast<float*>(take(pieces > 1 ? tiles * pieces * kSmallTile * kSmallTile * 4 : 0));
  k.arrived = reinterpret_cast<int32_t*>(take(kCut * 4));
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

// Four values of x: VEC: from i on, aligned for them, all there; else those of i + k * step that lie before `end`.
template <bool VEC>
__device__ __forceinline__ void value4(const Input& in, int64_t i, int step, int64_t end, float (&v)[4]) {
  if constexpr (VEC) {
    if (in.bf16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(in.x) + i);
      v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(in.x) + i);
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k * step < end ? value(in, i + k * step) : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void moment4(const float* m, int64_t i, int step, int64_t end, float (&v)[4]) {
  if constexpr (VEC) {
    const float4 w = *reinterpret_cast<const float4*>(m + i);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k * step < end ? m[i + k * step] : 0.0f;
  }
}

// m = momentum m + g, and the sum of the squares of v over a chunk of a matrix
// (fp64: squares of fp32 values do not overflow in it).
template <bool VEC>
__global__ __launch_bounds__(256) void k_muon_norm(const Input in, const Shape s, double* norms, int32_t* arrived) {
  if (skipped(in.scalars)) return;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kCut) arrived[threadIdx.x] = 0;
  __shared__ double part[4];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * s.size;
  const int64_t each = (s.size + s.chunks * 1024ll - 1) / (s.chunks * 1024ll) * 1024;
  const int64_t i0 = blockIdx.x * each, i1 = i0 + each < s.size ? i0 + each : s.size;
  const float f = factor(in);
  double sum = 0.0;
  for (int64_t i = i0 + (VEC ? 4 : 1) * threadIdx.x; i < i1; i += 1024) {
    float v[4];
    value4<VEC>(in, base + i, 256, base + i1, v);
    if (in.m) {
      float m[4];
      moment4<VEC>(in.m, base + i, 256, base + i1, m);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float g = v[k] * f;
        m[k] = __builtin_fmaf(in.momentum, m[k], g);
        v[k] = in.nesterov ? __builtin_fmaf(in.momentum, m[k], g) : m[k];
      }
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(in.m + base + i) = make_float4(m[0], m[1], m[2], m[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + 256 * k < i1) in.m[base + i + 256 * k] = m[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += static_cast<double>(v[k]) * v[k];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) part[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    norms[static_cast<int64_t>(blockIdx.y) * s.chunks + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and X^T, scaled, in fp16, zero in the padding: 64 x 64 values of v a
// workgroup, through LDS for the transposed one.  VEC: rows of v begin at
// multiples of four values.
template <bool VEC>
__global__ __launch_bounds__(256) void k_muon_convert(const Input in, const Shape s, const double* norms,
                                                      _Float16* x, _Float16* xt) {
  if (skipped(in.scalars)) return;
  constexpr int PITCH = 68;                     // 8-byte writes of rows, 2-byte reads of columns
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][PITCH];
  __shared__ double part[4];
  const int tid = threadIdx.x;
  const int rp = s.tall ? s.np : s.mp, cp = s.tall ? s.mp : s.np;    // padded rows, columns of v
  const int c0 = blockIdx.x % (cp / 64) * 64, r0 = blockIdx.x / (cp / 64) * 64;
  const float f = factor(in);
  const int64_t base = static_cast<int64_t>(blockIdx.y) * s.size;
  float v[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = r0 + 16 * k + tid / 16, c = c0 + tid % 16 * (VEC ? 4 : 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[k][i] = 0.0f;
    if (r < s.rows && c < s.cols) {
      const int64_t row = base + static_cast<int64_t>(r) * s.cols, i = row + c, end = row + s.cols;
      if (!in.m) {
        value4<VEC>(in, i, 16, end, v[k]);
      } else {
        moment4<VEC>(in.m, i, 16, end, v[k]);
        if (in.nesterov) {
          float g[4];
          value4<VEC>(in, i, 16, end, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[k][j] = __builtin_fmaf(in.momentum, v[k][j], g[j] * f);
        }
      }
    }
  }
  double sum = 0.0;
  for (int i = tid; i < s.chunks; i += 256) sum += norms[static_cast<int64_t>(blockIdx.y) * s.chunks + i];
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) part[tid / kWave] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  const double scale = sum > 0.0 || sum != sum ? kIn / sqrt(sum) : 0.0;
  _Float16* straight = (s.tall ? xt : x) + static_cast<int64_t>(blockIdx.y) * rp * cp;
  _Float16* turned = (s.tall ? x : xt) + static_cast<int64_t>(blockIdx.y) * rp * cp;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 16 * k + tid / 16;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(static_cast<float>(v[k][i] * scale)));
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(&tile[r][tid % 16 * 4]) =
          make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) tile[r][tid % 16 + 16 * i] = h[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int a = k * 32 + tid / 8, b = tid % 8 * 8;     // 8 columns of row a, 8 rows of column a
    const uint2 lo = *reinterpret_cast<const uint2*>(&tile[a][b]), hi = *reinterpret_cast<const uint2*>(&tile[a][b + 4]);
    *reinterpret_cast<uint4*>(straight + blocked(r0 + a, c0 + b, rp)) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = tile[b + 2 * i][a] | static_cast<uint32_t>(tile[b + 2 * i + 1][a]) << 16;
    *reinterpret_cast<uint4*>(turned + blocked(c0 + a, r0 + b, cp)) = make_uint4(w[0], w[1], w[2], w[3]);
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
  // GRAM: pieces of K, each a workgroup's; their fp32 sums and a counter for each tile (zero)
  int32_t pieces;
  float* parts; int32_t* arrived;
  // LAST: the true size of out and what is done with it
  int32_t rows, cols;
  uint16_t* o;
  float* p; uint16_t* p_bf16;
  int32_t vec;                  // their rows begin at multiples of four values
  double lr, weight_decay, scale;
  const mok_adamw_scalars* scalars;
};

// TT x TW tile of WT x WW waves, K-steps of KS (KS / 32 blocks of 64 bytes of a
// row, each four chunks of 16) in NS stages; PER_CU workgroups share a CU.
template <int TT_, int TW_, int WT_, int WW_, int KS_, int NS_, int PER_CU_> struct Geo16 {
  static constexpr int TT = TT_, TW = TW_, WT = WT_, WW = WW_, KS = KS_, NS = NS_, PER_CU = PER_CU_;
  static constexpr int WAVES = WT * WW, THREADS = 64 * WAVES, ROW = 64, KB = KS / 32;
  static constexpr int FT = TT / WT / 32, FW = TW / WW / 32;
  static constexpr int LT = KB * TT * ROW / 1024 / WAVES, LW = KB * TW * ROW / 1024 / WAVES, LPS = LT + LW;
  static constexpr int STAGE = KB * (TT + TW) * ROW, PITCH = 40;   // of 32 fp16 values on their way through LDS
  static constexpr int WIDE = 36, OWN = 32 * WIDE * 4;              // of 32 fp32 values; bytes of a wave
  static constexpr int LDS = NS * STAGE > WAVES * OWN ? NS * STAGE : WAVES * OWN;
  static_assert(LT >= 1 && LW >= 1 && LT <= 4 && LW <= 4 && NS >= 3 && LDS * PER_CU <= 160 * 1024, "tile shape");
};

constexpr int kGroup = 8;
// Tiles of a symmetric result that are computed: those that reach the diagonal or lie above it.
template <class G> __host__ __device__ inline int sym_tiles(int nt, int nw) {
  static_assert(G::TT % G::TW == 0, "whole tiles in a square of the diagonal");
  int n = 0;
  for (int r = 0; r < nt; ++r) n += nw - G::TT / G::TW * r > 0 ? nw - G::TT / G::TW * r : 0;
  return n;
}

template <class G, int EPI>
__device__ __forceinline__ void muon_tile(const Product& p, uint8_t* __restrict__ lds) {
  constexpr bool SYM = EPI == GRAM || EPI == POLY;
  if (skipped(p.scalars)) return;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // ---- which tile: each XCD a contiguous eighth of them
  // and in it kGroup rows of tiles side by side, column by column: what the
  // XCD's CUs work on at a time is near a square, whose operands are fewest.
  const int nt = (p.t_rows + G::TT - 1) / G::TT, nw = (p.w_rows + G::TW - 1) / G::TW;
  const int per = SYM ? sym_tiles<G>(nt, nw) : nt * nw, total = per * p.mats;
  const int id = EPI == GRAM ? blockIdx.x / p.pieces : blockIdx.x, piece = EPI == GRAM ? blockIdx.x % p.pieces : 0;
  const int q = total / 8, left = total % 8, x = id % 8;
  const int t = x * q + (x < left ? x : left) + id / 8;
  if (id / 8 >= q + (x < left)) return;
  const int mat = t / per;
  int tt = 0, tw = 0, at = t % per;
  if (SYM) {                                    // tile (tt, tw) is there if tw >= R tt
    constexpr int R = G::TT / G::TW;
    for (;; tt += kGroup) {
      const int rows = nt - tt < kGroup ? nt - tt : kGroup;
      int n = 0;
      for (int r = 0; r < rows; ++r) n += nw - R * (tt + r) > 0 ? nw - R * (tt + r) : 0;
      if (at < n) break;
      at -= n;
    }
    for (tw = R * tt;; ++tw) {
      int n = tw / R - tt + 1;
      n = n < kGroup ? n : kGroup;
      n = n < nt - tt ? n : nt - tt;
      if (at < n) break;
      at -= n;
    }
    tt += at;
  } else {
    tt = at / (kGroup * nw) * kGroup;
    const int rows = nt - tt < kGroup ? nt - tt : kGroup;
    at -= tt * nw;
    tw = at / rows;
    tt += at % rows;
  }
  const int t0 = tt * G::TT, w0 = tw * G::TW;
  int first = 0, steps = p.K / G::KS;           // K-steps of this workgroup
  if (EPI == GRAM && p.pieces > 1) {
    first = piece * steps / p.pieces;
    steps = (piece + 1) * steps / p.pieces - first;
  }

  // ---- loads: a lane's row and chunk of each KiB.  Rows past an operand's read
  // the next block's, or past the end zero: they reach only results past the
  // end, which are not stored.
  auto rsrc = [&](const _Float16* base, int64_t rows) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16*>(base), 0,
                                             static_cast<int32_t>(rows * p.K * 2), 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t rt = rsrc(p.t + mat * p.t_mat, p.t_rows), rw = rsrc(p.w + mat * p.w_mat, p.w_rows);
  uint32_t at_t[4], at_w[4];
  auto place = [&](int j, int tile_rows, int first, int rows) {
    const int kib = j * G::WAVES + wave, r = kib % (tile_rows / 16) * 16 + lane / 4;
    return (static_cast<uint32_t>(kib / (tile_rows / 16)) * rows + first + r) * 64u + ((lane & 3) ^ ((r >> 2) & 3)) * 16u;
  };
#pragma unroll
  for (int j = 0; j < G::LT; ++j) at_t[j] = place(j, G::TT, t0, p.t_rows);
#pragma unroll
  for (int j = 0; j < G::LW; ++j) at_w[j] = place(j, G::TW, w0, p.w_rows);
  const uint32_t step_t = static_cast<uint32_t>(p.t_rows) * (64u * G::KB), step_w = static_cast<uint32_t>(p.w_rows) * (64u * G::KB);
  auto stage = [&](int b) { return lds + b * G::STAGE; };
  auto issue_t = [&](int s, int b) {
    const uint32_t off = static_cast<uint32_t>(first + (s < steps ? s : steps - 1)) * step_t;   // past the end: nobody reads it
#pragma unroll
    for (int j = 0; j < G::LT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rt, (lds_ptr_t)(stage(b) + (j * G::WAVES + wave) * 1024), 16,
                                               at_t[j], off, 0, 0);
  };
  auto issue_w = [&](int s, int b) {
    const uint32_t off = static_cast<uint32_t>(first + (s < steps ? s : steps - 1)) * step_w;
#pragma unroll
    for (int j = 0; j < G::LW; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (lds_ptr_t)(stage(b) + G::KB * G::TT * G::ROW + (j * G::WAVES + wave) * 1024), 16, at_w[j], off, 0, 0);
  };

  // ---- main loop.  A step has k-slices of 16: fragments of a slice are read
  // while the one before it is multiplied, those of the next step's first with
  // the last, behind the barrier that says that this stage is read and the next
  // one has landed.  A stage is loaded again in two halves, W's behind the
  // barrier, T's before the next one: in one burst the loads would hold up the
  // matrix instructions behind them (measured: half the rate).
  const int wt = wave % G::WT * (G::TT / G::WT), ww = wave / G::WT * (G::TW / G::WW);
  f16x8_t wf[2][G::FW], tf[2][G::FT];
  const int fr = lane & 31, fh = lane >> 5;
  auto read = [&](int set, int b, int slice) {
    const int at = fr * G::ROW + ((2 * (slice & 1) + fh) ^ ((fr >> 2) & 3)) * 16;
    const uint8_t* T = stage(b) + (slice / 2 * G::TT + wt) * G::ROW + at;
    const uint8_t* W = stage(b) + (G::KB * G::TT + slice / 2 * G::TW + ww) * G::ROW + at;
#pragma unroll
    for (int i = 0; i < G::FW; ++i) wf[set][i] = __builtin_bit_cast(f16x8_t, chunk16(W + 32 * i * G::ROW));
#pragma unroll
    for (int j = 0; j < G::FT; ++j) tf[set][j] = __builtin_bit_cast(f16x8_t, chunk16(T + 32 * j * G::ROW));
  };
  f32x16_t acc[G::FW][G::FT];
  auto multiply = [&](int set) {
#pragma unroll
    for (int j = 0; j < G::FT; ++j)
#pragma unroll
      for (int i = 0; i < G::FW; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wf[set][i], tf[set][j], acc[i][j], 0, 0, 0);
  };
#pragma unroll
  for (int s = 0; s < G::NS; ++s) {
    issue_w(s, s);
    if (s + 1 < G::NS) issue_t(s, s);
  }
#pragma unroll
  for (int i = 0; i < G::FW; ++i)
#pragma unroll
    for (int j = 0; j < G::FT; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  constexpr int MF = G::FW * G::FT, RD = G::FW + G::FT;
  wait_vm_barrier<(G::NS - 2) * G::LPS + G::LW>();
  read(0, 0, 0);
  int buf = 0;
  for (int s = 0; s < steps; ++s) {
    const int next = buf + 1 == G::NS ? 0 : buf + 1;
#pragma unroll
    for (int slice = 0; slice + 1 < 2 * G::KB; ++slice) {
      read((slice + 1) & 1, buf, slice + 1);
      if (slice == 0) issue_t(s - 1 + G::NS, buf == 0 ? G::NS - 1 : buf - 1);
      multiply(slice & 1);
      if (slice == 0) interleave<MF, RD, G::LT>(); else interleave<MF, RD, 0>();
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vm_barrier<(G::NS - 2) * G::LPS>();
    read(0, next, 0);
    issue_w(s + G::NS, buf);
    multiply(1);
    interleave<MF, RD, G::LW>();
    __builtin_amdgcn_sched_barrier(0);
    buf = next;
  }
  wait_vm_barrier<0>();

  // ---- pieces of K: the workgroup that comes last adds the others' sums up,
  // all of them in order, whichever it is
  if constexpr (EPI == GRAM) {
    if (p.pieces > 1) {
      // Sums go and come as relaxed atomics of the whole GPU, which pass by the
      // XCDs' own L2s: a release and an acquire would write back and drop all
      // that these hold (measured: 19 us for 384 x 7168 instead of 9).  The wait
      // for the stores is what orders them before the count, and the branch on the
      // count what orders the loads behind it.  That is gfx950's way with such
      // stores and loads (each complete when vmcnt has counted it, none served from
      // an older line), an assumption on the hardware: the language promises it
      // for release and acquire alone.
      constexpr int64_t EACH = static_cast<int64_t>(G::TT) * G::TW;
      float* mine = p.parts + (static_cast<int64_t>(t) * p.pieces + piece) * EACH + tid;
#pragma unroll
      for (int i = 0; i < G::FW; ++i)
#pragma unroll
        for (int j = 0; j < G::FT; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            __hip_atomic_store(mine + ((i * G::FT + j) * 16 + k) * G::THREADS, acc[i][j][k], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      int32_t* came = reinterpret_cast<int32_t*>(lds);
      if (tid == 0) {
        *came = __hip_atomic_fetch_add(p.arrived + t, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (*came == p.pieces - 1)               // for the next launch
          __hip_atomic_store(p.arrived + t, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (*came != p.pieces - 1) return;
      asm volatile("" ::: "memory");
      float* all = p.parts + static_cast<int64_t>(t) * p.pieces * EACH + tid;
#pragma unroll
      for (int i = 0; i < G::FW; ++i)
#pragma unroll
        for (int j = 0; j < G::FT; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
#pragma unroll 2
      for (int s = 0; s < p.pieces; ++s) {
#pragma unroll
        for (int i = 0; i < G::FW; ++i)
#pragma unroll
          for (int j = 0; j < G::FT; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
              acc[i][j][k] += __hip_atomic_load(all + s * EACH + ((i * G::FT + j) * 16 + k) * G::THREADS,
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
    }
  }

  // ---- results, 32 x 32 at a time.  Lane (r, h) of a block has row r and
  // columns 8 g + 4 h .. + 3; the halves exchange, and it has columns 16 k + 8 h
  // .. + 7 of k = 0, 1.  The block is stored as it is, and turned through LDS.
  // What it is added to is loaded AHEAD blocks before: no load passes the
  // stores (X is replaced where it lies), and each would wait for memory.
  // A block is whole or not there at all (rows of operands come in 64s), so a
  // block's place is a scalar and a lane's place in it the same for all.
  constexpr int BLOCKS = G::FW * G::FT, AHEAD = BLOCKS < 4 ? BLOCKS : EPI == LAST_STEP ? 2 : 4;
  uint16_t* own = reinterpret_cast<uint16_t*>(lds + wave * G::OWN);
  float* wide = reinterpret_cast<float*>(own);
  const int64_t o_mat = static_cast<int64_t>(mat) * p.t_rows * p.w_rows;
  const int32_t o_bytes = static_cast<int32_t>(static_cast<int64_t>(p.t_rows) * p.w_rows * 2);
  const __amdgpu_buffer_rsrc_t r_add = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<_Float16*>(EPI == GRAM ? p.out : p.add) + o_mat, 0, o_bytes, 0x00020000);
  // Stored through plain pointers: a buffer store of 16 bytes with its offset in
  // a scalar register was seen to take its first four bytes from what the next
  // instruction wrote over them (16 lanes' last four, with other workgroups on
  // the CU); for these the compiler keeps the two apart.
  uint8_t* out = reinterpret_cast<uint8_t*>(p.out + o_mat);
  uint8_t* turned = reinterpret_cast<uint8_t*>(p.out_t + o_mat);
  const bool by_row = EPI == POLY || !p.rest_cols, by_col = EPI == POLY || p.rest_cols;
  const float* rest = EPI == GRAM ? nullptr : p.rest_in + static_cast<int64_t>(mat) * (by_row ? p.t_rows : p.w_rows);
  float keep = 1.0f, step = 0.0f;               // LAST_STEP
  if (EPI == LAST_STEP) {
    const double lr = p.scalars ? static_cast<double>(p.scalars->lr) : p.lr;
    keep = static_cast<float>(1.0 - lr * p.weight_decay);
    step = static_cast<float>(-lr * p.scale * kBack);
  }
  const int lane_at = fr * 64 + fh * 16;        // bytes of a lane's place in a block, k = 0
  const int64_t out0 = (static_cast<int64_t>(mat) * p.rows + t0 + wt) * p.cols + w0 + ww;   // LAST: the wave's first value
  u32x4_t add[AHEAD][2];
  float4 col_rest[AHEAD][4], old[AHEAD][4];    // old: p (LAST_STEP)
  float row_rest[AHEAD];
  auto row0_of = [&](int b) { return t0 + wt + 32 * (b / G::FW); };
  auto col0_of = [&](int b) { return w0 + ww + 32 * (b % G::FW); };
  auto there = [&](int b) { return row0_of(b) < p.t_rows && col0_of(b) < p.w_rows; };
  auto fetch = [&](int b) {
    if constexpr (EPI != GRAM) {
      if (!there(b)) return;
      const int set = b % AHEAD, at = (col0_of(b) / 32 * p.t_rows + row0_of(b)) * 64;   // below 2^31: sides up to 32768
      row_rest[set] = by_row ? rest[row0_of(b) + fr] : 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        add[set][k] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r_add, lane_at + 32 * k, at, 0));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          col_rest[set][2 * k + i] = by_col ? *reinterpret_cast<const float4*>(rest + col0_of(b) + 16 * k + 8 * fh + 4 * i)
                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
      if constexpr (EPI == LAST_STEP) {
        const float* from = p.p + out0 + static_cast<int64_t>(32 * (b / G::FW)) * p.cols + 32 * (b % G::FW);
        float* q = reinterpret_cast<float*>(old[set]);
        if (p.vec) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 8, c = lane % 8 * 4;
            if (row0_of(b) + r < p.rows && col0_of(b) + c < p.cols)
              old[set][i] = *reinterpret_cast<const float4*>(from + static_cast<int64_t>(r) * p.cols + c);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + lane / 32, c = lane % 32;
            if (row0_of(b) + r < p.rows && col0_of(b) + c < p.cols) q[i] = from[static_cast<int64_t>(r) * p.cols + c];
          }
        }
      }
    }
  };
#pragma unroll
  for (int b = 0; b < AHEAD; ++b) fetch(b);
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    if (there(b)) {
      const f32x16_t& a16 = acc[b % G::FW][b / G::FW];
      const int set = b % AHEAD, row = row0_of(b) + fr, col0 = col0_of(b) + 8 * fh;
      float f[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // columns 8 (2 k) + 4 h + i and 8 (2 k + 1) + 4 h + i: the upper half's first for the lower half's second
          const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a16[8 * k + i]),
                                                          __float_as_uint(a16[8 * k + 4 + i]), false, false);
          f[k][i] = __uint_as_float(s[0]) * p.c_acc;
          f[k][4 + i] = __uint_as_float(s[1]) * p.c_acc;
        }
      if constexpr (EPI != GRAM) {
        const float rr = row_rest[set];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 c0 = col_rest[set][2 * k], c1 = col_rest[set][2 * k + 1];
          const float rc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = static_cast<float>(
                __builtin_bit_cast(_Float16, static_cast<uint16_t>(add[set][k][i / 2] >> (16 * (i % 2)))));
            if (EPI == POLY) {          // b (G + D) + c (H H + D H + H D)
              const float d = row == col0 + 16 * k + i ? rr : 0.0f;
              f[k][i] = __builtin_fmaf(p.c_add, a + d, __builtin_fmaf(p.c_acc * (rc[i] + rr), a, f[k][i]));
            } else {                    // (a + rest) X + B X
              f[k][i] = __builtin_fmaf(__builtin_fmaf(rc[i] + rr, kBack, p.c_add), a, f[k][i]);
            }
          }
        }
      }
      if constexpr (EPI <= UPDATE) {
        uint16_t h[2][8];
        const int64_t at = (static_cast<int64_t>(col0_of(b) / 32) * p.t_rows + row0_of(b)) * 64;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          u32x4_t w;
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k][i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f[k][i]));
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = h[k][2 * i] | static_cast<uint32_t>(h[k][2 * i + 1]) << 16;
          *reinterpret_cast<u32x4_t*>(out + at + lane_at + 32 * k) = w;
        }
        if (SYM && row0_of(b) == col0_of(b)) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (row == col0 + 16 * k + i)
                p.rest_out[static_cast<int64_t>(mat) * p.t_rows + row] =
                    f[k][i] - static_cast<float>(__builtin_bit_cast(_Float16, h[k][i]));
        }
        if (!SYM || tw * G::TW >= (tt + 1) * G::TT) {
          const int64_t to = (static_cast<int64_t>(row0_of(b) / 32) * p.w_rows + col0_of(b)) * 64;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) own[(16 * k + 8 * fh + i) * G::PITCH + fr] = h[k][i];
          // (the reads' type says that they are of other memory than the writes; lanes read others' values)
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<u32x4_t*>(turned + to + lane * 16 + 1024 * k) =
                chunk16(reinterpret_cast<const uint8_t*>(own + (16 * k + lane / 4) * G::PITCH + lane % 4 * 8));
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
      } else {
        // rows of the block side by side, so that lanes run along a row of the result
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4*>(wide + fr * G::WIDE + 16 * k + 8 * fh + 4 * i) =
                make_float4(f[k][4 * i], f[k][4 * i + 1], f[k][4 * i + 2], f[k][4 * i + 3]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // lanes read others' values
        const int64_t to0 = out0 + static_cast<int64_t>(32 * (b / G::FW)) * p.cols + 32 * (b % G::FW);
        uint16_t* half = EPI == LAST_OUT ? p.o : p.p_bf16;
        if (p.vec) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 8, c = lane % 8 * 4;
            float4 v = *reinterpret_cast<const float4*>(wide + r * G::WIDE + c);
            if (row0_of(b) + r >= p.rows || col0_of(b) + c >= p.cols) continue;
            const int64_t to = to0 + static_cast<int64_t>(r) * p.cols + c;
            if constexpr (EPI == LAST_OUT) {
              v = make_float4(v.x * kBack, v.y * kBack, v.z * kBack, v.w * kBack);
            } else {
              const float4 o = old[set][i];
              v = make_float4(__builtin_fmaf(step, v.x, o.x * keep), __builtin_fmaf(step, v.y, o.y * keep),
                              __builtin_fmaf(step, v.z, o.z * keep), __builtin_fmaf(step, v.w, o.w * keep));
              *reinterpret_cast<float4*>(p.p + to) = v;
            }
            if (half) *reinterpret_cast<uint2*>(half + to) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          }
        } else {
          const float* q = reinterpret_cast<const float*>(old[set]);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + lane / 32, c = lane % 32;
            float v = wide[r * G::WIDE + c];
            if (row0_of(b) + r >= p.rows || col0_of(b) + c >= p.cols) continue;
            const int64_t to = to0 + static_cast<int64_t>(r) * p.cols + c;
            if constexpr (EPI == LAST_OUT) {
              v *= kBack;
            } else {
              v = __builtin_fmaf(step, v, q[i] * keep);
              p.p[to] = v;
            }
            if (half) half[to] = f32_to_bf16(v);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read before the next block's are written
      }
    }
    if (b + AHEAD < BLOCKS) fetch(b + AHEAD);
    __builtin_amdgcn_sched_barrier(0);           // one block's registers at a time
  }
}

template <class G, int EPI>
__global__ __launch_bounds__(G::THREADS, G::PER_CU) void k_muon_product(const Product p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[G::LDS];
  muon_tile<G, EPI>(p, lds);
}

using Half = Geo16<256, 128, 2, 2, 32, 3, 2>;
using Mid = Geo16<128, 128, 2, 2, 32, 4, 2>;
using Small = Geo16<64, 64, 2, 2, 64, 3, 3>;

template <class G, int EPI> int64_t tiles_of(const Product& p) {
  const int nt = (p.t_rows + G::TT - 1) / G::TT, nw = (p.w_rows + G::TW - 1) / G::TW;
  return static_cast<int64_t>(EPI <= POLY ? sym_tiles<G>(nt, nw) : nt * nw) * p.mats;
}
template <class G, int EPI> hipError_t run(const Product& p, hipStream_t s) {
  hipLaunchKernelGGL((k_muon_product<G, EPI>), dim3(static_cast<unsigned>(tiles_of<G, EPI>(p) * p.pieces)),
                     dim3(G::THREADS), 0, s, p);
  return hipGetLastError();
}
// The largest tile that leaves no CU idle and little of itself past the edges.
// Measured, all products of a call in one size: 2 x 4096 x 2048 256 x 128 tiles 883 us, 128 x 128 870,
// 64 x 64 1069; 2048 x 7168 982, 811, 937; 1024 x 1024 324, 215, 143; 48 x 333 x
// 190 (a third of each 128 x 128 tile past the edge) -, 139, 125.
// Near the border, calls with B X in 128 x 128 tiles and in 64 x 64, all else alike: 128 tiles (1024 x 2048) 176, 167
// us; 160 (512 x 5120) 155, 155; 168 (384 x 7168) 161, 157; 192 (512 x 6144) 158, 159, (768 x 4096) 170, 171, (12 x
// 512 x 512) 144, 142; 200 (640 x 5120) 170, 182; 216 (24 x 384 x 384) 131, 136; 256 (1024 x 4096) 229, 237.  With
// X X^T and G^2 in them: 108 tiles (3 x 1024 x 1024) 221, 195; 120 (12 x 512 x 512) 163, 142; 144 (4 x 1024 x 1024) 248,
// 246; 156 (2 x 1536 x 1536) 334, 340; 160 (16 x 512 x 512) 180, 175.
template <int EPI> hipError_t run(Product p, hipStream_t s) {
  p.pieces = 1;
  const int64_t half = tiles_of<Half, EPI>(p), mid = tiles_of<Mid, EPI>(p), small = tiles_of<Small, EPI>(p);
  if (half >= 768 && 20 * half <= 11 * mid) return run<Half, EPI>(p, s);
  if (mid >= 192 && 10 * mid <= 3 * small) return run<Mid, EPI>(p, s);
  if (EPI == GRAM) p.pieces = gram_pieces(small, p.K);
  return run<Small, EPI>(p, s);
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
  auto aligned = [](const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  const bool vec = sh.cols % 4 == 0 && aligned(in.x, in.bf16 ? 8 : 16) && aligned(in.m, 16);
  const dim3 chunks(sh.chunks, n), tiles(sh.mp / 64 * (sh.np / 64), n);
  if (vec) hipLaunchKernelGGL(k_muon_norm<true>, chunks, dim3(256), 0, s, in, sh, w.norms, w.arrived);
  else hipLaunchKernelGGL(k_muon_norm<false>, chunks, dim3(256), 0, s, in, sh, w.norms, w.arrived);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (vec) hipLaunchKernelGGL(k_muon_convert<true>, tiles, dim3(256), 0, s, in, sh, w.norms, w.x, w.xt[0]);
  else hipLaunchKernelGGL(k_muon_convert<false>, tiles, dim3(256), 0, s, in, sh, w.norms, w.x, w.xt[0]);
  e = hipGetLastError();
  for (int i = 0; i < a.ns.steps && e == hipSuccess; ++i) {
    const int64_t xm = static_cast<int64_t>(sh.mp) * sh.np, gm = static_cast<int64_t>(sh.mp) * sh.mp;
    Product g{};
    g.mats = a.n; g.scalars = a.scalars;
    g.t = g.w = w.x; g.t_rows = g.w_rows = sh.mp; g.K = sh.np; g.t_mat = g.w_mat = xm;
    g.out = g.out_t = w.g; g.c_acc = kBack; g.rest_out = w.g_rest; g.parts = w.parts; g.arrived = w.arrived;
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
      u.vec = a.cols % 4 == 0 && reinterpret_cast<uintptr_t>(a.p) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(a.p ? a.p_bf16 : a.out) % 8 == 0;
      u.lr = a.lr; u.weight_decay = a.weight_decay; u.scale = a.scale;
      e = a.p ? run<LAST_STEP>(u, s) : run<LAST_OUT>(u, s);
    }
  }
  return e;
}

}  // namespace mok
