// muon.h -- launcher of the orthogonalised update.
#pragma once

#include "mok_internal.h"

namespace mok {

constexpr int32_t kMuonMaxSide = 32768, kMuonMaxMats = 65535;

struct MuonArgs {
  // orthogonalise: x -> out (bf16); step: grad, m, p, p_bf16
  const void* x; int32_t x_bf16;               // x, or the gradient
  void* out;                                   // bf16
  float* p; void* p_bf16; float* m;            // step: p non-null
  int32_t n, rows, cols;
  mok_newton_schulz ns;
  double lr, momentum, weight_decay, grad_scale, scale;
  int32_t nesterov;
  const mok_adamw_scalars* scalars;
  void* ws;
};
size_t muon_ws_bytes(int32_t n, int32_t rows, int32_t cols);
hipError_t launch_muon(const MuonArgs& a, hipStream_t s);

}  // namespace mok
