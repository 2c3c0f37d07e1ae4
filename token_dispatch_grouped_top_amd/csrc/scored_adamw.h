// scored_adamw.h -- launchers of the scored route, its backward, the bias update
// and AdamW (kept out of mok_internal.h, by whose text the measured HBM bytes
// of the GEMMs are known to be of the present sources).
#pragma once

#include "mok_internal.h"

namespace mok {

// Scored route, its backward and the bias update (mok_router_desc, checked).
struct RouterArgs {
  int32_t E, k, G, gsize, top_groups;
  int32_t sigmoid, top2, renorm;
  float scale;
  int32_t log_m, chunk, wide, wide_bias;   // set by the launcher: how a row is split over lanes
};
hipError_t launch_route_scored(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                               const float* bias, int32_t T, int32_t* idx, float* gate,
                               int32_t* load, const RouteCount& rc, hipStream_t s);
hipError_t launch_route_scored_bwd(const RouterArgs& r, const void* logits, bool bf16, int64_t ld,
                                   int32_t T, const int32_t* idx, const float* dgate,
                                   void* dlogits, int64_t ldd, hipStream_t s);
hipError_t launch_bias_update(int32_t* load, int32_t n_layers, int32_t E, float rate, float* bias,
                              bool clear_load, hipStream_t s);

// AdamW over a list of tensors (checked): the units of a tensor (n > 0), the
// table's bytes, its writing, and the step.
constexpr int64_t kAdamwMaxUnits = (1 << 24) - 1;   // workgroups of a launch (2^32 threads)
int64_t adamw_units(int64_t n, bool mx);
size_t adamw_table_bytes(int64_t n);
hipError_t launch_adamw_table(const mok_adamw_tensor* tensors, int32_t n, void* table,
                              mok_adamw_plan& plan, hipStream_t s);
hipError_t launch_adamw(const void* table, const mok_adamw_plan& plan, const mok_adamw_hyper& h,
                        const mok_adamw_scalars* scalars, hipStream_t s);

}  // namespace mok
