// Launch entry points of the operators around the experts.
#pragma once

#include "kernels.h"

namespace moe {

// Rows in the alignment's order and back (rm: the plan's arrays and block_m).
hipError_t launch_permute(const void* x, int dt, int64_t T, int K, int H, const RowMap& rm, int E,
                          int64_t cap, void* rows, hipStream_t s);
// w null: weights 1
hipError_t launch_unpermute(const void* rows, int rdt, const float* w, const void* shared, int sdt,
                            int64_t T, int K, int H, const int32_t* inv_pos, int64_t cap,
                            void* out, int odt, hipStream_t s);
hipError_t launch_unpermute_backward(const void* dout, const void* rows, int dt, const float* w,
                                     int64_t T, int K, int H, const RowMap& rm, int E, int64_t cap,
                                     void* drows, float* dw, hipStream_t s);
hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, int64_t T,
                                 int E, int K, float* dlogits, hipStream_t s);

// The norms around a block (kind as moe_norm_kind; pointers of the call's
// parameter type) and the gate on its output.
constexpr int kNormNone = 0;
constexpr int kNormRms = 1;
constexpr int kNormLayer = 2;
struct NormSpec {
  int kind;
  float eps;
  const void* weight;
  const void* bias;
};
struct GateSpec {
  float alpha;
  const void* channel;
  const float* token;
};

hipError_t launch_norm(const void* x, int xdt, int64_t T, int H, const NormSpec& n, int pdt,
                       void* out, int odt, hipStream_t s);
// n null: r alone
hipError_t launch_norm_residual(const void* y, int ydt, const void* x, int xdt, int64_t T, int H,
                                const NormSpec& post, const GateSpec& gate, int pdt, void* r,
                                const NormSpec& pre, void* n, hipStream_t s);
hipError_t launch_combine_norm_residual(const void* y, int ydt, const float* w, int K,
                                        const void* shared, int sdt, const void* x, int xdt,
                                        int64_t T, int H, const NormSpec& post,
                                        const GateSpec& gate, int pdt, void* r,
                                        const NormSpec& pre, void* n, hipStream_t s);
// fp32 partial sums of a backward launch (all the parameter gradients)
int64_t norm_workspace_floats(int64_t T, int H);
// From e, the gradient of gate * norm(v): dv (+ dres, null: none; as v), the
// parameters' gradients and the gates', each where not null.
hipError_t launch_norm_backward(const void* e, int edt, const void* v, int vdt, const void* dres,
                                int64_t T, int H, const NormSpec& n, const GateSpec& gate, int pdt,
                                void* dv, float* dweight, float* dbias, float* dchannel,
                                float* dtoken, float* workspace, hipStream_t s);

}  // namespace moe
