// Host-side launchers of the experts' training kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// What the calls of one training step share.  Rows: expert e owns the rows offsets[e] ..
// offsets[e] + counts[e] - 1 of the `rows` of every row buffer, and row r holds pair
// sorted_ids[r]; counts == nullptr: one expert, whose row r is token r.
struct TrainRows {
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* sorted_ids;
  int64_t tokens;   // T
  int64_t rows;     // of the row buffers: the plan's cap, or T
  int K;
  int E, H, I;
};

// The gate and up values a forward keeps: [rows][2I] bf16, or [rows][2I] e4m3 codes and
// [rows][2I / 32] biased exponents of their blocks' scales (fp8).
struct SavedRows {
  void* h;
  uint8_t* scales;
  bool fp8;
};

// Room for partial sums: launches of few items split their contraction into parts whose sums are
// added by a second kernel, as far as the room goes.
struct PartSpace {
  float* part;
  int64_t bytes;
};
constexpr int kMaxParts = 16;
constexpr int64_t kCounterBytes = 256;
// no more is needed: the parts of a launch are no more items than it has compute units, and each
// has at most 256 x 256 sums
constexpr int64_t kPartBytes = (int64_t)64 << 20;

// act [rows][I] = silu(g) * u with g, u = w13 x; g and u kept
hipError_t launch_train_gate_up(const TrainRows& r, const void* x, const void* w13,
                                const SavedRows& saved, uint16_t* act, const PartSpace& space,
                                hipStream_t s);
// y [rows][H] = w2 act
hipError_t launch_train_down(const TrainRows& r, const void* w2, const uint16_t* act, void* y,
                             const PartSpace& space, hipStream_t s);
// from da = w2^T dy: act = silu(g) * u, and dh [rows][2I], the gradients of g and of u; counters
// (8) are cleared
hipError_t launch_train_dact(const TrainRows& r, const void* w2, const void* dy,
                             const SavedRows& saved, uint16_t* act, uint16_t* dh, int* counters,
                             const PartSpace& space, hipStream_t s);
// dx [rows][H] = w13^T dh, dw13 [E][2I][H] = sum over an expert's rows of dh x^T (x_rows: x by row)
// and dw2 [E][H][I] that of dy act^T, each where given; f32: the type of dw13 and dw2 is fp32, else
// bf16; counters: those that launch_train_dact has cleared (where there are tokens)
hipError_t launch_train_grads(const TrainRows& r, const void* w13, const uint16_t* dh, void* dx,
                              const uint16_t* x_rows, void* dw13, const uint16_t* act,
                              const void* dy, void* dw2, bool f32, const PartSpace& space,
                              int* counters, hipStream_t s);

// [T][H] values in blocks of 32 to e4m3 codes and the biased exponents of the blocks' scales
hipError_t launch_pack_fp8(const void* x, int dt, int64_t T, int H, uint8_t* codes,
                           uint8_t* scales, hipStream_t s);
hipError_t launch_unpack_fp8(const uint8_t* codes, const uint8_t* scales, int64_t T, int H,
                             void* x, int dt, hipStream_t s);

}  // namespace moe
