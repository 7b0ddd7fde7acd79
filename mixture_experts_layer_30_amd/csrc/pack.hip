// Activations kept in 8 bits and read back (the format: pack.h).
//
// Bound by HBM: 2 bytes read and 1 + 1/32 written an element (bf16), or the reverse.  A lane
// takes 8 neighbours of a row (one 16-byte load of bf16, two of fp32), the 4 lanes of a quad
// a block of 32, whose maximum needs two swaps within the quad.  A row is a whole number of
// blocks, so a tensor is one run of them whatever its rows.
// Measured, 16384 x 7168 bf16, 356 MB each way: packed in 69 to 82 us (5.2 to 4.3 TB/s), read back
// in 54 (6.6); 5003 x 3584 fp32 16.4 and 16.7 us (5.5 and 5.4); a copy of 1 GB 5.15 TB/s.
#include "block_kernels.h"
#include "pack.h"
#include "rows.h"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kPackThreads = 256;
constexpr int kPackUnroll = 4;   // pieces of 8 values a lane has in flight

// pieces: of 8 values, a multiple of 4
template <class S>
__global__ __launch_bounds__(kPackThreads) void pack_kernel(const typename S::T* __restrict__ x,
                                                            int64_t pieces,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int64_t first = (int64_t)blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
  float v[kPackUnroll][8];
#pragma unroll
  for (int u = 0; u < kPackUnroll; ++u) {
    const int64_t p = first + u * kPackThreads;
    if (p < pieces) load8f<S>(x + p * 8, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kPackUnroll; ++u) {
    const int64_t p = first + u * kPackThreads;
    if (p < pieces) {   // the quad's four lanes agree
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = abs_max(most, v[u][j]);
      const int byte = scale_byte(quad_max(most));
      *reinterpret_cast<uint2*>(codes + p * 8) = pack_e4m3x8(v[u], inverse_scale(byte));
      if ((p & 3) == 0) scales[p >> 2] = (uint8_t)byte;
    }
  }
}

template <class S>
__global__ __launch_bounds__(kPackThreads) void unpack_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              int64_t pieces,
                                                              typename S::T* __restrict__ x) {
  const int64_t first = (int64_t)blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
  uint2 c[kPackUnroll];
  int byte[kPackUnroll];
#pragma unroll
  for (int u = 0; u < kPackUnroll; ++u) {
    const int64_t p = first + u * kPackThreads;
    if (p < pieces) {
      c[u] = *reinterpret_cast<const uint2*>(codes + p * 8);
      byte[u] = scales[p >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kPackUnroll; ++u) {
    const int64_t p = first + u * kPackThreads;
    if (p < pieces) {
      float v[8];
      unpack_e4m3x8(c[u], scale_of(byte[u]), v);
      store8f<S>(x + p * 8, v);
    }
  }
}

unsigned pack_grid(int64_t pieces) {
  const int64_t per = kPackThreads * kPackUnroll;
  return (unsigned)((pieces + per - 1) / per);
}

}  // namespace

hipError_t launch_pack_fp8(const void* x, int dt, int64_t T, int H, uint8_t* codes,
                           uint8_t* scales, hipStream_t s) {
  const int64_t pieces = T * (H / 8);
  if (pieces == 0) return hipSuccess;
  if (dt == kDtF32)
    hipLaunchKernelGGL(pack_kernel<F32>, dim3(pack_grid(pieces)), dim3(kPackThreads), 0, s,
                       static_cast<const float*>(x), pieces, codes, scales);
  else
    hipLaunchKernelGGL(pack_kernel<BF16>, dim3(pack_grid(pieces)), dim3(kPackThreads), 0, s,
                       static_cast<const uint16_t*>(x), pieces, codes, scales);
  return hipGetLastError();
}

hipError_t launch_unpack_fp8(const uint8_t* codes, const uint8_t* scales, int64_t T, int H,
                             void* x, int dt, hipStream_t s) {
  const int64_t pieces = T * (H / 8);
  if (pieces == 0) return hipSuccess;
  if (dt == kDtF32)
    hipLaunchKernelGGL(unpack_kernel<F32>, dim3(pack_grid(pieces)), dim3(kPackThreads), 0, s,
                       codes, scales, pieces, static_cast<float*>(x));
  else
    hipLaunchKernelGGL(unpack_kernel<BF16>, dim3(pack_grid(pieces)), dim3(kPackThreads), 0, s,
                       codes, scales, pieces, static_cast<uint16_t*>(x));
  return hipGetLastError();
}

}  // namespace moe
