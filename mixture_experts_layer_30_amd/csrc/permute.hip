// Tokens in the rows of an alignment and back, with weights, and the gradients
// (what each computes: include/moe_layer.h).
//
// Everything here is bound by memory: a row element is moved once and takes at
// most one multiply-add.  The kernels go by token, not by row: a token's row is
// read once for its K copies (permute, unpermute_backward) and its K rows are
// summed in slot order in registers (unpermute), so no sum needs atomics.  The
// padding rows have no token; workgroups past the tokens' zero them, taking the
// alignment's blocks one by one (each belongs to one expert, whose rows end at
// offsets[e] + counts[e]).
#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kThreads = 256;
constexpr int kPadRows = 16;   // padding rows of one block that a workgroup zeroes at a time

// Zeroes the padding rows of work item `item`: rows sub * kPadRows .. of block
// item / subs (rows of nv 16-byte vectors).
__device__ __forceinline__ void zero_padding(int64_t item, int subs, int block_m, int E,
                                             const int32_t* counts, const int32_t* offsets,
                                             const int32_t* block_expert, int nv, u32x4* rows) {
  const int64_t b = item / subs;
  const int e = block_expert[b];
  if (e < 0 || e >= E) return;
  const int64_t lo = b * block_m + (item - b * subs) * kPadRows;
  int64_t end = lo + kPadRows;
  if (end > (b + 1) * block_m) end = (b + 1) * block_m;
  int64_t r = (int64_t)offsets[e] + counts[e];
  if (r < lo) r = lo;
  const u32x4 z = {0, 0, 0, 0};
  for (; r < end; ++r)
    for (int v = threadIdx.x; v < nv; v += kThreads) rows[r * nv + v] = z;
}

// rows[inv_pos[t*K + k]] = x[t].  tx lanes (a power of two) share a token and
// cover tx of its nv vectors; units = token groups x chunks of tx vectors.
__global__ __launch_bounds__(kThreads) void permute_kernel(
    const u32x4* __restrict__ x, int64_t T, int K, int nv, int tx_log2, int chunks, int64_t units,
    const int32_t* __restrict__ inv_pos, int64_t cap, u32x4* __restrict__ rows, int64_t pad_items,
    int pad_subs, int block_m, int E, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ block_expert) {
  const int tx = 1 << tx_log2;
  const int ty = kThreads >> tx_log2;
  for (int64_t u = blockIdx.x; u < units + pad_items; u += gridDim.x) {
    if (u >= units) {
      zero_padding(u - units, pad_subs, block_m, E, counts, offsets, block_expert, nv, rows);
      continue;
    }
    const int64_t g = u / chunks;
    const int v = (int)(u - g * chunks) * tx + (threadIdx.x & (tx - 1));
    const int64_t t = g * ty + (threadIdx.x >> tx_log2);
    if (t >= T || v >= nv) continue;
    const u32x4 d = x[t * nv + v];
    for (int k = 0; k < K; ++k) {
      const int64_t r = inv_pos[t * K + k];
      if (r >= 0 && r < cap) rows[r * nv + v] = d;
    }
  }
}

constexpr int kSlots = 4;   // rows in flight per thread

// out[t] = sum_k w[t][k] rows[inv_pos[t*K + k]] (+ shared[t]): a thread owns 8
// elements of a token.
template <class SR, class SS, class SO, bool kWeighted>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(
    const typename SR::T* __restrict__ rows, const float* __restrict__ w,
    const typename SS::T* __restrict__ shared, int64_t T, int K, int H, int tx_log2, int chunks,
    int64_t units, const int32_t* __restrict__ inv_pos, int64_t cap,
    typename SO::T* __restrict__ out) {
  const int tx = 1 << tx_log2;
  const int ty = kThreads >> tx_log2;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t g = u / chunks;
    const int h = ((int)(u - g * chunks) * tx + (threadIdx.x & (tx - 1))) * 8;
    const int64_t t = g * ty + (threadIdx.x >> tx_log2);
    if (t >= T || h >= H) continue;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kSlots) {
      float v[kSlots][8], wk[kSlots];
      bool use[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        use[j] = false;
        if (k0 + j < K) {
          const int64_t r = inv_pos[t * K + k0 + j];
          wk[j] = kWeighted ? w[t * K + k0 + j] : 1.0f;
          use[j] = r >= 0 && r < cap && wk[j] != 0.0f;
          if (use[j]) load8f<SR>(rows + r * H + h, v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (use[j]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(wk[j], v[j][i], acc[i]);
        }
    }
    if (shared) {
      float v[8];
      load8f<SS>(shared + t * H + h, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    store8f<SO>(out + t * H + h, acc);
  }
}

constexpr int kGradSlots = 8;   // slots whose dot products a pass over the token holds

// drows[r] = w[t][k] dout[t] and dw[t][k] = <dout[t], rows[r]> for the rows r of
// token t.  kWaves wavefronts share a token (its elements dealt 8 to a lane),
// kThreads / 64 / kWaves tokens a workgroup; the dot products of up to 8 slots
// run together, are summed over each wavefront and then in wavefront order.
template <class S, int kWaves>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(
    const typename S::T* __restrict__ dout, const typename S::T* rows,
    const float* __restrict__ w, int64_t T, int K, int H, int64_t units,
    const int32_t* __restrict__ inv_pos, int64_t cap, typename S::T* drows,
    float* __restrict__ dw, int64_t pad_items, int pad_subs, int block_m, int E,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ block_expert) {
  constexpr int kTokens = kThreads / kWave / kWaves;
  __shared__ float part[kThreads / kWave][kGradSlots];
  const int wave = threadIdx.x / kWave;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t u = blockIdx.x; u < units + pad_items; u += gridDim.x) {
    if (u >= units) {   // (only where drows is written)
      zero_padding(u - units, pad_subs, block_m, E, counts, offsets, block_expert,
                   H * S::kBytes / 16, reinterpret_cast<u32x4*>(drows));
      continue;
    }
    const int64_t t = u * kTokens + wave / kWaves;
    const bool live = t < T;
    for (int k0 = 0; k0 < K; k0 += kGradSlots) {
      int64_t r[kGradSlots];
      float wk[kGradSlots], acc[kGradSlots];
#pragma unroll
      for (int j = 0; j < kGradSlots; ++j) {
        r[j] = -1;
        wk[j] = 1.0f;
        acc[j] = 0.0f;
        if (live && k0 + j < K) {
          r[j] = inv_pos[t * K + k0 + j];
          if (r[j] >= cap) r[j] = -1;
          if (w) wk[j] = w[t * K + k0 + j];
        }
      }
      if (live)
        for (int h = ((wave % kWaves) * kWave + lane) * 8; h < H; h += kWaves * kWave * 8) {
          float g[8];
          load8f<S>(dout + t * H + h, g);
          if (dw) {
            float v[kGradSlots][8];
#pragma unroll
            for (int j = 0; j < kGradSlots; ++j)
              if (r[j] >= 0) load8f<S>(rows + r[j] * H + h, v[j]);
#pragma unroll
            for (int j = 0; j < kGradSlots; ++j)
              if (r[j] >= 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j] = fmaf(g[i], v[j][i], acc[j]);
              }
          }
          if (drows) {
#pragma unroll
            for (int j = 0; j < kGradSlots; ++j)
              if (r[j] >= 0) {
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = wk[j] * g[i];
                store8f<S>(drows + r[j] * H + h, s);
              }
          }
        }
      if (dw) {
#pragma unroll
        for (int j = 0; j < kGradSlots; ++j) acc[j] = wave_sum(acc[j]);
        if (kWaves == 1) {
#pragma unroll
          for (int j = 0; j < kGradSlots; ++j)
            if (live && lane == j && k0 + j < K) dw[t * K + k0 + j] = acc[j];
        } else {
#pragma unroll
          for (int j = 0; j < kGradSlots; ++j)
            if (lane == j) part[wave][j] = acc[j];
          __syncthreads();
          if (live && wave % kWaves == 0 && lane < kGradSlots && k0 + lane < K) {
            float sum = 0.0f;
            for (int i = 0; i < kWaves; ++i) sum += part[wave + i][lane];
            dw[t * K + k0 + lane] = sum;
          }
          __syncthreads();
        }
      }
    }
  }
}

// dlogits[t][e] = sum over the slots j with id e of w_j (dw_j - sum_i w_i dw_i).
// One wavefront a token, its slots held 64 to a register; each lane owns every
// 64th expert and looks the slots through in order.
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw,
    int64_t T, int E, int K, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t waves = (int64_t)gridDim.x * (kThreads / kWave);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; t < T;
       t += waves) {
    // at most 256 slots: 4 a lane
    int id[4];
    float g[4], s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = j * kWave + lane;
      id[j] = k < K ? ids[t * K + k] : -1;
      const bool used = id[j] >= 0 && id[j] < E;
      const float wk = used ? w[t * K + k] : 0.0f, d = used ? dw[t * K + k] : 0.0f;
      s = fmaf(wk, d, s);
      g[j] = wk;
      // (held until s is known)
      id[j] = used ? id[j] : -1;
    }
    s = wave_sum(s);
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = j * kWave + lane;
      g[j] = id[j] >= 0 ? g[j] * (dw[t * K + k] - s) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      for (int l = 0; l < kWave && j * kWave + l < K; ++l) {
        const int e = __builtin_amdgcn_readlane(id[j], l);
        const float ge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g[j]), l));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e == i * kWave + lane) o[i] += ge;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * kWave + lane < E) dlogits[t * E + i * kWave + lane] = o[i];
  }
}

namespace {

// Lanes that share a token: the smallest power of two covering its nv vectors,
// between 8 and the workgroup.
int lanes_log2(int nv) {
  int l = 3;
  while (l < 8 && (1 << l) < nv) ++l;
  return l;
}

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups; the kernels loop past it

unsigned grid_of(int64_t units) { return (unsigned)(units < kMaxGrid ? units : kMaxGrid); }

int pad_subs(int block_m) { return (block_m + kPadRows - 1) / kPadRows; }

template <class SR, class SS, class SO>
hipError_t launch_unpermute_t(const void* rows, const float* w, const void* shared, int64_t T,
                              int K, int H, const int32_t* inv_pos, int64_t cap, void* out,
                              hipStream_t s) {
  const int l = lanes_log2(H / 8);
  const int ty = kThreads >> l, chunks = (H / 8 + (1 << l) - 1) >> l;
  const int64_t units = (T + ty - 1) / ty * chunks;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid_of(units)), dim3(kThreads), 0, s,
                       static_cast<const typename SR::T*>(rows), w,
                       static_cast<const typename SS::T*>(shared), T, K, H, l, chunks, units,
                       inv_pos, cap, static_cast<typename SO::T*>(out));
  };
  if (w) go(unpermute_kernel<SR, SS, SO, true>);
  else go(unpermute_kernel<SR, SS, SO, false>);
  return hipGetLastError();
}

template <class SR, class SS>
hipError_t unpermute_out(const void* rows, const float* w, const void* shared, int64_t T, int K,
                         int H, const int32_t* inv_pos, int64_t cap, void* out, int odt,
                         hipStream_t s) {
  return odt == kDtF32
             ? launch_unpermute_t<SR, SS, F32>(rows, w, shared, T, K, H, inv_pos, cap, out, s)
             : launch_unpermute_t<SR, SS, BF16>(rows, w, shared, T, K, H, inv_pos, cap, out, s);
}

}  // namespace

hipError_t launch_permute(const void* x, int dt, int64_t T, int K, int H, const RowMap& rm, int E,
                          int64_t cap, void* rows, hipStream_t s) {
  const int nv = H / 8 * (dt == kDtF32 ? 2 : 1);
  const int l = lanes_log2(nv);
  const int ty = kThreads >> l, chunks = (nv + (1 << l) - 1) >> l;
  const int64_t units = (T + ty - 1) / ty * chunks;
  const int64_t pad = rm.block_m > 1 ? cap / rm.block_m * pad_subs(rm.block_m) : 0;
  hipLaunchKernelGGL(permute_kernel, dim3(grid_of(units + pad)), dim3(kThreads), 0, s,
                     static_cast<const u32x4*>(x), T, K, nv, l, chunks, units, rm.inv_pos, cap,
                     static_cast<u32x4*>(rows), pad, pad_subs(rm.block_m), rm.block_m, E,
                     rm.counts, rm.offsets, rm.block_expert);
  return hipGetLastError();
}

hipError_t launch_unpermute(const void* rows, int rdt, const float* w, const void* shared, int sdt,
                            int64_t T, int K, int H, const int32_t* inv_pos, int64_t cap,
                            void* out, int odt, hipStream_t s) {
  if (rdt == kDtF32)
    return sdt == kDtF32
               ? unpermute_out<F32, F32>(rows, w, shared, T, K, H, inv_pos, cap, out, odt, s)
               : unpermute_out<F32, BF16>(rows, w, shared, T, K, H, inv_pos, cap, out, odt, s);
  return sdt == kDtF32
             ? unpermute_out<BF16, F32>(rows, w, shared, T, K, H, inv_pos, cap, out, odt, s)
             : unpermute_out<BF16, BF16>(rows, w, shared, T, K, H, inv_pos, cap, out, odt, s);
}

hipError_t launch_unpermute_backward(const void* dout, const void* rows, int dt, const float* w,
                                     int64_t T, int K, int H, const RowMap& rm, int E, int64_t cap,
                                     void* drows, float* dw, hipStream_t s) {
  const int64_t pad =
      drows && rm.block_m > 1 ? cap / rm.block_m * pad_subs(rm.block_m) : 0;
  // one wavefront holds a token of up to 1024 elements in two steps; a longer one
  // takes the workgroup
  const bool one = H <= 1024;
  const int64_t units = one ? (T + 3) / 4 : T;
  auto go = [&](auto kernel, auto* type) {
    typedef std::remove_pointer_t<decltype(type)> E_;
    hipLaunchKernelGGL(kernel, dim3(grid_of(units + pad)), dim3(kThreads), 0, s,
                       static_cast<const E_*>(dout), static_cast<const E_*>(rows), w, T, K, H,
                       units, rm.inv_pos, cap, static_cast<E_*>(drows), dw, pad,
                       pad_subs(rm.block_m), rm.block_m, E, rm.counts, rm.offsets,
                       rm.block_expert);
  };
  if (dt == kDtF32) {
    if (one) go(unpermute_backward_kernel<F32, 1>, (float*)nullptr);
    else go(unpermute_backward_kernel<F32, 4>, (float*)nullptr);
  } else {
    if (one) go(unpermute_backward_kernel<BF16, 1>, (uint16_t*)nullptr);
    else go(unpermute_backward_kernel<BF16, 4>, (uint16_t*)nullptr);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, int64_t T,
                                 int E, int K, float* dlogits, hipStream_t s) {
  const int64_t units = (T + kThreads / kWave - 1) / (kThreads / kWave);
  hipLaunchKernelGGL(route_backward_kernel, dim3(grid_of(units)), dim3(kThreads), 0, s, ids, w, dw,
                     T, E, K, dlogits);
  return hipGetLastError();
}

}  // namespace moe
