// The norms before and after a block of a residual stream, with the block's
// gate and residual scale, and their gradients (what each computes:
// include/moe_layer.h).
//
// A workgroup holds one row at a time in registers, 8 elements of a lane's at a
// stride of the workgroup (kVec of them): the statistics, the normed row and
// the residual sum all come from one read.  Row sums go over the wavefront by
// lane permutations, then over the wavefronts in order through LDS; a layer
// norm sums the centred squares in a second pass over the registers, since the
// difference of the two raw moments loses the variance of a row far from zero.
//
// Parameter gradients are sums down the columns: each workgroup keeps those of
// its rows in registers and writes one fp32 row of partial sums; a second
// kernel adds the rows in order, so no atomics and the same result every run.
#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kMaxWaves = 16;

// Sums of kN values over the workgroup's `waves` wavefronts, in every lane.
// buf [kMaxWaves * kN]; consecutive calls alternate between two buffers (a
// wavefront may still read the last call's while another is in the next).
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], int waves, float* buf) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) buf[wave * kN + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float s = lane < waves ? buf[lane * kN + i] : 0.0f;   // (16 lanes at most hold one)
    s = dpp_add<kQuadXor1>(s);
    s = dpp_add<kQuadXor2>(s);
    s = dpp_add<kRowHalfMirror>(s);
    s = dpp_add<kRowMirror>(s);
    v[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), 0));
  }
}

// 8 parameters from p + h, or `none` where there are none
template <class SP>
__device__ __forceinline__ void load_param(const void* p, int h, float none, float* v) {
  if (p) {
    load8f<SP>(static_cast<const typename SP::T*>(p) + h, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
  }
}

// Elements of the row that this lane holds: vector j starts at h(j), in the row
// where h(j) < H.
template <int kVec>
struct Slice {
  int H;
  __device__ int h(int j) const { return ((int)threadIdx.x + j * (int)blockDim.x) * 8; }
  __device__ bool in(int j) const { return h(j) < H; }
};

// Mean (0 for RMS) and 1 / deviation of the row in v (elements past H are 0).
template <int kVec>
__device__ __forceinline__ void row_stats(const float (&v)[kVec][8], const Slice<kVec>& sl,
                                          const NormSpec& n, int waves, float* buf, int& parity,
                                          float& mean, float& rstd) {
  mean = 0.0f;
  if (n.kind == kNormLayer) {
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[j][i];
    block_sum<1>(s, waves, buf + parity * kMaxWaves);
    parity ^= 1;
    mean = s[0] / (float)sl.H;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (sl.in(j)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = v[j][i] - mean;
        q[0] = fmaf(d, d, q[0]);
      }
    }
  block_sum<1>(q, waves, buf + parity * kMaxWaves);
  parity ^= 1;
  rstd = 1.0f / sqrtf(q[0] / (float)sl.H + n.eps);
}

template <class SP, int kVec>
__device__ __forceinline__ void apply_norm(const float (&v)[kVec][8], const Slice<kVec>& sl,
                                           const NormSpec& n, float mean, float rstd, int j,
                                           float* out) {
  float w[8], b[8];
  load_param<SP>(n.weight, sl.h(j), 1.0f, w);
  load_param<SP>(n.bias, sl.h(j), 0.0f, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = fmaf((v[j][i] - mean) * rstd, w[i], b[i]);
}

template <class SX, class SO, class SP, int kVec>
__global__ __launch_bounds__(1024) void norm_kernel(const typename SX::T* x, int64_t T, int H,
                                                    NormSpec n, typename SO::T* out) {
  __shared__ float buf[2 * kMaxWaves];
  const int waves = blockDim.x / kWave;
  const Slice<kVec> sl{H};
  int parity = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (sl.in(j)) load8f<SX>(x + t * H + sl.h(j), v[j]);
    }
    float mean, rstd;
    row_stats<kVec>(v, sl, n, waves, buf, parity, mean, rstd);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (sl.in(j)) {
        float o[8];
        apply_norm<SP, kVec>(v, sl, n, mean, rstd, j, o);
        store8f<SO>(out + t * H + sl.h(j), o);
      }
  }
}

constexpr int kSlots = 4;   // pair rows in flight per lane

// r = x + gate * post(y), n = pre(r).  kCombine: y[t] = sum_k w[t][k] y[t*K + k]
// (+ shared[t]), in slot order as moe_combine sums it.
template <class SY, class SS, class SX, class SP, int kVec, bool kCombine>
__global__ __launch_bounds__(1024) void norm_residual_kernel(
    const typename SY::T* y, const float* __restrict__ w, int K,
    const typename SS::T* __restrict__ shared, const typename SX::T* x, int64_t T, int H,
    NormSpec post, GateSpec gate, typename SX::T* r, NormSpec pre, typename SY::T* n) {
  __shared__ float buf[2 * kMaxWaves];
  const int waves = blockDim.x / kWave;
  const Slice<kVec> sl{H};
  int parity = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[kVec][8], xr[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (!sl.in(j)) continue;
      load8f<SX>(x + t * H + sl.h(j), xr[j]);
      if (!kCombine) load8f<SY>(y + t * H + sl.h(j), v[j]);
    }
    if (kCombine) {
      for (int k0 = 0; k0 < K; k0 += kSlots) {
        float wk[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) wk[k] = k0 + k < K ? w[t * K + k0 + k] : 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (!sl.in(j)) continue;
          float p[kSlots][8];
#pragma unroll
          for (int k = 0; k < kSlots; ++k)
            if (wk[k] != 0.0f) load8f<SY>(y + (t * K + k0 + k) * H + sl.h(j), p[k]);
#pragma unroll
          for (int k = 0; k < kSlots; ++k)
            if (wk[k] != 0.0f) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[j][i] = fmaf(wk[k], p[k][i], v[j][i]);
            }
        }
      }
      if (shared) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (sl.in(j)) {
            float s[8];
            load8f<SS>(shared + t * H + sl.h(j), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += s[i];
          }
      }
    }
    float mean = 0.0f, rstd = 1.0f;
    if (post.kind != kNormNone) row_stats<kVec>(v, sl, post, waves, buf, parity, mean, rstd);
    const float a = gate.token ? gate.alpha * gate.token[t] : gate.alpha;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!sl.in(j)) continue;
      float u[8], c[8];
      if (post.kind != kNormNone) {
        apply_norm<SP, kVec>(v, sl, post, mean, rstd, j, u);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = v[j][i];
      }
      load_param<SP>(gate.channel, sl.h(j), 1.0f, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = fmaf(a * c[i], u[i], xr[j][i]);
      store8f<SX>(r + t * H + sl.h(j), v[j]);
    }
    if (n) {
      row_stats<kVec>(v, sl, pre, waves, buf, parity, mean, rstd);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (sl.in(j)) {
          float o[8];
          apply_norm<SP, kVec>(v, sl, pre, mean, rstd, j, o);
          store8f<SY>(n + t * H + sl.h(j), o);
        }
    }
  }
}

// With xh the normalised x and g = dn * weight:
//   dx = rstd (g - [LAYER] mean(g) - xh mean(g xh)) + dres,
//   dweight = sum_t dn xh, dbias = sum_t dn (partial sums of this workgroup's rows
//   to part_w, part_b [gridDim.x][H], where given).
template <class SO, class SX, class SP, int kVec>
__global__ __launch_bounds__(1024) void norm_backward_kernel(
    const typename SO::T* dn, const typename SX::T* x, const typename SX::T* dres, int64_t T,
    int H, NormSpec n, typename SX::T* dx, float* __restrict__ part_w,
    float* __restrict__ part_b) {
  __shared__ float buf[2 * kMaxWaves * 2];
  const int waves = blockDim.x / kWave;
  const Slice<kVec> sl{H};
  int parity = 0;
  const float inv_h = 1.0f / (float)H;
  float aw[kVec][8], ab[kVec][8];
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[j][i] = ab[j][i] = 0.0f;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[kVec][8], g[kVec][8], d[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = d[j][i] = 0.0f;
      if (!sl.in(j)) continue;
      load8f<SX>(x + t * H + sl.h(j), v[j]);
      load8f<SO>(dn + t * H + sl.h(j), d[j]);
    }
    float mean, rstd;
    row_stats<kVec>(v, sl, n, waves, buf + 2 * kMaxWaves, parity, mean, rstd);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float w[8];
      if (!sl.in(j)) continue;
      load_param<SP>(n.weight, sl.h(j), 1.0f, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = (v[j][i] - mean) * rstd;
        g[j][i] = d[j][i] * w[i];
        s[0] = fmaf(g[j][i], v[j][i], s[0]);
        s[1] += g[j][i];
        aw[j][i] = fmaf(d[j][i], v[j][i], aw[j][i]);
        ab[j][i] += d[j][i];
      }
    }
    block_sum<2>(s, waves, buf);
    const float mgx = s[0] * inv_h, mg = n.kind == kNormLayer ? s[1] * inv_h : 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!sl.in(j)) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (g[j][i] - mg - v[j][i] * mgx);
      if (dres) {
        float e[8];
        load8f<SX>(dres + t * H + sl.h(j), e);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += e[i];
      }
      store8f<SX>(dx + t * H + sl.h(j), o);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (!sl.in(j)) continue;
    if (part_w) store8f<F32>(part_w + (int64_t)blockIdx.x * H + sl.h(j), aw[j]);
    if (part_b) store8f<F32>(part_b + (int64_t)blockIdx.x * H + sl.h(j), ab[j]);
  }
}

// From dr: with u = post(y), a = alpha * token[t] and du = a * channel * dr:
//   dy from du as above (du itself without a norm), dweight, dbias likewise,
//   dchannel = sum_t a dr u,   dtoken[t] = sum_h alpha channel dr u.
template <class SX, class SY, class SP, int kVec>
__global__ __launch_bounds__(1024) void norm_residual_backward_kernel(
    const typename SX::T* dr, const typename SY::T* y, int64_t T, int H, NormSpec n,
    GateSpec gate, typename SY::T* dy, float* __restrict__ part_w, float* __restrict__ part_b,
    float* __restrict__ part_c, float* __restrict__ dtoken) {
  __shared__ float buf[2 * kMaxWaves + kMaxWaves * 3];
  const int waves = blockDim.x / kWave;
  const Slice<kVec> sl{H};
  int parity = 0;
  const float inv_h = 1.0f / (float)H;
  float aw[kVec][8], ab[kVec][8], ac[kVec][8];
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[j][i] = ab[j][i] = ac[j][i] = 0.0f;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[kVec][8], g[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = g[j][i] = 0.0f;
      if (!sl.in(j)) continue;
      load8f<SY>(y + t * H + sl.h(j), v[j]);
      load8f<SX>(dr + t * H + sl.h(j), g[j]);
    }
    float mean = 0.0f, rstd = 1.0f;
    if (n.kind != kNormNone)
      row_stats<kVec>(v, sl, n, waves, buf + 3 * kMaxWaves, parity, mean, rstd);
    const float a = gate.token ? gate.alpha * gate.token[t] : gate.alpha;
    // over the row: sums of g xh and g (without the factor a) and of channel dr u
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!sl.in(j)) continue;
      float w[8], b[8], c[8];
      load_param<SP>(n.weight, sl.h(j), 1.0f, w);
      load_param<SP>(n.bias, sl.h(j), 0.0f, b);
      load_param<SP>(gate.channel, sl.h(j), 1.0f, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (v[j][i] - mean) * rstd;
        const float u = fmaf(xh, w[i], b[i]);
        const float e = g[j][i];
        const float ce = c[i] * e;
        ac[j][i] = fmaf(a * e, u, ac[j][i]);
        aw[j][i] = fmaf(a * ce, xh, aw[j][i]);
        ab[j][i] = fmaf(a, ce, ab[j][i]);
        const float gw = ce * w[i];
        s[0] = fmaf(gw, xh, s[0]);
        s[1] += gw;
        s[2] = fmaf(ce, u, s[2]);
        v[j][i] = xh;
        g[j][i] = gw;
      }
    }
    block_sum<3>(s, waves, buf);
    if (dtoken && threadIdx.x == 0) dtoken[t] = gate.alpha * s[2];
    const float mgx = n.kind != kNormNone ? s[0] * inv_h : 0.0f;
    const float mg = n.kind == kNormLayer ? s[1] * inv_h : 0.0f;
    const float ar = a * rstd;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!sl.in(j)) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = ar * (g[j][i] - mg - v[j][i] * mgx);
      store8f<SY>(dy + t * H + sl.h(j), o);
    }
    __syncthreads();   // buf is written again by the next row's sums
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (!sl.in(j)) continue;
    const int64_t o = (int64_t)blockIdx.x * H + sl.h(j);
    if (part_w) store8f<F32>(part_w + o, aw[j]);
    if (part_b) store8f<F32>(part_b + o, ab[j]);
    if (part_c) store8f<F32>(part_c + o, ac[j]);
  }
}

// out[i][h] = sum over g < G, in order, of part[i][g][h]; zeros for G = 0.
// 16 lanes hold 64 columns, 16 groups of them G / 16 rows each.
struct ColumnSums {
  const float* part[3];
  float* out[3];
};
__global__ __launch_bounds__(256) void column_sum_kernel(ColumnSums c, int G, int H) {
  __shared__ f32x4 buf[16][16];
  const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int h = blockIdx.x * 64 + lane * 4;
  const float* part = c.part[blockIdx.y];
  float* out = c.out[blockIdx.y];
  const int per = (G + 15) / 16;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (h < H)
    for (int g = grp * per; g < G && g < (grp + 1) * per; ++g)
      s += *reinterpret_cast<const f32x4*>(part + (int64_t)g * H + h);
  buf[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && h < H) {
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = 0; g < 16; ++g) o += buf[g][lane];
    *reinterpret_cast<f32x4*>(out + h) = o;
  }
}

namespace {

struct Launch {
  int vec, threads;
};

// Vectors of 8 elements a lane holds (1 up to 8192 elements, where 1024 lanes
// cover the row) and the lanes.
Launch launch_for(int H, int vec) {
  const int nv = H / 8;
  if (nv > kMaxWaves * kWave) vec = 2;
  const int lanes = (nv + vec - 1) / vec;
  return {vec, (lanes + kWave - 1) / kWave * kWave};
}

// Workgroups of a backward launch: each writes a row of partial sums per
// parameter, so it takes 16 rows or more once there are 256 of them.
int backward_groups(int64_t T, int H) {
  const int waves = launch_for(H, 2).threads / kWave;
  int64_t g = T / 16;
  const int64_t most = 256 * (waves < 16 ? 16 / waves : 1);
  if (g > most) g = most;
  if (g < 256) g = 256;
  return (int)(g < T ? g : T);
}

unsigned rows_grid(int64_t T) { return (unsigned)(T < (1 << 20) ? T : (1 << 20)); }

template <class F>
hipError_t with_types(int a, int b, int c, F f) {
  auto third = [&](auto sa, auto sb) {
    if (c == kDtF32) f(sa, sb, F32());
    else f(sa, sb, BF16());
  };
  auto second = [&](auto sa) {
    if (b == kDtF32) third(sa, F32());
    else third(sa, BF16());
  };
  if (a == kDtF32) second(F32());
  else second(BF16());
  return hipGetLastError();
}

hipError_t column_sums(const ColumnSums& c, int n, int G, int H, hipStream_t s) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(column_sum_kernel, dim3((H + 63) / 64, n), dim3(256), 0, s, c, G, H);
  return hipGetLastError();
}

// The partial sums of the gradients asked for (out[i] not null), in `workspace`.
struct Partials {
  ColumnSums sums;
  int n;
  float* part[3];
  Partials(float* const* out, int count, float* workspace, int G, int H) : n(0) {
    for (int i = 0; i < count; ++i) {
      part[i] = out[i] ? workspace + (int64_t)n * G * H : nullptr;
      if (out[i]) {
        sums.part[n] = part[i];
        sums.out[n++] = out[i];
      }
    }
  }
};

}  // namespace

int64_t norm_workspace_floats(int64_t T, int H) {
  return 3 * (int64_t)backward_groups(T, H) * H;
}

hipError_t launch_norm(const void* x, int xdt, int64_t T, int H, const NormSpec& n, int pdt,
                       void* out, int odt, hipStream_t s) {
  const Launch l = launch_for(H, 1);
  return with_types(xdt, odt, pdt, [&](auto sx, auto so, auto sp) {
    typedef decltype(sx) SX;
    typedef decltype(so) SO;
    typedef decltype(sp) SP;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(rows_grid(T)), dim3(l.threads), 0, s,
                         static_cast<const typename SX::T*>(x), T, H, n,
                         static_cast<typename SO::T*>(out));
    };
    if (l.vec == 1) go(norm_kernel<SX, SO, SP, 1>);
    else go(norm_kernel<SX, SO, SP, 2>);
  });
}

hipError_t launch_norm_residual(const void* y, int ydt, const void* x, int xdt, int64_t T, int H,
                                const NormSpec& post, const GateSpec& gate, int pdt, void* r,
                                const NormSpec& pre, void* n, hipStream_t s) {
  const Launch l = launch_for(H, 1);
  return with_types(ydt, xdt, pdt, [&](auto sy, auto sx, auto sp) {
    typedef decltype(sy) SY;
    typedef decltype(sx) SX;
    typedef decltype(sp) SP;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(rows_grid(T)), dim3(l.threads), 0, s,
                         static_cast<const typename SY::T*>(y), nullptr, 0, nullptr,
                         static_cast<const typename SX::T*>(x), T, H, post, gate,
                         static_cast<typename SX::T*>(r), pre, static_cast<typename SY::T*>(n));
    };
    if (l.vec == 1) go(norm_residual_kernel<SY, SY, SX, SP, 1, false>);
    else go(norm_residual_kernel<SY, SY, SX, SP, 2, false>);
  });
}

hipError_t launch_combine_norm_residual(const void* y, int ydt, const float* w, int K,
                                        const void* shared, int sdt, const void* x, int xdt,
                                        int64_t T, int H, const NormSpec& post,
                                        const GateSpec& gate, int pdt, void* r,
                                        const NormSpec& pre, void* n, hipStream_t s) {
  const Launch l = launch_for(H, 1);
  return with_types(ydt, xdt, pdt, [&](auto sy, auto sx, auto sp) {
    typedef decltype(sy) SY;
    typedef decltype(sx) SX;
    typedef decltype(sp) SP;
    auto shared_type = [&](auto ss) {
      typedef decltype(ss) SS;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(rows_grid(T)), dim3(l.threads), 0, s,
                           static_cast<const typename SY::T*>(y), w, K,
                           static_cast<const typename SS::T*>(shared),
                           static_cast<const typename SX::T*>(x), T, H, post, gate,
                           static_cast<typename SX::T*>(r), pre, static_cast<typename SY::T*>(n));
      };
      if (l.vec == 1) go(norm_residual_kernel<SY, SS, SX, SP, 1, true>);
      else go(norm_residual_kernel<SY, SS, SX, SP, 2, true>);
    };
    if (sdt == kDtF32) shared_type(F32());
    else shared_type(BF16());
  });
}

hipError_t launch_norm_backward(const void* dn, int odt, const void* x, int xdt, const void* dres,
                                int64_t T, int H, const NormSpec& n, int pdt, void* dx,
                                float* dweight, float* dbias, float* workspace, hipStream_t s) {
  const Launch l = launch_for(H, 2);
  const int G = backward_groups(T, H);
  float* const out[2] = {dweight, dbias};
  const Partials p(out, 2, workspace, G, H);
  if (T > 0) {
    const hipError_t e = with_types(odt, xdt, pdt, [&](auto so, auto sx, auto sp) {
      typedef decltype(so) SO;
      typedef decltype(sx) SX;
      typedef decltype(sp) SP;
      hipLaunchKernelGGL((norm_backward_kernel<SO, SX, SP, 2>), dim3(G), dim3(l.threads), 0, s,
                         static_cast<const typename SO::T*>(dn),
                         static_cast<const typename SX::T*>(x),
                         static_cast<const typename SX::T*>(dres), T, H, n,
                         static_cast<typename SX::T*>(dx), p.part[0], p.part[1]);
    });
    if (e != hipSuccess) return e;
  }
  return column_sums(p.sums, p.n, G, H, s);
}

hipError_t launch_norm_residual_backward(const void* dr, int xdt, const void* y, int ydt,
                                         int64_t T, int H, const NormSpec& post,
                                         const GateSpec& gate, int pdt, void* dy, float* dweight,
                                         float* dbias, float* dchannel, float* dtoken,
                                         float* workspace, hipStream_t s) {
  const Launch l = launch_for(H, 2);
  const int G = backward_groups(T, H);
  float* const out[3] = {dweight, dbias, dchannel};
  const Partials p(out, 3, workspace, G, H);
  if (T > 0) {
    const hipError_t e = with_types(xdt, ydt, pdt, [&](auto sx, auto sy, auto sp) {
      typedef decltype(sx) SX;
      typedef decltype(sy) SY;
      typedef decltype(sp) SP;
      hipLaunchKernelGGL((norm_residual_backward_kernel<SX, SY, SP, 2>), dim3(G),
                         dim3(l.threads), 0, s, static_cast<const typename SX::T*>(dr),
                         static_cast<const typename SY::T*>(y), T, H, post, gate,
                         static_cast<typename SY::T*>(dy), p.part[0], p.part[1], p.part[2],
                         dtoken);
    });
    if (e != hipSuccess) return e;
  }
  return column_sums(p.sums, p.n, G, H, s);
}

}  // namespace moe
