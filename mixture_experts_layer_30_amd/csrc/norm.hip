// The norms before and after a block of a residual stream, with the block's
// gate and residual scale, and their gradients (what each computes:
// include/moe_layer.h).
//
// All of it is bound by memory.  A workgroup holds one row at a time in
// registers, so that the statistics, the normed row, the residual sum and the
// next norm come from one read, and asks for its next row before it works on
// this one.  Row sums go over the wavefront by lane permutations, then over the
// wavefronts in order through LDS.  A layer norm takes a second pass over the
// registers: an fp32 mean m of a row far from zero is off by a few units in its last
// place, so the mean d of x - m is summed next to the squares of x - m (one more
// addition an element), and x - m - d, mean((x - m)^2) - d^2 are used.  What is left
// of the error goes by the row's deviation and no longer by its mean.
//
// Rows are read and written through buffer descriptors of the row's length: a
// lane past its end reads zeros and writes nothing, and a row that is not there
// (no bias, a slot of weight 0) has length 0, so the kernels have no branches
// around their loads and address rows from scalar registers.
//
// Parameter gradients are sums down the columns: each workgroup keeps those of
// its rows in registers and writes one fp32 row of partial sums; a second
// kernel adds the rows in order, so no atomics and the same result every run.
//
// Measured on MI355X, inputs that no cache holds (a copy of 1 GB runs at 5.1 TB/s):
// RMS norm of 16384 x 4096 bf16 46 us (5.8 TB/s), layer norm 48, gated residual on an
// fp32 stream with the next layer norm at the same size 134-140 us (5.8-6.0 TB/s), RMS
// norm gradients of 8192 x 7168 with a gradient that passes by 92 us (5.1 TB/s; both
// launches), layer norm's of 4099 x 3584 with all gates 25 us (3.5 TB/s, vector
// instructions as much as memory), the end of a layer pass, combine to next norm, of
// 128 x 7168 with 8 pair rows a token 7 us (8192 tokens 214 us, 6.0 TB/s).  Rows past
// 8192 elements: forward 5.2-5.9 TB/s, gradients 3.2-5.2.  The pairs of times at the
// choices below are of builds that differ in that choice alone, the layer norms' from
// before the second pass over the mean, which costs them 0-5%.
#include "block_kernels.h"
#include "common.h"
#include "rows.h"

namespace moe {

constexpr int kMaxWaves = 16;

typedef __amdgpu_buffer_rsrc_t Row;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Row t of the rows of `bytes` bytes at p (raw 32-bit elements, range checked);
// a row that is not there where p is null.
__device__ __forceinline__ Row row_at(const void* p, int64_t t, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(static_cast<const char*>(p) + t * (int64_t)bytes), 0, p ? bytes : 0,
      0x00020000);
}

// Cache policy of a load or store: 2 is non-temporal.  Results are stored so: they
// take no room from rows that are still to be read (RMS norm of 2048 x 4096 7.8 ->
// 6.2 us, the gated residual of 16384 x 1024 28 -> 23; a product that reads the
// result next runs at the same speed).  Pair rows, read once, are loaded so too
// (2048 tokens of 3584, 8 pair rows each: 37 -> 34 us); other rows are not (loading
// them so costs the same two 10-20%).
constexpr int kCached = 0, kStreamed = 2;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {   // v_cvt_pk_bf16_f32
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// N (4 or 8) consecutive elements as they are in memory, converted when they are
// used, four at a time: a load in flight is waited for where its values are
// needed, and the values that stay live are the shorter ones.
template <class S, int N>
struct Raw;
template <int N>
struct Raw<BF16, N> {
  uint32_t q[N / 2];
  template <int kPolicy>
  __device__ __forceinline__ void load(Row r, uint32_t h) {
    if constexpr (N == 8) {
      const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(r, h * 2, 0, kPolicy);
      q[0] = a.x; q[1] = a.y; q[2] = a.z; q[3] = a.w;
    } else {
      const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(r, h * 2, 0, kPolicy);
      q[0] = a.x; q[1] = a.y;
    }
  }
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) q[j] = pack2(f, f);
  }
  __device__ __forceinline__ void get4(int j, float* v) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(q[2 * j + i] << 16);
      v[2 * i + 1] = __uint_as_float(q[2 * j + i] & 0xffff0000u);
    }
  }
  // The values are converted anew after this, not kept in twice the registers.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) asm volatile("" : "+v"(q[j]));
  }
};
template <int N>
struct Raw<F32, N> {
  u32x4 q[N / 4];
  template <int kPolicy>
  __device__ __forceinline__ void load(Row r, uint32_t h) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      q[j] = __builtin_amdgcn_raw_buffer_load_b128(r, h * 4 + 16 * j, 0, kPolicy);
  }
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) q[j] = __builtin_bit_cast(u32x4, f32x4{f, f, f, f});
  }
  __device__ __forceinline__ void get4(int j, float* v) const {
    const f32x4 a = __builtin_bit_cast(f32x4, q[j]);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  __device__ __forceinline__ void keep() {}
};

template <class S, int N, int kPolicy>
__device__ __forceinline__ void put(Row r, uint32_t h, const float* v) {
  if constexpr (S::kBytes == 4) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(u32x4, f32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]}), r,
          h * 4 + 16 * j, 0, kPolicy);
  } else if constexpr (N == 8) {
    __builtin_amdgcn_raw_buffer_store_b128(
        u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])}, r,
        h * 2, 0, kPolicy);
  } else {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, r, h * 2, 0,
                                          kPolicy);
  }
}

// What a lane, one of `lanes`, holds of a row: kV vectors of kN elements, `lanes`
// vectors apart; vector j starts at h(j).
template <int kN, int kV>
struct Slice {
  static constexpr int N = kN, V = kV;
  uint32_t H, lane, lanes;
  __device__ __forceinline__ uint32_t h(int j) const { return (lane + j * lanes) * N; }
  __device__ __forceinline__ bool in(int j) const { return h(j) < H; }
};

// A lane's elements of a row, or of a parameter.
template <class S, class L>
struct Part {
  Raw<S, L::N> q[L::V];
  template <int kPolicy>
  __device__ __forceinline__ void load(Row r, const L& sl) {
#pragma unroll
    for (int j = 0; j < L::V; ++j) q[j].template load<kPolicy>(r, sl.h(j));
  }
  // Parameter p, or `none` for each element where there is none.
  __device__ __forceinline__ void param(const void* p, float none, const L& sl) {
    load<kCached>(row_at(p, 0, sl.H * S::kBytes), sl);
    if (!p && none != 0.0f) {
#pragma unroll
      for (int j = 0; j < L::V; ++j) q[j].fill(none);
    }
  }
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int j = 0; j < L::V; ++j) q[j].keep();
  }
};

// f(j, q) for every group of four elements that a lane holds.
template <class L, class F>
__device__ __forceinline__ void each4(F f) {
#pragma unroll
  for (int j = 0; j < L::V; ++j)
#pragma unroll
    for (int q = 0; q < L::N / 4; ++q) f(j, q);
}

// Sums over each row of 16 lanes, in every lane of it: a step of all kN at a time, since
// one that takes the step before's result has to wait two cycles for it.
template <int kN>
__device__ __forceinline__ void lane_row_sums(float (&v)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = dpp_add<kQuadXor1>(v[i]);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = dpp_add<kQuadXor2>(v[i]);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = dpp_add<kRowHalfMirror>(v[i]);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = dpp_add<kRowMirror>(v[i]);
}

// v, the same in every lane, in a scalar register.
__device__ __forceinline__ float scalar(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}

__device__ __forceinline__ float at_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Buffers of block_sum, two taken in turn (a wavefront may still read the last call's
// while another is in the next).
template <int kN>
struct SumBuffers {
  f32x4 (*buf)[kN * kMaxWaves];
  int next;
  __device__ __forceinline__ f32x4* take() {
    next ^= 1;
    return buf[next];
  }
};

// Sums of kN <= 4 values over the row's `waves` wavefronts, the workgroup's from
// `first` on, in every lane.  Each row of 16 lanes leaves its sums in buf, four of a
// wavefront together; every wavefront then adds up its part of them, value i's on its
// lanes 16 i .. 16 i + 15.  (Sums of whole wavefronts first take six instructions more
// a value.)
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], int waves, f32x4* buf, int first = 0) {
  const int lane = threadIdx.x & (kWave - 1);
  lane_row_sums(v);
  if (waves == 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      v[i] = scalar((at_lane(v[i], 0) + at_lane(v[i], 16)) +
                    (at_lane(v[i], 32) + at_lane(v[i], 48)));
    return;
  }
  if (lane % 16 == 0) {
    float* p = reinterpret_cast<float*>(buf) + threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < kN; ++i) p[i * kMaxWaves * 4] = v[i];
  }
  __syncthreads();
  const uint32_t col = (uint32_t)(lane % kMaxWaves - first);
  f32x4 q = {0.0f, 0.0f, 0.0f, 0.0f};
  if (lane < kN * kMaxWaves && col < (uint32_t)waves) q = buf[lane];
  float s[1] = {(q[0] + q[1]) + (q[2] + q[3])};
  lane_row_sums(s);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = at_lane(s[0], i * kMaxWaves);
}

// 1 / deviation, from the mean of the squares of a row less an approximate mean, and the
// mean that those still have.
__device__ __forceinline__ float rstd_of(float squares, float inv_h, float eps, float rest) {
  const float v = fmaf(-rest, rest, fmaf(squares, inv_h, eps));
  return rsqrtf(v < eps ? eps : v);   // (a NaN stays)
}

// 1 / deviation of the row in v, whose elements past the end are 0; for a layer
// norm the row's mean is taken from it first.
template <class L>
__device__ __forceinline__ float center_and_rstd(float (&v)[L::V][L::N], const L& sl, int kind,
                                                 float eps, float inv_h, int waves,
                                                 SumBuffers<2>& buf) {
  auto sum = [&] {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < L::V; ++j)
#pragma unroll
      for (int i = 0; i < L::N; ++i) m += v[j][i];
    return m;
  };
  auto squares = [&] {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < L::V; ++j)
#pragma unroll
      for (int i = 0; i < L::N; ++i) s = fmaf(v[j][i], v[j][i], s);
    return s;
  };
  auto take = [&](float mean) {
#pragma unroll
    for (int j = 0; j < L::V; ++j) {
      const float c = sl.in(j) ? mean : 0.0f;
#pragma unroll
      for (int i = 0; i < L::N; ++i) v[j][i] -= c;
    }
  };
  if (kind == kNormLayer) {
    float m[1] = {sum()};
    block_sum<1>(m, waves, buf.take());
    take(m[0] * inv_h);
    float s[2] = {squares(), sum()};
    block_sum<2>(s, waves, buf.take());
    const float rest = s[1] * inv_h;
    const float rstd = rstd_of(s[0], inv_h, eps, rest);
    take(rest);
    return rstd;
  }
  float s[1] = {squares()};
  block_sum<1>(s, waves, buf.take());
  return rstd_of(s[0], inv_h, eps, 0.0f);
}

// v = v * rstd * weight + bias, element by element; `bias` as the norm has it, kHeld:
// loaded already, in pb.
template <bool kHeld, class SP, class L>
__device__ __forceinline__ void scale_and_shift(float (&v)[L::V][L::N], const L& sl, float rstd,
                                                const Part<SP, L>& weight, const void* bias,
                                                Part<SP, L>& pb) {
  if (bias) {
    if (kHeld) pb.keep();
    else pb.param(bias, 0.0f, sl);
    each4<L>([&](int j, int q) {
      float w[4], b[4];
      weight.q[j].get4(q, w);
      pb.q[j].get4(q, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][4 * q + i] = fmaf(v[j][4 * q + i] * rstd, w[i], b[i]);
    });
  } else {
    each4<L>([&](int j, int q) {
      float w[4];
      weight.q[j].get4(q, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][4 * q + i] *= rstd * w[i];
    });
  }
}

template <class S, class L>
__device__ __forceinline__ void put_row(void* p, int64_t t, const L& sl,
                                        const float (&v)[L::V][L::N]) {
  const Row r = row_at(p, t, sl.H * S::kBytes);
#pragma unroll
  for (int j = 0; j < L::V; ++j) put<S, L::N, kStreamed>(r, sl.h(j), v[j]);
}

template <class SX, class SO, class SP, class L, bool kHeld>
__global__ __launch_bounds__(1024) void norm_kernel(const void* x, int64_t T, int H, NormSpec n,
                                                    void* out) {
  __shared__ f32x4 sums[2][2 * kMaxWaves];
  SumBuffers<2> buf{sums, 0};
  const int waves = blockDim.x / kWave;
  const L sl{(uint32_t)H, threadIdx.x, blockDim.x};
  const uint32_t xb = H * SX::kBytes;
  const float inv_h = 1.0f / (float)H;
  Part<SX, L> rx;
  Part<SP, L> pw, pb;
  rx.template load<kCached>(row_at(x, blockIdx.x, xb), sl);
  pw.param(n.weight, 1.0f, sl);
  if (kHeld) pb.param(n.bias, 0.0f, sl);
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[L::V][L::N];
    each4<L>([&](int j, int q) { rx.q[j].get4(q, &v[j][4 * q]); });
    if (t + gridDim.x < T) rx.template load<kCached>(row_at(x, t + gridDim.x, xb), sl);
    pw.keep();
    const float rstd = center_and_rstd(v, sl, n.kind, n.eps, inv_h, waves, buf);
    scale_and_shift<kHeld>(v, sl, rstd, pw, n.bias, pb);
    put_row<SO>(out, t, sl, v);
  }
}

// r = x + gate * post(y), n = pre(r).  kCombine: y[t] = sum_k w[t][k] y[t*K + k]
// (+ shared[t]), in slot order as moe_combine sums it.  kHeld: biases, channel and the
// token's gate are loaded ahead of the next row, where otherwise a load in the row's
// turn, issued after the next row's loads, waits for those too.
template <class SY, class SS, class SX, class SP, class L, bool kCombine, bool kHeld>
__global__ __launch_bounds__(1024) void norm_residual_kernel(
    const void* y, const float* __restrict__ w, int K, const void* shared, const void* x,
    int64_t T, int H, NormSpec post, GateSpec gate, void* r, NormSpec pre, void* n) {
  constexpr int N = L::N, V = L::V;
  __shared__ f32x4 sums[2][2 * kMaxWaves];
  SumBuffers<2> buf{sums, 0};
  const int waves = blockDim.x / kWave;
  const L sl{(uint32_t)H, threadIdx.x, blockDim.x};
  const uint32_t xb = H * SX::kBytes, yb = H * SY::kBytes, sb = H * SS::kBytes;
  const float inv_h = 1.0f / (float)H;
  Part<SX, L> rx;
  Part<SY, L> ry;
  Part<SP, L> pw, qw, pb, pc, qb;
  float token = 0.0f;
  auto fetch_token = [&](int64_t t) {
    if (kHeld && gate.token)
      token = __int_as_float(
          __builtin_amdgcn_raw_buffer_load_b32(row_at(gate.token, t, 4), 0, 0, kCached));
  };
  if (!kCombine) {
    fetch_token(blockIdx.x);
    rx.template load<kCached>(row_at(x, blockIdx.x, xb), sl);
    ry.template load<kCached>(row_at(y, blockIdx.x, yb), sl);
  }
  pw.param(post.weight, 1.0f, sl);
  qw.param(pre.weight, 1.0f, sl);
  if (kHeld) {
    pb.param(post.bias, 0.0f, sl);
    pc.param(gate.channel, 1.0f, sl);
    qb.param(pre.bias, 0.0f, sl);
  }
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[V][N], g = 1.0f;
    Part<SX, L> cx;
    if constexpr (kCombine) {
      // pair rows in flight: 64 bytes a lane
      constexpr int kSlots = N * V * SY::kBytes <= 16 ? 4 : N * V * SY::kBytes <= 32 ? 2 : 1;
      Part<SS, L> rs;
      fetch_token(t);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) v[j][i] = 0.0f;
      for (int k0 = 0; k0 < K; k0 += kSlots) {
        Part<SY, L> p[kSlots];
        float wk[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) wk[k] = k0 + k < K ? w[t * K + k0 + k] : 0.0f;
        // (a slot of weight 0: a row of no bytes, which reads zeros)
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
          p[k].template load<kStreamed>(
              wk[k] != 0.0f ? row_at(y, t * K + k0 + k, yb) : row_at(nullptr, 0, 0), sl);
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
          each4<L>([&](int j, int q) {
            float e[4];
            p[k].q[j].get4(q, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][4 * q + i] = fmaf(wk[k], e[i], v[j][4 * q + i]);
          });
      }
      rs.template load<kCached>(row_at(shared, t, sb), sl);
      cx.template load<kCached>(row_at(x, t, xb), sl);
      if (shared)
        each4<L>([&](int j, int q) {
          float e[4];
          rs.q[j].get4(q, e);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][4 * q + i] += e[i];
        });
    } else {
      cx = rx;
      g = token;
      each4<L>([&](int j, int q) { ry.q[j].get4(q, &v[j][4 * q]); });
      if (t + gridDim.x < T) {
        fetch_token(t + gridDim.x);
        rx.template load<kCached>(row_at(x, t + gridDim.x, xb), sl);
        ry.template load<kCached>(row_at(y, t + gridDim.x, yb), sl);
      }
    }
    pw.keep();
    qw.keep();
    const float rstd =
        post.kind != kNormNone
            ? center_and_rstd(v, sl, post.kind, post.eps, inv_h, waves, buf)
            : 1.0f;
    const float a =
        gate.token ? gate.alpha * (!kHeld ? gate.token[t] : kCombine ? token : g) : gate.alpha;
    if (post.bias || gate.channel) {
      if (kHeld) {
        pb.keep();
        pc.keep();
      } else {
        pb.param(post.bias, 0.0f, sl);
        pc.param(gate.channel, 1.0f, sl);
      }
      each4<L>([&](int j, int q) {
        float w4[4], b4[4], c4[4], x4[4];
        pw.q[j].get4(q, w4);
        pb.q[j].get4(q, b4);
        pc.q[j].get4(q, c4);
        cx.q[j].get4(q, x4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& e = v[j][4 * q + i];
          e = fmaf(a * c4[i], fmaf(e * rstd, w4[i], b4[i]), x4[i]);
        }
      });
    } else {
      const float ar = a * rstd;
      each4<L>([&](int j, int q) {
        float w4[4], x4[4];
        pw.q[j].get4(q, w4);
        cx.q[j].get4(q, x4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][4 * q + i] = fmaf(v[j][4 * q + i] * ar, w4[i], x4[i]);
      });
    }
    put_row<SX>(r, t, sl, v);
    if (n) {
      const float rstd2 = center_and_rstd(v, sl, pre.kind, pre.eps, inv_h, waves, buf);
      scale_and_shift<kHeld>(v, sl, rstd2, qw, pre.bias, qb);
      put_row<SY>(n, t, sl, v);
    }
  }
}

// Gradients of v -> gate * norm(v) and of its parameters, from the gradient e of
// the result: with a = alpha * token[t], f = channel * weight, xh the normalised
// row and g = f e,
//   dv = a rstd (g - [LAYER] mean(g) - xh mean(g xh)) (+ dres),
//   dtoken[t] = alpha sum_h e channel (xh weight + bias)
//             = alpha (sum_h g xh + sum_h e channel bias),
// and down the columns only two sums are needed,
//   S1 = sum_t a e xh,  S0 = sum_t a e:
//   dweight = channel S1,  dbias = channel S0,  dchannel = weight S1 + bias S0.
// A workgroup takes `rows` rows at a time, each on `waves` wavefronts, and adds their
// sums up at the end; the partial sums go to part1, part0 [gridDim.x][H] where given.
// One reduction a row; a layer norm has one before it, of the row and the sums that do
// not need its mean, and the second's are of the centred row and then of what is left of
// its mean.  The norm before a block is the case without gates, with dres.
template <class SE, class SV, class SP, class L, bool kDres, bool kSum0>
__global__ __launch_bounds__(1024) void norm_backward_kernel(
    const void* e, const void* v, const void* dres, int64_t T, int H, int waves, int rows,
    NormSpec n, GateSpec gate, void* dv, float* part1, float* part0, float* __restrict__ dtoken) {
  constexpr int N = L::N, V = L::V;
  __shared__ f32x4 sums[2][kMaxWaves * 3];
  SumBuffers<3> buf{sums, 0};
  extern __shared__ f32x4 staged[];
  // the row of the workgroup's `rows` at a time that this wavefront works on
  const int row = rows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWave / waves) : 0;
  const int first = row * waves;
  const L sl{(uint32_t)H, threadIdx.x - first * kWave, (uint32_t)waves * kWave};
  const int64_t step = (int64_t)gridDim.x * rows;
  const uint32_t vb = H * SV::kBytes, eb = H * SE::kBytes;
  const float inv_h = 1.0f / (float)H;
  const bool layer = n.kind == kNormLayer;
  const bool bias_sum = dtoken && n.bias;
  // 16 elements a lane leave no registers for the next row's, and none for a row as fp32
  // values, which are converted anew at each use there (8 elements: 4099 x 3584, layer
  // norm, all gates, 26.1 us then, 24.1 held; the arithmetic is as much as the loads).
  constexpr bool kAhead = N * V <= 8;
  // channel bias, which every row of a token gradient takes: loaded with each row 31.4
  // us instead of 28.7 (4099 x 3584, layer norm, all gates)
  constexpr bool kHeld = kSum0 && kAhead;
  float s1[V][N], s0[kSum0 ? V : 1][N], f[V][N], cb[kHeld ? V : 1][N];
  Part<SV, L> rv, rr;
  Part<SE, L> re;
  // (rows past the last: of no bytes, they read zeros and store nothing)
  auto at = [&](const void* p, int64_t t, uint32_t bytes) {
    return t < T ? row_at(p, t, bytes) : row_at(nullptr, 0, 0);
  };
  // The token's gate comes with the row: loaded after the next row's loads, it waits
  // for them (8192 x 3584, layer norm, all gates, 45.2 us instead of 43.1).
  float token = 0.0f;
  auto fetch = [&](int64_t t) {
    if (gate.token)
      token = __int_as_float(
          __builtin_amdgcn_raw_buffer_load_b32(at(gate.token, t, 4), 0, 0, kCached));
    rv.template load<kCached>(at(v, t, vb), sl);
    re.template load<kCached>(at(e, t, eb), sl);
    if (kDres) rr.template load<kCached>(at(dres, t, vb), sl);
  };
  if (kAhead) fetch((int64_t)blockIdx.x * rows + row);
  {
    Part<SP, L> pw, pb, pc;
    pw.param(n.weight, 1.0f, sl);
    if (kHeld) pb.param(n.bias, 0.0f, sl);
    pc.param(gate.channel, 1.0f, sl);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        float w[4], b[4], c[4];
        pw.q[j].get4(q, w);
        if (kHeld) pb.q[j].get4(q, b);
        pc.q[j].get4(q, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kHeld) cb[j][4 * q + i] = c[i] * b[i];
          f[j][4 * q + i] = w[i] * c[i];
          s1[j][4 * q + i] = 0.0f;
          if (kSum0) s0[j][4 * q + i] = 0.0f;
        }
      }
  }
  // vmcnt(0), once: with loads from before the loop still open, the wait for a row in
  // the loop has to cover both ways into it, and takes the last row's stores too (that
  // size 51.9 us instead of 43.7).
  __builtin_amdgcn_s_waitcnt(0x0F70);
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < T; t0 += step) {
    const int64_t t = t0 + row;
    const bool live = t < T;
    if (!kAhead) fetch(t);
    Part<SV, L> cv = rv, cr = rr;
    Part<SE, L> ce = re;
    const float a = !live ? 0.0f : gate.token ? gate.alpha * token : gate.alpha;
    if (kAhead && t0 + step < T) fetch(t + step);
    float eb = 0.0f;   // sum of e channel bias
    if (bias_sum && kHeld) {
      each4<L>([&](int j, int q) {
        float d[4];
        ce.q[j].get4(q, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) eb = fmaf(d[i], cb[j][4 * q + i], eb);
      });
    } else if (bias_sum) {
      Part<SP, L> pb, pc;
      pb.param(n.bias, 0.0f, sl);
      pc.param(gate.channel, 1.0f, sl);
      each4<L>([&](int j, int q) {
        float b[4], c[4], d[4];
        pb.q[j].get4(q, b);
        pc.q[j].get4(q, c);
        ce.q[j].get4(q, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) eb = fmaf(d[i], c[i] * b[i], eb);
      });
    }
    float mean = 0.0f, g_sum = 0.0f;
    if (layer) {
      // of the row, g, and e channel bias
      float m[3] = {0.0f, 0.0f, eb};
      each4<L>([&](int j, int q) {
        float x[4], d[4];
        cv.q[j].get4(q, x);
        ce.q[j].get4(q, d);
        m[0] += (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) m[1] = fmaf(d[i], f[j][4 * q + i], m[1]);
      });
      if (!kAhead) cv.keep();
      if (!kAhead) ce.keep();
      block_sum<3>(m, waves, buf.take(), first);
      mean = m[0] * inv_h;
      g_sum = m[1];
      eb = m[2];
    }
    // of the centred squares, g times the centred row, and what the centred row still sums
    // to, or e channel bias where the row is not centred
    float s[3] = {0.0f, 0.0f, layer ? 0.0f : eb};
    float held[kAhead ? V : 1][N];   // the centred row
    each4<L>([&](int j, int q) {
      float x[4], d[4];
      cv.q[j].get4(q, x);
      ce.q[j].get4(q, d);
      if (layer) {
        const float c = sl.in(j) ? mean : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] -= c;
        s[2] += (x[0] + x[1]) + (x[2] + x[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[0] = fmaf(x[i], x[i], s[0]);
        s[1] = fmaf(d[i] * f[j][4 * q + i], x[i], s[1]);
        if (kAhead) held[j][4 * q + i] = x[i];
      }
    });
    if (!kAhead) cv.keep();
    if (!kAhead) ce.keep();
    block_sum<3>(s, waves, buf.take(), first);
    float rest = 0.0f;
    if (layer) {
      rest = s[2] * inv_h;
      s[1] = fmaf(-rest, g_sum, s[1]);
    } else {
      eb = s[2];
    }
    const float rstd = n.kind == kNormNone ? 1.0f : live ? rstd_of(s[0], inv_h, n.eps, rest) : 0.0f;
    if (dtoken && live && sl.lane == 0) dtoken[t] = gate.alpha * fmaf(s[1], rstd, eb);
    // dv = (ar e) f - ag - ((x - mean - rest) rstd) agx  (rstd by itself: its cube overflows
    // for rows as small as 1e-13)
    const float ar = a * rstd;
    const float agx = n.kind != kNormNone ? ar * (rstd * (s[1] * inv_h)) : 0.0f;
    const float ag = layer ? ar * (g_sum * inv_h) : 0.0f;
    // (below four roundings of a normed value of 1 it is not worth the subtractions: layer
    // norm of 8192 x 7168 78 us, with them in every row 81)
    if constexpr (kAhead)
      if (layer && !(fabsf(rest * rstd) <= 0x1p-22f)) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) held[j][i] -= rest;
      }
    const Row out = at(dv, t, vb);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float o[N];
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        float x[4], d[4];
        if constexpr (kAhead) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = held[j][4 * q + i];
        } else {
          cv.q[j].get4(q, x);
          if (layer) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (x[i] - mean) - rest;
          }
        }
        ce.q[j].get4(q, d);
        float* oq = o + 4 * q;
        if (kDres) {
          cr.q[j].get4(q, oq);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) oq[i] = 0.0f;
        }
        if (layer) {
#pragma unroll
          for (int i = 0; i < 4; ++i) oq[i] -= ag;
        }
        if (kSum0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s0[j][4 * q + i] = fmaf(a, d[i], s0[j][4 * q + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 4 * q + i;
          const float er = ar * d[i];
          s1[j][k] = fmaf(er, x[i], s1[j][k]);
          oq[i] = fmaf(er, f[j][k], fmaf(-agx, x[i] * rstd, oq[i]));
        }
      }
      put<SV, N, kStreamed>(out, sl.h(j), o);
    }
  }
  // The rows' sums into those of the first: its wavefronts add the others' in order.
  auto join = [&](float (&s)[V][N]) {
    if (row > 0)
      each4<L>([&](int j, int q) {
        const float* p = &s[j][4 * q];
        staged[((row - 1) * (V * N / 4) + j * (N / 4) + q) * sl.lanes + sl.lane] =
            f32x4{p[0], p[1], p[2], p[3]};
      });
    __syncthreads();
    if (row == 0)
      for (int r = 1; r < rows; ++r)
        each4<L>([&](int j, int q) {
          const f32x4 d = staged[((r - 1) * (V * N / 4) + j * (N / 4) + q) * sl.lanes + sl.lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][4 * q + i] += d[i];
        });
    __syncthreads();
  };
  if (rows > 1) {
    if (part1) join(s1);
    if constexpr (kSum0) join(s0);
    if (row > 0) return;
  }
  const Row r1 = row_at(part1, blockIdx.x, H * 4), r0 = row_at(part0, blockIdx.x, H * 4);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    put<F32, N, kCached>(r1, sl.h(j), s1[j]);
    if (kSum0) put<F32, N, kCached>(r0, sl.h(j), s0[j]);
  }
}

// The parameters' gradients from the partial sums [G][H] of S1 and S0 (null: not
// asked for), added in a fixed order; zeros for G = 0.  A workgroup takes 32
// columns: 8 lanes of 4 columns, kSumGroups groups of lanes with every
// kSumGroups-th row each; then 8 groups add up a run of those sums each, and one
// the 8.
struct ParamGrads {
  const float *part1, *part0;
  const void *weight, *bias, *channel;
  float *dweight, *dbias, *dchannel;
};
constexpr int kSumLanes = 8, kSumGroups = 64;
template <class SP>
__global__ __launch_bounds__(kSumLanes* kSumGroups) void param_grads_kernel(ParamGrads p, int G,
                                                                            int H) {
  __shared__ f32x4 buf[2][kSumGroups][kSumLanes];
  const int lane = threadIdx.x % kSumLanes, grp = threadIdx.x / kSumLanes;
  const int h = (blockIdx.x * kSumLanes + lane) * 4;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  auto param = [&](const void* q, float none, float* o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = none;
    if (q && grp == 0 && h < H) {
      Raw<SP, 4> r;
      r.template load<kCached>(row_at(q, 0, H * SP::kBytes), h);
      r.get4(0, o);
    }
  };
  float w[4], b[4], c[4];
  param(p.weight, 1.0f, w);
  param(p.bias, 0.0f, b);
  param(p.channel, 1.0f, c);
  f32x4 s[2] = {zero, zero};
  const float* part[2] = {p.part1, p.part0};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (part[k] && h < H) {
#pragma unroll 4
      for (int g = grp; g < G; g += kSumGroups)
        s[k] += *reinterpret_cast<const f32x4*>(part[k] + (int64_t)g * H + h);
    }
#pragma unroll
  for (int k = 0; k < 2; ++k) buf[k][grp][lane] = s[k];
  __syncthreads();
  constexpr int kRun = kSumGroups / 8;
  if (grp < 8) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      s[k] = buf[k][grp * kRun][lane];
#pragma unroll
      for (int g = 1; g < kRun; ++g) s[k] += buf[k][grp * kRun + g][lane];
      buf[k][grp * kRun][lane] = s[k];   // (read by this lane alone)
    }
  }
  __syncthreads();
  if (grp != 0 || h >= H) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int g = 1; g < 8; ++g) s[k] += buf[k][g * kRun][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.dweight) p.dweight[h + i] = c[i] * s[0][i];
    if (p.dbias) p.dbias[h + i] = c[i] * s[1][i];
    if (p.dchannel) p.dchannel[h + i] = fmaf(b[i], s[1][i], w[i] * s[0][i]);
  }
}

namespace {

// Lanes of a workgroup that hold `elements` of a row each.
int threads_for(int H, int elements) {
  return ((H + elements - 1) / elements + kWave - 1) / kWave * kWave;
}

// Elements of a lane: 8 while 1024 lanes cover the row, else 16.
int lane_elements(int H) { return H > 8 * kMaxWaves * kWave ? 16 : 8; }

// Workgroups of a forward launch: `per_cu` wavefronts a CU, each workgroup looping
// over its rows.  The norm alone takes 32 (layer norm of 16384 x 4096 52 us, with 16
// 62); the kernels with a residual, which have more in flight a row, 16 (that size
// 95 us, with 32 102; 8192 x 7168 one workgroup a row 124 us, 85 so).
unsigned forward_groups(int64_t T, int threads, int per_cu) {
  const int groups = per_cu * kWave / threads;
  const int64_t most = 256 * (groups > 1 ? groups : 1);
  return (unsigned)(T < most ? T : most);
}

// Whether a residual launch has parameters or gates besides the norms' weights: its
// kernel holds them, or loads them ahead, where the lanes hold 8 elements (8192 x 3584
// all gates and layer norm 46 us, loaded in each row's turn 57; two layer norms with
// biases 47, so 59; a token gate 43, so 46).  It has more registers to keep, and those
// without any take none of it (fp32 stream of 8192 x 4096 94.5 us, so 96).
bool extras(const NormSpec& post, const GateSpec& gate, const NormSpec& pre) {
  return post.bias || pre.bias || gate.channel || gate.token;
}

// A backward launch: `groups` workgroups of `rows` rows at a time, `waves` wavefronts
// each.
struct BackwardShape {
  int waves, rows, groups;
};

// Each workgroup writes a row of partial sums per parameter, so there are few and
// large ones: 16 wavefronts a CU, its registers' worth, in one workgroup of as many
// rows as they hold, no more than give every CU one (16384 x 128 11.6 us, a workgroup
// to each row and 16 wavefronts of them a CU 14.4; 16384 x 1024 20.8, so 25.2; 16384 x
// 4096 75.5, so 77.9; 4099 x 3584, layer norm and all gates, 26.2, so 25.8).  Rows of
// more than 8 wavefronts: a workgroup to each, 8 rows or more once there are 256 of
// them, two a CU where the lanes hold 8 elements.
BackwardShape backward_shape(int64_t T, int H) {
  const int elements = lane_elements(H), waves = threads_for(H, elements) / kWave;
  const int64_t each = (T + 255) / 256;
  int64_t rows = kMaxWaves / waves, groups = 256;
  if (rows > each) rows = each > 1 ? each : 1;
  if (waves > kMaxWaves / 2) {
    const int64_t most = elements > 8 ? 256 : 512;
    if (T / 8 > groups) groups = T / 8 < most ? T / 8 : most;
  }
  const int64_t turns = (T + rows - 1) / rows;
  return {waves, (int)rows, (int)(turns < groups ? turns : groups)};
}

// f(a, b, c, layout): the types and how a lane's `elements` lie -- vectors of 16
// bytes of the wider of the row types, a and b, so that a wavefront's load covers
// whole lines (fp32 rows in vectors of 8 elements, two loads that each leave every
// other 16 bytes: residual of 16384 x 4096 158 us, so 145).
template <class F>
hipError_t with_types(int a, int b, int c, int elements, F f) {
  auto layout = [&](auto sa, auto sb, auto sc) {
    constexpr int N = decltype(sa)::kBytes == 2 && decltype(sb)::kBytes == 2 ? 8 : 4;
    if (elements == 8) f(sa, sb, sc, Slice<N, 8 / N>());
    else f(sa, sb, sc, Slice<N, 16 / N>());
  };
  auto third = [&](auto sa, auto sb) {
    if (c == kDtF32) layout(sa, sb, F32());
    else layout(sa, sb, BF16());
  };
  auto second = [&](auto sa) {
    if (b == kDtF32) third(sa, F32());
    else third(sa, BF16());
  };
  if (a == kDtF32) second(F32());
  else second(BF16());
  return hipGetLastError();
}

}  // namespace

int64_t norm_workspace_floats(int64_t T, int H) {
  // (a launch of a few more than 256 rows takes half as many workgroups as one of 256:
  // what is asked for never falls as T grows, so that the largest batch's serves all)
  const int groups = backward_shape(T, H).groups;
  const int64_t least = T < 256 ? T : 256;
  return 2 * (groups > least ? groups : least) * H;
}

hipError_t launch_norm(const void* x, int xdt, int64_t T, int H, const NormSpec& n, int pdt,
                       void* out, int odt, hipStream_t s) {
  const int e = lane_elements(H), threads = threads_for(H, e);
  return with_types(xdt, odt, pdt, e, [&](auto sx, auto so, auto sp, auto layout) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(forward_groups(T, threads, 32)), dim3(threads), 0, s, x, T, H,
                         n, out);
    };
    typedef decltype(sx) SX;
    typedef decltype(so) SO;
    typedef decltype(sp) SP;
    typedef decltype(layout) L;
    // (a bias loaded with each row waits for the next row's: 16384 x 4096 48.2 us, so 50.6)
    if constexpr (L::N * L::V <= 8)
      if (n.bias) return go(norm_kernel<SX, SO, SP, L, true>);
    go(norm_kernel<SX, SO, SP, L, false>);
  });
}

hipError_t launch_norm_residual(const void* y, int ydt, const void* x, int xdt, int64_t T, int H,
                                const NormSpec& post, const GateSpec& gate, int pdt, void* r,
                                const NormSpec& pre, void* n, hipStream_t s) {
  // bf16 rows of more than 4096 on half the lanes: two workgroups fit a CU (of 7168:
  // 14 wavefronts of 65 registers do not share one, 7 of 110 do; 8192 rows 97 -> 85
  // us, one row 3.4 -> 3.2).  Up to 4096 that costs as much as it gives (16384 rows of
  // 4096 95 -> 100 us, 1024 rows 7.0 -> 6.4).
  // Nor with a bias from 8 rows a CU on: the parameters that 8 elements leave room to
  // hold are worth more there (7168, layer norm, all gates, 8192 rows 97 -> 87 us, 2048
  // 22.9 -> 21.4, but 1024 12.6 -> 13.2).
  const bool held = (post.bias || pre.bias) && T >= 8 * 256;
  const bool half = ydt == kDtBF16 && xdt == kDtBF16 && H > 4096 && !held;
  const int e = half ? 16 : lane_elements(H);
  const int threads = threads_for(H, e);
  // With an fp32 stream, rows of 6 to 8 wavefronts and no post layer norm (whose two more
  // reductions want a second workgroup to run beside), one workgroup a CU from 32 rows for
  // each on: channel gate and next layer norm, 16384 rows of 3328, 3584, 4096 111, 128, 133
  // us, with two 124, 128, 141; a token gate 111, 120, 135, so 121, 129, 139.  Of fewer rows
  // a CU has too little in flight: 2048 rows of 2816 with it 15.6 us, with two 13.3, 4096
  // 27.0 and 23.7, 1024 of 4096 10.8 and 10.1.  4 wavefronts a row 37.3, so 36.0.  Without
  // gates or biases two (8192 x 4096 72 us, with one 78).
  const bool few =
      xdt == kDtF32 && post.kind != kNormLayer && threads > 5 * kWave && T >= 32 * 256;
  return with_types(ydt, xdt, pdt, e, [&](auto sy, auto sx, auto sp, auto layout) {
    auto go = [&](auto kernel, int per_cu) {
      hipLaunchKernelGGL(kernel, dim3(forward_groups(T, threads, per_cu)), dim3(threads), 0, s, y,
                         nullptr, 0, nullptr, x, T, H, post, gate, r, pre, n);
    };
    typedef decltype(sy) SY;
    typedef decltype(sx) SX;
    typedef decltype(sp) SP;
    typedef decltype(layout) L;
    if constexpr (L::N * L::V <= 8)
      if (extras(post, gate, pre))
        return go(norm_residual_kernel<SY, SY, SX, SP, L, false, true>, few ? 8 : 16);
    go(norm_residual_kernel<SY, SY, SX, SP, L, false, false>, 16);
  });
}

hipError_t launch_combine_norm_residual(const void* y, int ydt, const float* w, int K,
                                        const void* shared, int sdt, const void* x, int xdt,
                                        int64_t T, int H, const NormSpec& post,
                                        const GateSpec& gate, int pdt, void* r,
                                        const NormSpec& pre, void* n, hipStream_t s) {
  const int e = lane_elements(H), threads = threads_for(H, e);
  return with_types(ydt, xdt, pdt, e, [&](auto sy, auto sx, auto sp, auto layout) {
    auto go = [&](auto ss) {
      auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(forward_groups(T, threads, 16)), dim3(threads), 0, s, y, w,
                           K, shared, x, T, H, post, gate, r, pre, n);
      };
      typedef decltype(sy) SY;
      typedef decltype(ss) SS;
      typedef decltype(sx) SX;
      typedef decltype(sp) SP;
      typedef decltype(layout) L;
      if constexpr (L::N * L::V <= 8)
        if (extras(post, gate, pre))
          return launch(norm_residual_kernel<SY, SS, SX, SP, L, true, true>);
      launch(norm_residual_kernel<SY, SS, SX, SP, L, true, false>);
    };
    if (sdt == kDtF32) go(F32());
    else go(BF16());
  });
}

hipError_t launch_norm_backward(const void* e, int edt, const void* v, int vdt, const void* dres,
                                int64_t T, int H, const NormSpec& n, const GateSpec& gate, int pdt,
                                void* dv, float* dweight, float* dbias, float* dchannel,
                                float* dtoken, float* workspace, hipStream_t s) {
  const BackwardShape shape = backward_shape(T, H);
  const int G = shape.groups, threads = shape.waves * shape.rows * kWave;
  const int elements = lane_elements(H);
  const int staged = (threads - shape.waves * kWave) * elements * 4;
  ParamGrads p{nullptr, nullptr, n.weight, n.bias, gate.channel, dweight, dbias, dchannel};
  // (no tokens: zeros, whatever the parameters that the sums would be multiplied with)
  if (T == 0) p.weight = p.bias = p.channel = nullptr;
  float* part1 = dweight || dchannel ? workspace : nullptr;
  float* part0 = dbias || (dchannel && n.bias) ? workspace + (int64_t)G * H : nullptr;
  p.part1 = part1;
  p.part0 = part0;
  if (T > 0) {
    const hipError_t st = with_types(edt, vdt, pdt, elements, [&](auto se, auto sv, auto sp, auto layout) {
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(G), dim3(threads), staged, s, e, v, dres, T, H, shape.waves,
                           shape.rows, n, gate, dv, part1, part0, dtoken);
      };
      typedef decltype(se) SE;
      typedef decltype(sv) SV;
      typedef decltype(sp) SP;
      typedef decltype(layout) L;
      if (dres && part0) go(norm_backward_kernel<SE, SV, SP, L, true, true>);
      else if (dres) go(norm_backward_kernel<SE, SV, SP, L, true, false>);
      else if (part0) go(norm_backward_kernel<SE, SV, SP, L, false, true>);
      else go(norm_backward_kernel<SE, SV, SP, L, false, false>);
    });
    if (st != hipSuccess) return st;
  }
  if (!dweight && !dbias && !dchannel) return hipSuccess;
  const dim3 grid((H + 4 * kSumLanes - 1) / (4 * kSumLanes)), block(kSumLanes * kSumGroups);
  if (pdt == kDtF32) hipLaunchKernelGGL(param_grads_kernel<F32>, grid, block, 0, s, p, G, H);
  else hipLaunchKernelGGL(param_grads_kernel<BF16>, grid, block, 0, s, p, G, H);
  return hipGetLastError();
}

}  // namespace moe
