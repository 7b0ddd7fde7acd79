// Tokens in the rows of an alignment and back, with weights, and the gradients
// (what each computes: include/moe_layer.h).
//
// Everything here is bound by memory: a row element is moved once and takes at
// most one multiply-add.  The kernels go by token or by pair, not by alignment
// row: a token's row is read once for its K copies (permute), its K rows are
// summed in slot order in registers (unpermute), and a pair's dot product stays
// in one wavefront (unpermute_backward), so no sum needs atomics.  The padding
// rows have no token; workgroups past the others' zero them, expert by expert.
//
// A unit of work is kLanes vectors of 16 bytes of one token's or pair's row, on
// as many lanes: a wavefront where the row fills one (its row index and weight
// then sit in scalar registers, and its loads take the row's address from them),
// else the smallest power of two of lanes that holds the row, several rows to a
// wavefront (16384 tokens of 64, 8 experts each: permute 4.9 us, with a wavefront a
// row 16; unpermute 8.1 and 15; of 256: unpermute 14.5 and 20).
//
// Measured on MI355X, inputs that no cache holds (a copy of 1 GB runs at 5.1 TB/s):
// 16384 tokens of 3584 bf16 to 8 experts each 211 us (1.09 GB with the padding, 5.1
// TB/s); the tokens' gradient from 32768 rows of 7168 90 us (5.9 TB/s); the gradients
// of 65536 rows of 7168 with 16 thousand padding rows 409 us (2.3 GB, 5.7 TB/s).  Units
// by alignment row, so that the rows are read and written in order and the tokens
// gathered, run the last one in 470 us.
#include "block_kernels.h"
#include "common.h"
#include "rows.h"

namespace moe {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// Row loads and stores, past the caches (non-temporal) where kStream says so.
template <bool kStream>
__device__ __forceinline__ u32x4 row_load(const u32x4* p) {
  return kStream ? __builtin_nontemporal_load(p) : *p;
}
template <bool kStream>
__device__ __forceinline__ void row_store(u32x4* p, u32x4 v) {
  if constexpr (kStream) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// The 16 / kBytes elements of a vector as fp32, and back.
template <class S>
struct Vec {
  static constexpr int N = 16 / S::kBytes;
};
template <class S>
__device__ __forceinline__ void unpack(u32x4 r, float* v) {
  if constexpr (S::kBytes == 2) {
    const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(q[j] << 16);
      v[2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
    }
  } else {
    const f32x4 a = __builtin_bit_cast(f32x4, r);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
}
template <class S>
__device__ __forceinline__ u32x4 pack(const float* v) {
  if constexpr (S::kBytes == 2) {
    u32x4 r;
    r.x = pack_bf16x2(v[0], v[1]);
    r.y = pack_bf16x2(v[2], v[3]);
    r.z = pack_bf16x2(v[4], v[5]);
    r.w = pack_bf16x2(v[6], v[7]);
    return r;
  } else {
    return __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
  }
}

// N (4 or 8) consecutive elements of the tokens' own buffers, whose type may
// differ from the rows'.
template <class S, int N>
__device__ __forceinline__ void load_n(const typename S::T* p, float* v) {
  if constexpr (N == 8) {
    load8f<S>(p, v);
  } else if constexpr (S::kBytes == 4) {
    unpack<F32>(*reinterpret_cast<const u32x4*>(p), v);
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
}
template <class S, int N>
__device__ __forceinline__ void store_n(typename S::T* p, const float* v) {
  if constexpr (N == 8) store8f<S>(p, v);
  else store_out4<S>(p, f32x4{v[0], v[1], v[2], v[3]});
}

// Sum over the aligned group of kLanes lanes, in every lane of it.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (kLanes == 64) {
    return wave_sum(v);
  } else {
    v = dpp_add<kQuadXor1>(v);
    v = dpp_add<kQuadXor2>(v);
    v = dpp_add<kRowHalfMirror>(v);
    if constexpr (kLanes >= 16) v = dpp_add<kRowMirror>(v);
    if constexpr (kLanes == 32)   // lane i and lane i ^ 16 (ds_swizzle, bit mode: xor mask 16)
      v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));
    return v;
  }
}

// The unit that this lane works on in workgroup b; scalar where it is the
// wavefront's.
template <int kLanes>
__device__ __forceinline__ uint32_t unit_of(uint32_t b) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t first = (b * kWaves + wave) * (kWave / kLanes);
  return kLanes == kWave ? first : first + (threadIdx.x & (kWave - 1)) / kLanes;
}

// The padding rows: expert e's are offsets[e] + counts[e] .. offsets[e + 1] - 1,
// one run of memory, zeroed by `subs` workgroups.
struct Padding {
  const int32_t* counts;
  const int32_t* offsets;
  int subs;
};

// Zeroes share item % subs of the padding rows (of nv vectors) of expert item / subs.
__device__ __forceinline__ void zero_padding(uint32_t item, const Padding& pad, int nv, int64_t cap,
                                             u32x4* rows) {
  const uint32_t e = item / (uint32_t)pad.subs;
  int64_t first = (int64_t)pad.offsets[e] + pad.counts[e], end = pad.offsets[e + 1];
  if (first < 0) first = 0;
  if (end > cap) end = cap;
  const u32x4 z = {0, 0, 0, 0};
  const int64_t stride = (int64_t)pad.subs * kThreads;
  for (int64_t i = first * nv + (item - e * pad.subs) * kThreads + threadIdx.x; i < end * nv;
       i += stride)
    row_store<true>(rows + i, z);
}

// rows[inv_pos[t*K + k]] = x[t] (rows of nv vectors; a token takes `chunks`
// units), then the padding rows in `pads` items.
template <int kLanes, bool kStream>
__global__ __launch_bounds__(kThreads) void permute_kernel(
    const u32x4* __restrict__ x, uint32_t T, int K, int nv, uint32_t chunks, uint32_t groups,
    const int32_t* __restrict__ inv_pos, int64_t cap, u32x4* __restrict__ rows, uint32_t pads,
    Padding pad) {
  for (uint32_t b = blockIdx.x; b < groups + pads; b += gridDim.x) {
    if (b >= groups) {
      zero_padding(b - groups, pad, nv, cap, rows);
      continue;
    }
    const uint32_t u = unit_of<kLanes>(b);
    const uint32_t t = u / chunks;
    const int v = (u - t * chunks) * kLanes + threadIdx.x % kLanes;
    if (t >= T || v >= nv) continue;
    const u32x4 d = x[(int64_t)t * nv + v];
    const int32_t* pos = inv_pos + (int64_t)t * K;
    for (int k = 0; k < K; ++k) {
      const int64_t r = pos[k];
      if (r >= 0 && r < cap) row_store<kStream>(rows + r * nv + v, d);
    }
  }
}

constexpr int kSlots = 4;   // rows in flight per lane (8: 98 us for 89 at 32768 rows of 7168)

// out[t] = sum_k w[t][k] rows[inv_pos[t*K + k]] (+ shared[t]); w null: ones.
template <class SR, class SS, class SO, int kLanes, bool kStream>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(
    const u32x4* __restrict__ rows, const float* __restrict__ w,
    const typename SS::T* __restrict__ shared, uint32_t T, int K, int nv, uint32_t chunks,
    uint32_t groups, const int32_t* __restrict__ inv_pos, int64_t cap,
    typename SO::T* __restrict__ out) {
  constexpr int N = Vec<SR>::N;
  for (uint32_t b = blockIdx.x; b < groups; b += gridDim.x) {
    const uint32_t u = unit_of<kLanes>(b);
    const uint32_t t = u / chunks;
    const int v = (u - t * chunks) * kLanes + threadIdx.x % kLanes;
    if (t >= T || v >= nv) continue;
    const int32_t* pos = inv_pos + (int64_t)t * K;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kSlots) {
      u32x4 d[kSlots];
      float wk[kSlots];
      bool use[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        use[j] = false;
        if (k0 + j < K) {
          const int64_t r = pos[k0 + j];
          wk[j] = w ? w[(int64_t)t * K + k0 + j] : 1.0f;
          use[j] = r >= 0 && r < cap && wk[j] != 0.0f;
          if (use[j]) d[j] = row_load<kStream>(rows + r * nv + v);
        }
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (use[j]) {
          float y[N];
          unpack<SR>(d[j], y);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(wk[j], y[i], acc[i]);
        }
    }
    const int64_t o = ((int64_t)t * nv + v) * N;
    if (shared) {
      float s[N];
      load_n<SS, N>(shared + o, s);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += s[i];
    }
    store_n<SO, N>(out + o, acc);
  }
}


// drows[r] = w[p] dout[t] and dw[p] = <dout[t], rows[r]> for the row r of pair p
// = t*K + k, a unit each: dout's row is read K times over, from the caches.  A
// lane reads an element of rows before it writes that of drows (they may be one
// buffer).
template <class S, int kLanes, bool kStream>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(
    const u32x4* __restrict__ dout, const u32x4* rows, const float* __restrict__ w,
    uint32_t pairs, int K, int nv, uint32_t groups, const int32_t* __restrict__ inv_pos,
    int64_t cap, u32x4* drows, float* __restrict__ dw, uint32_t pads, Padding pad) {
  constexpr int N = Vec<S>::N;
  // vectors of a row in flight per lane (16384 x 8 rows of 1032: 1 149 us, 2 141, 4 131;
  // a row on part of a wavefront has one)
  constexpr int kSteps = kLanes == kWave ? 4 : 1;
  for (uint32_t b = blockIdx.x; b < groups + pads; b += gridDim.x) {
    if (b >= groups) {   // (there are none where drows is null)
      zero_padding(b - groups, pad, nv, cap, drows);
      continue;
    }
    const uint32_t p = unit_of<kLanes>(b);
    const int lane = threadIdx.x % kLanes;
    // (a group past the pairs keeps its lanes: they take part in the sums)
    const int64_t r = p < pairs ? inv_pos[p] : -1;
    const bool used = r >= 0 && r < cap;
    const float wk = w && p < pairs ? w[p] : 1.0f;
    // one sum per vector in flight: shorter chains of additions, and closer to the product
    float acc[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) acc[i] = 0.0f;
    if (used) {
      const u32x4* g0 = dout + (int64_t)(p / (uint32_t)K) * nv;
      const int64_t r0 = r * nv;
      for (int v0 = lane; v0 < nv; v0 += kSteps * kLanes) {
        u32x4 dg[kSteps], dv[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          if (v0 + i * kLanes < nv) {
            dg[i] = g0[v0 + i * kLanes];
            if (dw) dv[i] = row_load<kStream>(rows + r0 + v0 + i * kLanes);
          }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          if (v0 + i * kLanes < nv) {
            float g[N], y[N];
            unpack<S>(dg[i], g);
            if (dw) {
              unpack<S>(dv[i], y);
#pragma unroll
              for (int j = 0; j < N; ++j) acc[i] = fmaf(g[j], y[j], acc[i]);
            }
            if (drows) {
#pragma unroll
              for (int j = 0; j < N; ++j) g[j] *= wk;
              row_store<true>(drows + r0 + v0 + i * kLanes, pack<S>(g));
            }
          }
      }
    }
    if (dw) {
#pragma unroll
      for (int i = kSteps / 2; i > 0; i /= 2)
#pragma unroll
        for (int j = 0; j < i; ++j) acc[j] += acc[j + i];
      const float dot = lanes_sum<kLanes>(acc[0]);
      if (lane == 0 && p < pairs) dw[p] = dot;
    }
  }
}

// dlogits[t][e] = sum over the slots j with id e of w_j (dw_j - sum_i w_i dw_i), slots of
// weight 0 left out of both sums: the way back does not read their rows, so that their
// dw may be anything.
// One wavefront a token, its slots held 64 to a register (kSlotRegs of them); each
// lane owns every 64th expert (kOutRegs) and looks the slots through in order.
template <int kSlotRegs, int kOutRegs>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw,
    int64_t T, int E, int K, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < T; t += (int64_t)gridDim.x * kWaves) {
    int id[kSlotRegs];
    float g[kSlotRegs], d[kSlotRegs];
#pragma unroll
    for (int j = 0; j < kSlotRegs; ++j) {
      const int k = j * kWave + lane;
      const bool there = k < K;
      id[j] = there ? ids[t * K + k] : -1;
      g[j] = there ? w[t * K + k] : 0.0f;
      d[j] = there ? dw[t * K + k] : 0.0f;
      if (id[j] < 0 || id[j] >= E) {   // unused: whatever its weight and gradient hold
        id[j] = -1;
        g[j] = 0.0f;
      }
      if (g[j] == 0.0f) d[j] = 0.0f;
    }
    // in 64 bits: with one weight near 1, its dw less the sum is what the others leave
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kSlotRegs; ++j)
      for (int l = 0; l < kWave && j * kWave + l < K; ++l)
        s = fma((double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(g[j]), l)),
                (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(d[j]), l)), s);
#pragma unroll
    for (int j = 0; j < kSlotRegs; ++j) g[j] = (float)((double)g[j] * ((double)d[j] - s));
    float o[kOutRegs];
#pragma unroll
    for (int i = 0; i < kOutRegs; ++i) o[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kSlotRegs; ++j)
      for (int l = 0; l < kWave && j * kWave + l < K; ++l) {
        const int e = __builtin_amdgcn_readlane(id[j], l);
        const float ge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g[j]), l));
#pragma unroll
        for (int i = 0; i < kOutRegs; ++i) o[i] += e == i * kWave + lane ? ge : 0.0f;
      }
#pragma unroll
    for (int i = 0; i < kOutRegs; ++i)
      if (i * kWave + lane < E) dlogits[t * E + i * kWave + lane] = o[i];
  }
}

namespace {

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups; the kernels loop past it

unsigned grid_of(int64_t groups) { return (unsigned)(groups < kMaxGrid ? groups : kMaxGrid); }

// When rows go past the caches.  Loads: where the pairs' rows are more than 96 MB,
// of which a last-level cache of 256 MB keeps little until they are read (MI355X, sums
// over 8 rows of 3584 a token: 1024 tokens, 59 MB, cached 11.5 us, past the caches
// 12.2; 2048 tokens 29.4 and 25.1).  Stores of the tokens' copies: where rows are whole
// 128-byte lines, since a line that two rows share is otherwise written twice in part
// (16384 tokens to 8 rows of 1024 bf16 each: cached 62 us, past the caches 53; of 1032
// 79 and 94).  Stores of the gradients, whose rows each wavefront also reads: always (8
// rows of 1024 a token, 16384 tokens: cached 116 us, so 104; of 1032, 4096 tokens 38
// and 30).
bool many(int64_t pairs, int nv) { return pairs * nv > (int64_t)96 << 16; }
bool whole_lines(int nv) { return nv % 8 == 0; }

template <class F>
void with_flag(bool flag, F f) {
  if (flag) f(std::integral_constant<bool, true>());
  else f(std::integral_constant<bool, false>());
}

// f(lanes): the lanes of a unit as a constant, for rows of nv vectors.
template <class F>
hipError_t with_lanes(int nv, F f) {
  if (nv > 32) f(std::integral_constant<int, 64>());
  else if (nv > 16) f(std::integral_constant<int, 32>());
  else if (nv > 8) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 8>());
  return hipGetLastError();
}

// Workgroups that `units` units of `lanes` lanes take.
int64_t groups_of(int64_t units, int lanes) {
  const int per = kThreads / lanes;
  return (units + per - 1) / per;
}

// Workgroups for an expert's padding, 8 stores a lane each if every row that the
// plan has room for beyond its pairs were padding: up to 16 (1024 in all where
// there are few experts, whose max-padded slots may be long).  Block-wise padding
// leaves at most block_m - 1 rows an expert, max padding any number.
Padding padding_of(const RowMap& rm, int E, int64_t cap, int64_t pairs, int nv) {
  const int64_t rows = (cap - pairs + E - 1) / E;
  const int64_t want = (rows * nv + 8 * kThreads - 1) / (8 * kThreads);
  const int64_t most = 1024 / E > 16 ? 1024 / E : 16;
  return Padding{rm.counts, rm.offsets, (int)(want < 1 ? 1 : want < most ? want : most)};
}

template <class SR, class SS, class SO>
hipError_t launch_unpermute_t(const void* rows, const float* w, const void* shared, int64_t T,
                              int K, int H, const int32_t* inv_pos, int64_t cap, void* out,
                              hipStream_t s) {
  const int nv = H / Vec<SR>::N;
  return with_lanes(nv, [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value;
    const int chunks = (nv + kLanes - 1) / kLanes;
    const int64_t groups = groups_of(T * chunks, kLanes);
    with_flag(many(T * K, nv), [&](auto stream) {
      hipLaunchKernelGGL((unpermute_kernel<SR, SS, SO, kLanes, decltype(stream)::value>),
                         dim3(grid_of(groups)), dim3(kThreads), 0, s,
                         static_cast<const u32x4*>(rows), w,
                         static_cast<const typename SS::T*>(shared), (uint32_t)T, K, nv,
                         (uint32_t)chunks, (uint32_t)groups, inv_pos, cap,
                         static_cast<typename SO::T*>(out));
    });
  });
}

template <class SR, class SS>
hipError_t unpermute_out(const void* rows, const float* w, const void* shared, int64_t T, int K,
                         int H, const int32_t* inv_pos, int64_t cap, void* out, int odt,
                         hipStream_t s) {
  return odt == kDtF32
             ? launch_unpermute_t<SR, SS, F32>(rows, w, shared, T, K, H, inv_pos, cap, out, s)
             : launch_unpermute_t<SR, SS, BF16>(rows, w, shared, T, K, H, inv_pos, cap, out, s);
}

template <class S>
hipError_t unpermute_backward_t(const void* dout, const void* rows, const float* w, int64_t T,
                                int K, int H, const RowMap& rm, int E, int64_t cap, void* drows,
                                float* dw, hipStream_t s) {
  const int nv = H / Vec<S>::N;
  const Padding pad = padding_of(rm, E, cap, T * K, nv);
  const int64_t pads = drows ? E * pad.subs : 0;
  return with_lanes(nv, [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value;
    const int64_t groups = groups_of(T * K, kLanes);
    with_flag(many(T * K, nv), [&](auto stream) {
      hipLaunchKernelGGL((unpermute_backward_kernel<S, kLanes, decltype(stream)::value>),
                         dim3(grid_of(groups + pads)), dim3(kThreads), 0, s,
                         static_cast<const u32x4*>(dout), static_cast<const u32x4*>(rows), w,
                         (uint32_t)(T * K), K, nv, (uint32_t)groups, rm.inv_pos, cap,
                         static_cast<u32x4*>(drows), dw, (uint32_t)pads, pad);
    });
  });
}

}  // namespace

hipError_t launch_permute(const void* x, int dt, int64_t T, int K, int H, const RowMap& rm, int E,
                          int64_t cap, void* rows, bool zeroed, hipStream_t s) {
  const int nv = dt == kDtF32 ? H / 4 : H / 8;
  const Padding pad = padding_of(rm, E, cap, T * K, nv);
  const int64_t pads = zeroed ? E * pad.subs : 0;
  return with_lanes(nv, [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value;
    const int chunks = (nv + kLanes - 1) / kLanes;
    const int64_t groups = groups_of(T * chunks, kLanes);
    with_flag(whole_lines(nv), [&](auto stream) {
      hipLaunchKernelGGL((permute_kernel<kLanes, decltype(stream)::value>),
                         dim3(grid_of(groups + pads)), dim3(kThreads), 0, s,
                         static_cast<const u32x4*>(x), (uint32_t)T, K, nv, (uint32_t)chunks,
                         (uint32_t)groups, rm.inv_pos, cap, static_cast<u32x4*>(rows),
                         (uint32_t)pads, pad);
    });
  });
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
  return dt == kDtF32 ? unpermute_backward_t<F32>(dout, rows, w, T, K, H, rm, E, cap, drows, dw, s)
                      : unpermute_backward_t<BF16>(dout, rows, w, T, K, H, rm, E, cap, drows, dw,
                                                   s);
}

hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, int64_t T,
                                 int E, int K, float* dlogits, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid_of((T + kWaves - 1) / kWaves)), dim3(kThreads), 0, s, ids,
                       w, dw, T, E, K, dlogits);
  };
  // (K <= E <= 256)
  if (E <= kWave) go(route_backward_kernel<1, 1>);
  else if (K <= kWave) go(route_backward_kernel<1, 4>);
  else go(route_backward_kernel<4, 4>);
  return hipGetLastError();
}

}  // namespace moe
