// The experts' products of a training step on gfx950.
//
// For a row of expert e with token x, gate and up values (g, u) = W13 x, a = silu(g) * u and
// y = W2 a.  From dy, the gradient of y:
//
//   da = W2^T dy     dg = da * u * s (1 + g (1 - s)), du = da * g s     with s = 1 / (1 + e^-g)
//   dx = W13^T (dg, du)     dW13 = sum over the expert's rows of (dg, du) x^T
//   dW2 = sum over the expert's rows of dy a^T
//
// Six products in three forms, by which index runs along memory.  In the forward both operands
// have the contraction there ("along"); in da and dx the weights have it across their rows; in
// the weights' gradients both operands do, since the contraction is over rows ("across").
// All run on one tile: 256 features x 256 rows (or features), 8 wavefronts as 2 x 4 of
// 128 x 64 with 16x16x32 bf16 MFMAs, the contraction in steps of 32 through a ring of 4 stages
// of 32 KB in LDS, filled by direct loads three steps ahead.
//
//   along   a stage's 256 rows of 64 bytes; 16-byte segment s of row r at s ^ ((r >> 1) & 3);
//           a fragment is one 16-byte read
//   across  a stage's 32 rows of 512 bytes in 16 chunks of two, k and k + 8, 64 bytes between
//           the chunks; the segments of the second row at s ^ 3.  A fragment is two transposing
//           8-byte reads (a lane's 4 values of one column from 4 rows): the gaps put the 4 rows
//           that a read takes together in different quarters of the banks, and the swizzle k
//           and k + 8 in different halves of those, so that 32 lanes meet every bank once
//
// Direct loads go through buffer descriptors, whose range check writes zeros for what lies
// outside: rows past an expert's last one, features past an edge that is no multiple of 256.
// So every step runs the same instructions, and nothing outside a matrix is read.
//
// The features of a tile are dealt to MFMA rows so that a lane's sums of two neighbouring MFMA
// tiles are 8 neighbours in memory (feature(): 16-byte stores, 64 bytes of a row side by side).
#include <type_traits>

#include "pack.h"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kTile = 256;                    // features, and rows, of a tile
constexpr int kStep = 32;                     // contraction of a stage
constexpr int kStages = 4;
constexpr int kAlong = kTile * kStep * 2;     // bytes of an operand's stage
constexpr int kChunk = 2 * kTile * 2 + 64;    // two rows and a gap
constexpr int kAcross = 16 * kChunk;
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxE = 256;
constexpr int TM = 8;                         // a wavefront's MFMA tiles of features
constexpr uint32_t kOutside = 0xfffffff0u;    // an offset that every descriptor refuses

template <bool kAAcross, bool kBAcross>
struct Smem {
  static constexpr int kA = kAAcross ? kAcross : kAlong;
  static constexpr int kB = kBAcross ? kAcross : kAlong;
  uint8_t a[kStages][kA];   // the features' operand
  uint8_t b[kStages][kB];   // the rows'
  int tok[kTile];
  int pre[kMaxE + 1];
  int wsum[kWaves];
};

enum Op { kGateUp, kDown, kDAct, kDX, kDW13, kDW2 };

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void* LdsPtr;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* LdsVec4;

__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

__device__ __forceinline__ void load_lds16(Rsrc r, uint32_t lane_off, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 16, (int)lane_off, (int)off, 0, 0);
}

__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void wait_lgkm0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (0x7 << 4) | (0 << 8));
}

// what a lane is, in the block and in an MFMA
struct Lane {
  int tid, lane, wave, wm, wn, m, g;
  __device__ __forceinline__ Lane() {
    tid = threadIdx.x;
    lane = tid & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(tid / kWave);   // so that its indices stay scalar
    wm = wave >> 2;
    wn = wave & 3;
    m = lane & 15;
    g = lane >> 4;
  }
};

// Feature (of a tile's 256) of MFMA tile tm (of 8 of wavefront row wm), row 4c + j: the pair of
// tiles tm, tm ^ 1 holds 32 neighbours, and lane group c of the two 8 neighbours, 4 in each.
// Which tile has the first 4 alternates with c, so that the transposing reads of one tile use
// both halves of the 16-byte segments and with them every bank.
__device__ __forceinline__ int feature(int wm, int tm, int c, int j) {
  return wm * 128 + 32 * (tm >> 1) + 8 * c + 4 * ((c ^ tm) & 1) + j;
}

// The 8 sums of a lane in a pair of tiles, in the order of their features
__device__ __forceinline__ void in_order(int g, f32x4 even, f32x4 odd, float* v) {
  const f32x4 lo = g & 1 ? odd : even, hi = g & 1 ? even : odd;
  v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
  v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
}

// ------------------------------------------------------------------ filling a stage
//
// A wavefront's two direct loads j = 0, 1 fill KB 2 wave + j of an operand's 16 KB.

// Contraction along memory: load j holds rows 16 (2 wave + j) .. + 15, 4 lanes a row.
// row_off(r): the byte offset of the operand's row r, or kOutside.
struct Along {
  Rsrc r;
  uint32_t off[2];
  template <class F>
  __device__ __forceinline__ void set(const Lane& l, Rsrc rs, F row_off) {
    r = rs;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 16 * (2 * l.wave + j) + (l.lane >> 2);
      const uint32_t o = row_off(row);
      off[j] = o == kOutside ? o : o + (uint32_t)(((l.lane & 3) ^ ((row >> 1) & 3)) << 4);
    }
  }
  __device__ __forceinline__ void issue(const Lane& l, int step, uint8_t* stage) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      load_lds16(r, off[j], (uint32_t)step * (kStep * 2), stage + (2 * l.wave + j) * 1024);
  }
};

// Chunk q = 2 wave + j of a stage: its first row, and the row and the 16-byte segment that a
// lane fetches.
__device__ __forceinline__ int chunk_row(int q) { return (q & 7) | (q >> 3) << 4; }
__device__ __forceinline__ int across_row(const Lane& l, int j) {
  return chunk_row(2 * l.wave + j) + ((l.lane >> 5) << 3);
}
__device__ __forceinline__ int across_seg(const Lane& l) {
  return (l.lane & 31) ^ (3 * (l.lane >> 5));
}

// Contraction across memory: rows of `row_bytes`, `rows` of them, the tile's features from
// byte 2 f0.
struct Across {
  const uint8_t* base;
  uint32_t off[2];
  uint32_t row_bytes;
  int rows;
  __device__ __forceinline__ void set(const Lane& l, const void* p, uint32_t bytes, int n, int f0) {
    base = static_cast<const uint8_t*>(p);
    row_bytes = bytes;
    rows = n;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t col = (uint32_t)f0 * 2 + (uint32_t)across_seg(l) * 16;
      off[j] = col < bytes ? (uint32_t)across_row(l, j) * bytes + col : kOutside;
    }
  }
  __device__ __forceinline__ void issue(const Lane& l, int step, uint8_t* stage) {
    // the stage's rows alone: any number of them, of matrices of any size, and the rest zeros
    const int left = min(kStep, rows - step * kStep);
    const Rsrc r = make_rsrc(base + (size_t)step * kStep * row_bytes, (uint32_t)left * row_bytes);
#pragma unroll
    for (int j = 0; j < 2; ++j) load_lds16(r, off[j], 0, stage + (2 * l.wave + j) * kChunk);
  }
};

// p / K for 0 <= p < 2^31, as a product with mul = ceil(2^(31 + shift) / K), 2^shift >= K:
// the error of mul, below K <= 2^shift, times p stays below one part of the quotient
struct Divider {
  uint32_t mul;
  int shift;
};
__device__ __forceinline__ uint32_t divided(const Divider& d, uint32_t p) {
  return __umulhi(p * 2, d.mul) >> d.shift;
}

// ------------------------------------------------------------------ reading fragments

// 8 values of the contraction for this lane's column, from byte `at` and 4 chunks further
__device__ __forceinline__ u32x4 read_across(const uint8_t* at) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsVec4)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsVec4)(at + 4 * kChunk));
  const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
  return u32x4{a.x, a.y, b.x, b.y};
}

// the byte of a stage of which this lane's transposing reads of row group g, row r, start
__device__ __forceinline__ int across_at(const Lane& l) {
  return ((l.m >> 2) + 8 * (l.g >> 1)) * kChunk + (l.g & 1) * (kTile * 2);
}

template <bool kIsAcross>
__device__ __forceinline__ void read_features(const Lane& l, const uint8_t* stage, u32x4 (&f)[TM]) {
  if constexpr (kIsAcross) {
    const int c = l.m & 3;   // the 4 features this lane points at
    const int at = across_at(l) + l.wm * 256 + ((c ^ (3 * (l.g & 1))) << 4) + ((c & 1) << 3);
    const uint8_t* even = stage + at;
    const uint8_t* odd = stage + (at ^ 8);
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) f[tm] = read_across((tm & 1 ? odd : even) + (tm >> 1) * 64);
  } else {
    const int at = (l.wm * 128 + l.m) * 64 + ((l.g ^ ((l.m >> 1) & 3)) << 4);
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) f[tm] = *reinterpret_cast<const u32x4*>(stage + at + tm * 1024);
  }
}

// the rows of wavefront column wn: tiles of 16 wn, wn + 4, ...
template <bool kIsAcross, int TN>
__device__ __forceinline__ void read_rows(const Lane& l, const uint8_t* stage, u32x4 (&f)[TN]) {
  if constexpr (kIsAcross) {
    const int c = l.m & 3;
    const int at = across_at(l) + (((2 * l.wn + (c >> 1)) ^ (3 * (l.g & 1))) << 4) + ((c & 1) << 3);
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) f[tn] = read_across(stage + at + tn * 128);
  } else {
    const int at = (l.wn * 16 + l.m) * 64 + ((l.g ^ ((l.m >> 1) & 3)) << 4);
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) f[tn] = *reinterpret_cast<const u32x4*>(stage + at + tn * 4096);
  }
}

// ------------------------------------------------------------------ the product
//
// Step t works on fragments read before it while those of step t + 1 are read.  Before its
// barrier: stage t + 1 has landed (the loads of later stages may stay in flight) and this
// wavefront's reads of stage t are done; after it stage t's slot is free for stage t + 4.
// The next item may fill the ring at once: every read was waited for at the last barrier.

// The ring's slots come as pointers that do not alias, so that a read waits for the direct loads
// into its own slot alone: the compiler otherwise has every transposing read wait for all of them
// (measured: 620 TFLOP/s where both operands are read so, against the figures below).
template <bool kAAcross, bool kBAcross, int TN, class LA, class LB>
__device__ __forceinline__ void product(const Lane& l, uint8_t* __restrict__ a0,
                                        uint8_t* __restrict__ a1, uint8_t* __restrict__ a2,
                                        uint8_t* __restrict__ a3, uint8_t* __restrict__ b0,
                                        uint8_t* __restrict__ b1, uint8_t* __restrict__ b2,
                                        uint8_t* __restrict__ b3, LA& la, LB& lb, int nk,
                                        f32x4 (&acc)[TM][TN]) {
#pragma unroll
  for (int tm = 0; tm < TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) acc[tm][tn] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (nk == 0) return;

  u32x4 fa[2][TM], fb[2][TN];
  auto slot_a = [&](auto s) -> uint8_t* {
    constexpr int k = decltype(s)::value % kStages;
    if constexpr (k == 0) return a0;
    else if constexpr (k == 1) return a1;
    else if constexpr (k == 2) return a2;
    else return a3;
  };
  auto slot_b = [&](auto s) -> uint8_t* {
    constexpr int k = decltype(s)::value % kStages;
    if constexpr (k == 0) return b0;
    else if constexpr (k == 1) return b1;
    else if constexpr (k == 2) return b2;
    else return b3;
  };
  auto issue = [&](int t, auto s) {
    la.issue(l, t, slot_a(s));
    lb.issue(l, t, slot_b(s));
  };
  auto read = [&](auto s) {
    constexpr int k = decltype(s)::value;
    read_features<kAAcross>(l, slot_a(s), fa[k & 1]);
    read_rows<kBAcross, TN>(l, slot_b(s), fb[k & 1]);
  };
  auto ops = [&](auto s) {
    constexpr int k = decltype(s)::value & 1;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
        acc[tm][tn] = mfma16x16x32(fa[k][tm], fb[k][tn], acc[tm][tn]);
  };
  // step t, of slot s: the steady form (t + 4 < nk) has no conditions
  auto steady = [&](int t, auto s) {
    constexpr int k = decltype(s)::value;
    wait_vm<8>();
    wait_lgkm0();
    barrier();
    issue(t + 4, s);
    read(std::integral_constant<int, k + 1>{});
    ops(s);
    // the direct loads, then the reads one by one between the first ops, and no op moved
    // past the next barrier, whose wait would then find the matrix pipe empty
    constexpr int kReads = TM * (kAAcross ? 2 : 1) + TN * (kBAcross ? 2 : 1);
    constexpr int kOps = TM * TN;
    __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);       // VMEM
#pragma unroll
    for (int i = 0; i < (kReads < kOps ? kReads : kOps); ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // DS read
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto last = [&](int t, auto s) {
    constexpr int k = decltype(s)::value;
    if (t + 3 < nk) wait_vm<8>();
    else if (t + 2 < nk) wait_vm<4>();
    else wait_vm<0>();
    wait_lgkm0();
    barrier();
    if (t + 4 < nk) issue(t + 4, s);
    if (t + 1 < nk) read(std::integral_constant<int, k + 1>{});
    ops(s);
    __builtin_amdgcn_sched_barrier(0);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;

  issue(0, C0{});
  if (nk > 1) issue(1, C1{});
  if (nk > 2) issue(2, C2{});
  if (nk > 3) issue(3, C3{});
  if (nk > 3) wait_vm<12>();
  else if (nk == 3) wait_vm<8>();
  else if (nk == 2) wait_vm<4>();
  else wait_vm<0>();
  barrier();
  read(C0{});
  int t = 0;
  for (; t + 7 < nk; t += 4) {
    steady(t, C0{});
    steady(t + 1, C1{});
    steady(t + 2, C2{});
    steady(t + 3, C3{});
  }
  // 1 to 7 steps left
  last(t, C0{});
  if (t + 1 < nk) last(t + 1, C1{});
  if (t + 2 < nk) last(t + 2, C2{});
  if (t + 3 < nk) last(t + 3, C3{});
  if (t + 4 < nk) last(t + 4, C0{});
  if (t + 5 < nk) last(t + 5, C1{});
  if (t + 6 < nk) last(t + 6, C2{});
}

// ------------------------------------------------------------------ storing

__device__ __forceinline__ u32x4 bf16x8_of(const float* v) {
  u32x4 q;
  q.x = pack_bf16x2(v[0], v[1]);
  q.y = pack_bf16x2(v[2], v[3]);
  q.z = pack_bf16x2(v[4], v[5]);
  q.w = pack_bf16x2(v[6], v[7]);
  return q;
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<u32x4*>(p) = bf16x8_of(v);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const u32x4 q = *reinterpret_cast<const u32x4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// the largest of v over the 4 lane groups of a column: 32 features
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}

struct Args {
  TrainRows r;
  Divider div;
  const uint16_t* w;    // the product's weights
  const uint16_t* in;   // its rows (x, act, dy or dh)
  uint16_t* act;
  uint16_t* dh;
  uint16_t* out;
  uint16_t* h;          // kept values: bf16, or codes
  uint8_t* scales;
};

// 8 neighbours of the kept values of one row: columns col .. col + 7 of 2I
template <bool kFp8>
__device__ __forceinline__ void keep8(const Args& a, size_t row, int col, const float* v,
                                      bool first, bool in) {
  const size_t at = row * (size_t)(2 * a.r.I) + col;
  if constexpr (kFp8) {
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = abs_max(most, v[j]);
    const int byte = scale_byte(column_max(most));   // every lane takes part
    if (in) {
      *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.h) + at) =
          pack_e4m3x8(v, inverse_scale(byte));
      if (first) a.scales[at / 32] = (uint8_t)byte;
    }
  } else {
    if (in) store8(a.h + at, v);
  }
}

template <bool kFp8>
__device__ __forceinline__ void kept8(const Args& a, size_t row, int col, float* v) {
  const size_t at = row * (size_t)(2 * a.r.I) + col;
  if constexpr (kFp8)
    unpack_e4m3x8(*reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.h) + at),
                  scale_of(a.scales[at / 32]), v);
  else
    load8(a.h + at, v);
}

// One item of the products over rows: features f0 .. of the tile, rows row0 .. row0 + n - 1 of
// expert e, n <= 64 TN.
template <Op kOp, bool kFp8, int TN, class Sm>
__device__ __forceinline__ void rows_item(const Args& a, const Lane& l, Sm& sm, int e, int f0,
                                          int64_t row0, int n) {
  const int H = a.r.H, I = a.r.I;
  f32x4 acc[TM][TN];
  Along rows;
  // rows: of x by token, or of the row buffer
  const int Kdim = kOp == kGateUp || kOp == kDAct ? H : kOp == kDown ? I : 2 * I;
  const uint32_t row_bytes = (uint32_t)Kdim * 2;
  if (kOp == kGateUp && a.r.counts) {
    rows.set(l, make_rsrc(a.in, (uint32_t)a.r.tokens * row_bytes), [&](int j) -> uint32_t {
      const int t = sm.tok[j];
      return t < 0 ? kOutside : (uint32_t)t * row_bytes;
    });
  } else {
    rows.set(l, make_rsrc(a.in + (size_t)row0 * Kdim, (uint32_t)n * row_bytes),
             [&](int j) -> uint32_t { return j < n ? (uint32_t)j * row_bytes : kOutside; });
  }
  const int nk = Kdim / kStep;
  if constexpr (kOp == kGateUp || kOp == kDown) {
    Along feats;
    const size_t mat = (kOp == kGateUp ? (size_t)2 : (size_t)1) * I * H;
    const uint16_t* w = a.w + (size_t)e * mat;
    feats.set(l, make_rsrc(w, (uint32_t)(mat * 2)), [&](int r) -> uint32_t {
      const int tm = (r >> 4) & 7, c = (r >> 2) & 3, j = r & 3;
      int f;
      if (kOp == kGateUp) {
        // of four MFMA tiles two are gate's and two up's, of the same 32 columns
        f = f0 + 64 * (r >> 7) + (feature(0, tm & 1, c, j) + 32 * (tm >> 2));
        if (f >= I) return kOutside;
        if (tm & 2) f += I;
      } else {
        f = f0 + feature(r >> 7, tm, c, j);
        if (f >= H) return kOutside;
      }
      return (uint32_t)f * row_bytes;
    });
    product<false, false, TN>(l, sm.a[0], sm.a[1], sm.a[2], sm.a[3], sm.b[0], sm.b[1],
                             sm.b[2], sm.b[3], feats, rows, nk, acc);
  } else {
    Across feats;
    const int F = kOp == kDAct ? I : H;
    feats.set(l, a.w + (size_t)e * Kdim * F, (uint32_t)F * 2, Kdim, f0);
    product<true, false, TN>(l, sm.a[0], sm.a[1], sm.a[2], sm.a[3], sm.b[0], sm.b[1],
                             sm.b[2], sm.b[3], feats, rows, nk, acc);
  }

#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    const int j = (l.wn + 4 * tn) * 16 + l.m;
    const bool in = j < n;
    const size_t row = (size_t)(row0 + j);
    if constexpr (kOp == kGateUp) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = f0 + 64 * l.wm + 32 * q + 8 * l.g;
        float gv[8], uv[8], av[8];
        in_order(l.g, acc[4 * q][tn], acc[4 * q + 1][tn], gv);
        in_order(l.g, acc[4 * q + 2][tn], acc[4 * q + 3][tn], uv);
#pragma unroll
        for (int x = 0; x < 8; ++x) av[x] = silu(gv[x]) * uv[x];
        const bool here = in && i < I;
        keep8<kFp8>(a, row, i, gv, l.g == 0, here);
        keep8<kFp8>(a, row, I + i, uv, l.g == 0, here);
        if (here) store8(a.act + row * I + i, av);
      }
    } else {
#pragma unroll
      for (int p = 0; p < TM / 2; ++p) {
        const int f = f0 + 128 * l.wm + 32 * p + 8 * l.g;
        float v[8];
        in_order(l.g, acc[2 * p][tn], acc[2 * p + 1][tn], v);
        if constexpr (kOp == kDAct) {
          if (in && f < I) {
            float gv[8], uv[8], av[8], dg[8], du[8];
            kept8<kFp8>(a, row, f, gv);
            kept8<kFp8>(a, row, I + f, uv);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float s = sigmoid(gv[x]), gs = gv[x] * s;
              av[x] = gs * uv[x];
              dg[x] = v[x] * uv[x] * (s * (1.0f + gv[x] * (1.0f - s)));
              du[x] = v[x] * gs;
            }
            store8(a.act + row * I + f, av);
            store8(a.dh + row * (2 * (size_t)I) + f, dg);
            store8(a.dh + row * (2 * (size_t)I) + I + f, du);
          }
        } else {
          if (in && f < H) store8(a.out + row * H + f, v);
        }
      }
    }
  }
}

// the rows of expert e, inside the row buffers whatever the plan says
__device__ __forceinline__ int expert_rows(const TrainRows& r, int e, int64_t* row0) {
  *row0 = 0;
  if (!r.counts || r.tokens == 0) return (int)r.tokens;   // without tokens the plan holds nothing
  const int64_t off = r.offsets[e];
  const int64_t n = r.counts[e];
  if (off < 0 || off >= r.rows) return 0;
  *row0 = off;
  return (int)(n < 0 ? 0 : n < r.rows - off ? n : r.rows - off);
}

// Persistent workgroups over (expert, feature tile, span of up to 256 rows), spans fastest, one
// run of items per XCD (workgroup b runs on XCD b % 8), so that the spans that share a weight
// tile run side by side on one L2.
template <Op kOp, bool kFp8>
__global__ __launch_bounds__(kThreads, 1) void rows_kernel(Args a) {
  __shared__ __attribute__((aligned(1024))) Smem<kOp == kDAct || kOp == kDX, false> sm;
  const Lane l;
  const int nexp = a.r.counts ? a.r.E : 1;
  const int per_tile = kOp == kGateUp ? kTile / 2 : kTile;
  const int F = kOp == kGateUp || kOp == kDAct ? a.r.I : a.r.H;
  const int ntiles = (F + per_tile - 1) / per_tile;
  {
    int u = 0;
    if (l.tid < nexp) {
      int64_t row0;
      u = ntiles * ((expert_rows(a.r, l.tid, &row0) + kTile - 1) / kTile);
    }
    int incl = u;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(incl, d, kWave);
      if (l.lane >= d) incl += v;
    }
    if (l.lane == kWave - 1) sm.wsum[l.wave] = incl;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) before += v < l.wave ? sm.wsum[v] : 0;
    if (l.tid < nexp) sm.pre[l.tid + 1] = before + incl;
    if (l.tid == 0) sm.pre[0] = 0;
    __syncthreads();
  }
  const int total = __builtin_amdgcn_readfirstlane(sm.pre[nexp]);
  const int nc = (int)gridDim.x / 8;
  const int xcd = (int)blockIdx.x % 8, c = (int)blockIdx.x / 8;
  const int per = (total + 7) / 8;
  const int hi = min(total, (xcd + 1) * per);
  for (int it = xcd * per + c; it < hi; it += nc) {
    int lo = 0, up = nexp;   // the last expert with pre[e] <= it
    while (up - lo > 1) {
      const int mid = (lo + up) >> 1;
      if (__builtin_amdgcn_readfirstlane(sm.pre[mid]) <= it) lo = mid;
      else up = mid;
    }
    const int e = lo;
    int64_t first;
    const int n = __builtin_amdgcn_readfirstlane(expert_rows(a.r, e, &first));
    const int spans = (n + kTile - 1) / kTile;
    const int at = it - __builtin_amdgcn_readfirstlane(sm.pre[e]);
    const int tile = at / spans, span = at - tile * spans;
    const int64_t row0 = __builtin_amdgcn_readfirstlane((int)first) + (int64_t)span * kTile;
    const int nrows = min(kTile, n - span * kTile);
    if (kOp == kGateUp && a.r.counts) {
      __syncthreads();   // the previous item's loads have their tokens
      if (l.tid < kTile) {
        const int p = l.tid < nrows ? a.r.sorted_ids[row0 + l.tid] : -1;
        const uint32_t t = divided(a.div, (uint32_t)p & 0x7fffffffu);
        sm.tok[l.tid] = p >= 0 && t < (uint64_t)a.r.tokens ? (int)t : -1;
      }
      __syncthreads();
    }
    const int f0 = tile * per_tile;
    if (nrows > 128) rows_item<kOp, kFp8, 4>(a, l, sm, e, f0, row0, nrows);
    else if (nrows > 64) rows_item<kOp, kFp8, 2>(a, l, sm, e, f0, row0, nrows);
    else rows_item<kOp, kFp8, 1>(a, l, sm, e, f0, row0, nrows);
  }
}

// Gradients of the weights: [E][N][M] from rows of M features (the side along memory of the
// result) and rows of N.  An item is one 256 x 256 tile of one expert's matrix, its
// contraction the expert's rows; an expert without rows gets zeros.
struct WeightArgs {
  TrainRows r;
  const uint16_t* m_rows;
  const uint16_t* n_rows;
  void* out;
  int M, N;
};

template <class TOut>
__global__ __launch_bounds__(kThreads, 1) void weights_kernel(WeightArgs a) {
  __shared__ __attribute__((aligned(1024))) Smem<true, true> sm;
  const Lane l;
  const int E = a.r.counts ? a.r.E : 1;
  const int tm_n = (a.M + kTile - 1) / kTile, tn_n = (a.N + kTile - 1) / kTile;
  const int64_t each = (int64_t)tm_n * tn_n, total = E * each;
  const int nc = (int)gridDim.x / 8;
  const int xcd = (int)blockIdx.x % 8, c = (int)blockIdx.x / 8;
  const int64_t per = (total + 7) / 8;
  const int64_t hi = total < (xcd + 1) * per ? total : (xcd + 1) * per;
  for (int64_t it = xcd * per + c; it < hi; it += nc) {
    // tiles in bands of 4 along N, so that those at work together share their operands
    const int e = (int)(it / each);
    const int at = (int)(it - e * each);
    const int band = at / (4 * tm_n), in_band = at - band * 4 * tm_n;
    const int width = min(4, tn_n - 4 * band);
    const int tm = in_band / width, tn = 4 * band + in_band - tm * width;
    const int m0 = tm * kTile, n0 = tn * kTile;
    int64_t first;
    const int n = __builtin_amdgcn_readfirstlane(expert_rows(a.r, e, &first));
    const int64_t row0 = __builtin_amdgcn_readfirstlane((int)first);
    const int nk = (n + kStep - 1) / kStep;
    f32x4 acc[TM][4];
    Across nr;
    nr.set(l, a.n_rows + (size_t)row0 * a.N, (uint32_t)a.N * 2, n, n0);
    Across mr;
    mr.set(l, a.m_rows + (size_t)row0 * a.M, (uint32_t)a.M * 2, n, m0);
    product<true, true, 4>(l, sm.a[0], sm.a[1], sm.a[2], sm.a[3], sm.b[0], sm.b[1], sm.b[2],
                           sm.b[3], mr, nr, nk, acc);
    TOut* out = static_cast<TOut*>(a.out) + (size_t)e * a.M * a.N;
#pragma unroll
    for (int tn4 = 0; tn4 < 4; ++tn4) {
      const int j = n0 + (l.wn + 4 * tn4) * 16 + l.m;
#pragma unroll
      for (int p = 0; p < TM / 2; ++p) {
        const int f = m0 + 128 * l.wm + 32 * p + 8 * l.g;
        float v[8];
        in_order(l.g, acc[2 * p][tn4], acc[2 * p + 1][tn4], v);
        if (j < a.N && f < a.M) store8(out + (size_t)j * a.M + f, v);
      }
    }
  }
}

// compute units of the device current at the first call, as a multiple of the 8 XCDs
int workgroups() {
  static const int n = [] {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        cus < 8)
      cus = 256;
    return cus / 8 * 8;
  }();
  return n;
}

unsigned grid_of(int64_t items) {
  const int64_t g = (items + 7) / 8 * 8;
  return (unsigned)(g < workgroups() ? (g < 8 ? 8 : g) : workgroups());
}

Divider divider(int K) {
  Divider d{0, 0};
  while ((1 << d.shift) < K) ++d.shift;
  d.mul = (uint32_t)((((uint64_t)1 << (31 + d.shift)) + K - 1) / K);
  return d;
}

template <Op kOp, bool kFp8>
hipError_t launch_rows(const Args& a, hipStream_t s) {
  const int per_tile = kOp == kGateUp ? kTile / 2 : kTile;
  const int F = kOp == kGateUp || kOp == kDAct ? a.r.I : a.r.H;
  // spans: one for each 256 rows, and a short one an expert
  const int64_t pairs = a.r.counts ? a.r.tokens * a.r.K : a.r.tokens;
  const int64_t spans = pairs / kTile + (a.r.counts ? (a.r.E < pairs ? a.r.E : pairs) : 1);
  const int64_t items = spans * ((F + per_tile - 1) / per_tile);
  if (pairs == 0) return hipSuccess;
  if (items >= (int64_t)1 << 31) return hipErrorInvalidValue;
  hipLaunchKernelGGL((rows_kernel<kOp, kFp8>), dim3(grid_of(items)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_weights(const WeightArgs& a, bool f32, hipStream_t s) {
  const int64_t items = (int64_t)(a.r.counts ? a.r.E : 1) * ((a.M + kTile - 1) / kTile) *
                        ((a.N + kTile - 1) / kTile);
  const dim3 grid(grid_of(items)), block(kThreads);
  if (f32) hipLaunchKernelGGL(weights_kernel<float>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(weights_kernel<uint16_t>, grid, block, 0, s, a);
  return hipGetLastError();
}

Args args_of(const TrainRows& r) {
  Args a{};
  a.r = r;
  a.div = divider(r.K);
  return a;
}

}  // namespace

hipError_t launch_train_gate_up(const TrainRows& r, const void* x, const void* w13,
                                const SavedRows& saved, uint16_t* act, hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w13);
  a.in = static_cast<const uint16_t*>(x);
  a.act = act;
  a.h = static_cast<uint16_t*>(saved.h);
  a.scales = saved.scales;
  return saved.fp8 ? launch_rows<kGateUp, true>(a, s) : launch_rows<kGateUp, false>(a, s);
}

hipError_t launch_train_down(const TrainRows& r, const void* w2, const uint16_t* act, void* y,
                             hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w2);
  a.in = act;
  a.out = static_cast<uint16_t*>(y);
  return launch_rows<kDown, false>(a, s);
}

hipError_t launch_train_dact(const TrainRows& r, const void* w2, const void* dy,
                             const SavedRows& saved, uint16_t* act, uint16_t* dh, hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w2);
  a.in = static_cast<const uint16_t*>(dy);
  a.act = act;
  a.dh = dh;
  a.h = static_cast<uint16_t*>(saved.h);
  a.scales = saved.scales;
  return saved.fp8 ? launch_rows<kDAct, true>(a, s) : launch_rows<kDAct, false>(a, s);
}

hipError_t launch_train_dx(const TrainRows& r, const void* w13, const uint16_t* dh, void* dx,
                           hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w13);
  a.in = dh;
  a.out = static_cast<uint16_t*>(dx);
  return launch_rows<kDX, false>(a, s);
}

hipError_t launch_train_dw13(const TrainRows& r, const uint16_t* x_rows, const uint16_t* dh,
                             void* dw13, bool f32, hipStream_t s) {
  return launch_weights(WeightArgs{r, x_rows, dh, dw13, r.H, 2 * r.I}, f32, s);
}

hipError_t launch_train_dw2(const TrainRows& r, const uint16_t* act, const void* dy, void* dw2,
                            bool f32, hipStream_t s) {
  return launch_weights(WeightArgs{r, act, static_cast<const uint16_t*>(dy), dw2, r.I, r.H}, f32, s);
}

}  // namespace moe
