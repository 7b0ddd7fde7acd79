// The experts' products of a training step on gfx950.
//
// For a row of expert e with token x, gate and up values (g, u) = W13 x, a = silu(g) * u and
// y = W2 a.  From dy, the gradient of y:
//
//   da = W2^T dy     dg = da * u * s (1 + g (1 - s)), du = da * g s     with s = 1 / (1 + e^-g)
//   dx = W13^T (dg, du)     dW13 = sum over the expert's rows of (dg, du) x^T
//   dW2 = sum over the expert's rows of dy a^T
//
// Sums, s and the gradients dg and du are fp32.  a, dg and du are rounded to bf16 once, as operands
// of the next product (bf16 is what the matrix instruction takes; fp32 operands would cost 16 times
// the time), g and u as the caller has them kept, partial sums not at all.
//
// Six products in three forms, by which index runs along memory.  In the forward both operands
// have the contraction there ("along"); in da and dx the weights have it across their rows; in
// the weights' gradients both operands do, since the contraction is over rows ("across").
//
// All run on one tile, 256 features x 256 rows (or features), by 8 wavefronts as 2 x 4 of
// 128 x 64 with 16x16x32 bf16 MFMAs, in blocks of 64 of the contraction.  A block is four units
// of 16 KB, the halves of either operand, each with two slots in LDS that direct loads fill.  A
// wavefront takes a block in four phases, a quarter of its tile each (16 MFMAs), in the order
// (A0,Bf) (A0,Bg) (A1,Bg) (A1,Bf), f and g changing places with the block: each phase needs one
// set of fragments that is not in registers yet, and refills the slot that the phase before has
// read.  So a load has seven phases to land, and 96 KB a CU are in flight.
// (Blocks of 32 in a ring of four stages read 64 bytes of a row at a time, half a line, and the
// 32 KB of L1 hold the other half no longer than a step: Mixtral-shaped gate/up of 4096 tokens
// at 985 TFLOP/s.)
//
//   along   a unit's 128 rows of 128 bytes; 16-byte segment s of row r at s ^ ((r >> 1) & 7);
//           a fragment is one 16-byte read
//   across  a unit's 64 rows of 256 bytes in 16 chunks of four, k, k + 8, k + 16, k + 24, with
//           64 bytes between the chunks; the segments of the second and fourth at s ^ 3.  A
//           fragment is two transposing 8-byte reads (a lane's 4 values of one column from 4
//           rows): the gaps put the 4 rows that a read takes together in different quarters of
//           the banks, the swizzle k and k + 8 in different halves of those, so that 32 lanes
//           meet every bank once
//
// Direct loads go through buffer descriptors, whose range check (of the lane's and the scalar
// offset together) writes zeros for what lies outside: rows past an expert's last one, features
// past an edge that is no multiple of 256, blocks past the end.  So every block runs the same
// instructions, and nothing outside a matrix is read.  The blocks of a workgroup's items are one
// stream: the loads of an item begin while the one before is worked on.
//
// Measured (kernel times; the matrix pipe busy, at the clock that the power limit leaves, 1.8 to
// 2.1 of 2.4 GHz).  Bound by the matrix pipe and, between its turns, by barriers and LDS:
//   8 experts of 4096 x 14336, 4096 tokens, K = 2: gate/up 1.77 ms, 1.09 PFLOP/s (61%); down 1.01,
//   0.95; da 1.05, 0.91; dx 1.95, 0.99 (55%); both weights' gradients 2.74, 1.05 (54%); these and
//   dx in one launch 4.40 to 4.61, 1.04 to 1.09 (57%)
//   one expert of 7168 x 2048, 4096 rows: gate/up 186 to 211 us, 1.14 to 1.29 PFLOP/s (62%)
// Bound by memory, 64 experts of 3584 x 2560, 128 tokens, K = 8: da 293 us, 4.0 TB/s (the gradients
// written before still leave the caches); dx 426, 5.5; the weights' gradients 840 to 900 us, 3.5 GB
// of them (stores alone 646, the rest alone 405: a workgroup's stores and loads wait for each
// other in one order); in one launch 1.21 to 1.31 ms
//
// The features of a tile are dealt to MFMA rows so that a lane's sums of two neighbouring MFMA
// tiles are 8 neighbours in memory (feature(): 16-byte stores, 64 bytes of a row side by side).
#include <type_traits>

#include "pack.h"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kTile = 256;                // features, and rows, of a tile
constexpr int kHalf = 128;
constexpr int kBlock = 64;                // contraction of a block
constexpr int kChunk = 4 * kHalf * 2 + 64;   // four rows and a gap, across
constexpr int kUnit = 16 * kChunk;        // bytes of a unit (along: 16 KB of them)
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxE = 256;
constexpr int TM = 8, TN = 4;             // a wavefront's MFMA tiles of features, and of rows
constexpr uint32_t kOutside = 0xfffffff0u;    // an offset that every descriptor refuses

// The units: each a variable of its own, see stream()
#define TRAIN_UNITS                                                                          \
  __shared__ __attribute__((aligned(128))) uint8_t a00[kUnit], a01[kUnit], a10[kUnit], a11[kUnit]; \
  __shared__ __attribute__((aligned(128))) uint8_t b00[kUnit], b01[kUnit], b10[kUnit], b11[kUnit]; \
  const Units units{a00, a01, a10, a11, b00, b01, b10, b11}

// [half][slot] of the features' operand, and of the rows'
struct Units {
  uint8_t *a00, *a01, *a10, *a11, *b00, *b01, *b10, *b11;
};

// what a job keeps in LDS: the experts' rows, and its own order of the items
struct Smem {
  int first[kMaxE], rows[kMaxE];
  int pre[kMaxE + 1], pre_light[kMaxE + 1];
  int wsum[2][kWaves];
  int claim[4];   // WeightsJob: its next items
};

enum Op { kGateUp, kDown, kDAct, kDX };
// The contraction whole, or in parts whose sums are kept by row, or by pair
enum Split { kWhole, kByRow, kByPair };

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void* LdsPtr;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* LdsVec4;

// A value that is the same in every lane, in a scalar register: descriptors are built of them
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ const uint8_t* uniform(const void* p) {
  const uint64_t v = (uint64_t)p;
  return (const uint8_t*)((uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v));
}

__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(uniform(p)), 0, uniform(bytes),
                                           0x00020000);
}

__device__ __forceinline__ void load_lds16(Rsrc r, uint32_t lane_off, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 16, (int)lane_off, (int)uniform(off), 0,
                                           0);
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

// what a lane is, in the workgroup and in an MFMA
struct Lane {
  int tid, lane, wave, wm, wn, m, g;
  __device__ __forceinline__ explicit Lane(int thread) {
    tid = thread;
    lane = tid & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(tid / kWave);   // so that its indices stay scalar
    wm = wave >> 2;
    wn = wave & 3;
    m = lane & 15;
    g = lane >> 4;
  }
  // The same, worked out again: what is used between items alone keeps no register over the
  // product, whose sums and fragments take 224 of 256.
  __device__ __forceinline__ Lane again() const {
    int t = tid;
    asm volatile("" : "+v"(t));
    return Lane(t);
  }
};

// Feature (of a half's 64 of wavefront row wm) of MFMA tile t (of 4), row 4c + j: a pair of tiles
// t, t ^ 1 holds 32 neighbours, and lane group c of the two 8 neighbours, 4 in each.  Which tile
// has the first 4 alternates with c, so that the transposing reads of one tile use both halves
// of the 16-byte segments and with them every bank.
__device__ __forceinline__ int feature(int t, int c, int j) {
  return 32 * (t >> 1) + 8 * c + 4 * ((c ^ t) & 1) + j;
}

// The 8 sums of a lane in a pair of tiles, in the order of their features
__device__ __forceinline__ void in_order(int g, f32x4 even, f32x4 odd, float* v) {
  const f32x4 lo = g & 1 ? odd : even, hi = g & 1 ? even : odd;
  v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
  v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
}

// the row of a lane's sums in MFMA tile tn
__device__ __forceinline__ int tile_row(const Lane& l, int tn) { return (l.wn + 4 * tn) * 16 + l.m; }

// ------------------------------------------------------------------ filling a unit
//
// A wavefront's two direct loads j = 0, 1 fill KB (or chunk) 2 wave + j of a unit's 16.  at()
// sets the block that issue() loads; `live` false: zeros.  Rows and features that the result has
// no place for may hold anything (their sums are not stored), rows of the contraction that are
// not there hold zeros.

// Contraction along memory: load j has rows 16 wave + 8 j .. + 7 of the half, 8 lanes a row.
__device__ __forceinline__ int along_row(const Lane& l, int j) {
  return 16 * l.wave + 8 * j + (l.lane >> 3);
}
__device__ __forceinline__ uint32_t along_seg(const Lane& l, int j) {
  return (uint32_t)(((l.lane & 7) ^ ((4 * j + (l.lane >> 4)) & 7)) << 4);   // (row >> 1) & 7
}

struct Along {
  const uint8_t* base;
  uint32_t bytes, half, off[2], k, n;
  // row_off(r): the byte offset of row r of the first half; the second half's are `half_bytes`
  // further
  template <class F>
  __device__ __forceinline__ void set(const Lane& l, const void* p, uint32_t all, uint32_t half_bytes,
                                      F row_off) {
    base = uniform(p);
    bytes = uniform(all);
    half = uniform(half_bytes);
#pragma unroll
    for (int j = 0; j < 2; ++j) off[j] = row_off(along_row(l, j)) + along_seg(l, j);
  }
  __device__ __forceinline__ void at(int block, bool live) {
    k = (uint32_t)block * (kBlock * 2);
    n = uniform(live ? bytes : 0);
  }
  __device__ __forceinline__ void issue(const Lane& l, int h, uint8_t* unit) const {
    const Rsrc r = make_rsrc(base, n);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      load_lds16(r, off[j], k + (h ? half : 0), unit + (2 * l.wave + j) * 1024);
  }
};

// The same with rows of their own places.
struct Gathered {
  const uint8_t* base;
  uint32_t bytes, off[2][2], k, n;
  // row_off(r): the byte offset of the operand's row r, or kOutside
  template <class F>
  __device__ __forceinline__ void set(const Lane& l, const void* p, uint32_t all, F row_off) {
    base = uniform(p);
    bytes = uniform(all);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t o = row_off(kHalf * h + along_row(l, j));
        off[h][j] = o == kOutside ? o : o + along_seg(l, j);
      }
  }
  __device__ __forceinline__ void at(int block, bool live) {
    k = (uint32_t)block * (kBlock * 2);
    n = uniform(live ? bytes : 0);
  }
  __device__ __forceinline__ void issue(const Lane& l, int h, uint8_t* unit) const {
    const Rsrc r = make_rsrc(base, n);
#pragma unroll
    for (int j = 0; j < 2; ++j) load_lds16(r, off[h][j], k, unit + (2 * l.wave + j) * 1024);
  }
};

// Contraction across memory: `rows` rows of `row_bytes`, the tile's features from f0 on.  Chunk q
// has rows (q & 7) + 32 (q >> 3) and the three that follow 8 apart, 16 lanes a row.
struct Across {
  const uint8_t* base;
  uint32_t off, row_bytes, col, left;
  int rows;
  __device__ __forceinline__ void set(const Lane& l, const void* p, uint32_t bytes, int n, int f0) {
    base = uniform(p);
    row_bytes = uniform(bytes);
    rows = uniform(n);
    col = uniform((uint32_t)f0 * 2);
    const uint32_t row = (uint32_t)(((2 * l.wave) & 7) + 32 * (l.wave >> 2) + 8 * l.g);
    off = row * bytes + (uint32_t)((l.lane & 15) ^ (3 * (l.g & 1))) * 16;
  }
  // The descriptor holds the block's rows alone: any number of them, of matrices of any size,
  // and the rest zeros.  Blocks come in order: the base moves on with them.
  __device__ __forceinline__ void at(int block, bool live) {
    if (block > 0) base += (size_t)kBlock * row_bytes;
    left = uniform(live ? (uint32_t)min(kBlock, rows - block * kBlock) * row_bytes : 0);
  }
  __device__ __forceinline__ void issue(const Lane& l, int h, uint8_t* unit) const {
    const Rsrc r = make_rsrc(base, left);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      load_lds16(r, off, (uint32_t)j * row_bytes + col + (uint32_t)h * (kHalf * 2),
                 unit + (2 * l.wave + j) * kChunk);
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
//
// [ks]: the two steps of 32 of a block

// 8 values of the contraction for this lane's column, from byte `at` and 4 rows further
__device__ __forceinline__ u32x4 read_across(const uint8_t* at) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsVec4)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsVec4)(at + 4 * kChunk));
  const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
  return u32x4{a.x, a.y, b.x, b.y};
}

// 4 tiles of features
template <bool kIsAcross>
__device__ __forceinline__ void read_features(const Lane& l, const uint8_t* unit, u32x4 (&f)[2][4]) {
  if constexpr (kIsAcross) {
    const int r = l.m >> 2, c = l.m & 3;   // the row and the 4 features this lane points at
    const int at = r * kChunk + l.g * (kHalf * 2) + l.wm * 128 + ((c ^ (3 * (l.g & 1))) << 4) +
                   ((c & 1) << 3);
    const uint8_t* even = unit + at;
    const uint8_t* odd = unit + (at ^ 8);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f[ks][t] = read_across((t & 1 ? odd : even) + (t >> 1) * 64 + ks * 8 * kChunk);
  } else {
    const int at = (l.wm * 64 + l.m) * 128 + ((l.g ^ ((l.m >> 1) & 7)) << 4);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f[ks][t] = *reinterpret_cast<const u32x4*>(unit + (at ^ (ks * 64)) + t * 2048);
  }
}

// 2 tiles of rows
template <bool kIsAcross>
__device__ __forceinline__ void read_rows(const Lane& l, const uint8_t* unit, u32x4 (&f)[2][2]) {
  if constexpr (kIsAcross) {
    const int r = l.m >> 2, c = l.m & 3;
    const int at = r * kChunk + l.g * (kHalf * 2) +
                   (((2 * l.wn + (c >> 1)) ^ (3 * (l.g & 1))) << 4) + ((c & 1) << 3);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t) f[ks][t] = read_across(unit + at + t * 128 + ks * 8 * kChunk);
  } else {
    const int at = (l.wn * 16 + l.m) * 128 + ((l.g ^ ((l.m >> 1) & 7)) << 4);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        f[ks][t] = *reinterpret_cast<const u32x4*>(unit + (at ^ (ks * 64)) + t * 8192);
  }
}

// ------------------------------------------------------------------ the stream
//
// Phase of block s    reads           refills (with s + 2)
//   0  (A0,Bf)        A0 of s         Bf
//   1  (A0,Bg)        Bg of s         A0
//   2  (A1,Bg)        A1 of s         Bg
//   3  (A1,Bf)        Bg of s + 1     A1
//
// A phase is two turns: loads and reads, then the 16 ops.  The wavefronts 4 .. 7 are a turn
// behind 0 .. 3, with whom they share the SIMDs, so that one wavefront of a SIMD has the matrix
// pipe while the other reads (with all eight in step, and reads a phase ahead of their use, the
// pipe stood still around each barrier: busy half the time, measured).  A barrier ends each turn.
// A slot is refilled in the phase after the one that reads it, when the wavefronts behind have
// read it too; what a phase reads has landed, for every wavefront, at the end of the turn of
// loads before: all but the last six units' loads, 12 of a wavefront.
//
// A job's items have an even number of blocks (a last one that is not worked on), so that slots
// and f, g are known at compile time.
//
// Each unit's slot is an LDS variable of its own, so that a read is known to wait for the loads
// into its own slot alone: the compiler otherwise has a transposing read wait for all of them
// (measured in a ring of four stages: 620 against 990 TFLOP/s).
//
// Job: kAAcross, kBAcross; first(), next(it), kEnd: the places of this workgroup's items;
// item(it); and of an item blocks(); two(): whether the rows' second half holds any; load(a, b):
// sets the loaders; store(acc).  kEmptyLast: no item with blocks comes after one without; claim()
// and claimed(): at the start and the end of an item (see WeightsJob); what claim() gives also goes
// to store().
template <class Job>
__device__ __forceinline__ void stream(const Lane& l, Job& job, const Units& u) {
  constexpr bool kAA = Job::kAAcross, kBA = Job::kBAcross;
  typename Job::A la;
  typename Job::B lb;
  using Z = std::integral_constant<int, 0>;
  using O = std::integral_constant<int, 1>;
  auto unit_a = [&](auto h, auto slot) __attribute__((always_inline)) -> uint8_t* {
    constexpr int k = 2 * decltype(h)::value + decltype(slot)::value;
    if constexpr (k == 0) return u.a00;
    else if constexpr (k == 1) return u.a01;
    else if constexpr (k == 2) return u.a10;
    else return u.a11;
  };
  auto unit_b = [&](auto h, auto slot) __attribute__((always_inline)) -> uint8_t* {
    constexpr int k = 2 * decltype(h)::value + decltype(slot)::value;
    if constexpr (k == 0) return u.b00;
    else if constexpr (k == 1) return u.b01;
    else if constexpr (k == 2) return u.b10;
    else return u.b11;
  };

  // the loads' place in the stream: block `at` of item `item`
  int item = job.first(), at = -1, blocks = 0, even = 0;
  if (item == Job::kEnd) return;
  auto enter = [&]() __attribute__((always_inline)) {
    const typename Job::Item x = job.item(item);
    blocks = job.blocks(x);
    even = (blocks + 1) & ~1;
    if (even > 0) job.load(l.again(), x, la, lb);
    else if (Job::kEmptyLast) item = Job::kEnd;
  };
  enter();
  // may_end: an item may end here
  auto advance = [&](auto may_end) __attribute__((always_inline)) {
    ++at;
    if constexpr (decltype(may_end)::value) {
      while (at >= even && item != Job::kEnd) {
        item = uniform(job.next(item));
        at = 0;
        if (item != Job::kEnd) enter();
      }
    }
    const bool live = item != Job::kEnd && at < blocks;
    la.at(at, live);
    lb.at(at, live);
  };

  u32x4 fa[2][4], fb[2][2][2];   // [ks][tile], [half][ks][tile]
  f32x4 acc[TM][TN];

  advance(std::true_type{});
  lb.issue(l, 0, u.b00);
  la.issue(l, 0, u.a00);
  lb.issue(l, 1, u.b10);
  la.issue(l, 1, u.a10);
  advance(std::false_type{});
  lb.issue(l, 1, u.b11);
  la.issue(l, 0, u.a01);
  lb.issue(l, 0, u.b01);
  la.issue(l, 1, u.a11);
  wait_vm<0>();
  barrier();
  read_rows<kBA>(l, u.b00, fb[0]);
  wait_lgkm0();
  barrier();

  auto ops = [&](auto ha, auto hb, auto first) __attribute__((always_inline)) {
    constexpr int i = decltype(ha)::value, j = decltype(hb)::value;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int tn = 0; tn < 2; ++tn)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          f32x4& c = acc[4 * i + t][2 * j + tn];
          c = mfma16x16x32(fa[ks][t], fb[j][ks][tn],
                           decltype(first)::value && ks == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : c);
        }
  };
  // the end of a turn of loads and reads, the ops, and the end of theirs
  auto work = [&](auto ha, auto hb, auto any, auto first, auto landed) __attribute__((always_inline)) {
    if constexpr (!decltype(landed)::value) wait_vm<12>();
    wait_lgkm0();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    if constexpr (decltype(any)::value) {
      __builtin_amdgcn_s_setprio(1);
      ops(ha, hb, first);
      __builtin_amdgcn_s_setprio(0);
    }
    __builtin_amdgcn_sched_barrier(0);
    barrier();
  };
  // a block in slot `s`, whose Bf is half s; `two`: its second half of rows is worked on;
  // `fresh`: one of an item's first two, whose loads have landed but those of the last two phases
  auto block = [&](auto s_c, auto two_c, auto fresh_c) __attribute__((always_inline)) {
    constexpr int s = decltype(s_c)::value, f = s;
    constexpr bool two = decltype(two_c)::value, fresh = decltype(fresh_c)::value;
    using S = std::integral_constant<int, s>;
    using N = std::integral_constant<int, s ^ 1>;
    using F = std::integral_constant<int, f>;
    using G = std::integral_constant<int, f ^ 1>;
    using DoF = std::integral_constant<bool, two || f == 0>;
    using DoG = std::integral_constant<bool, two || f == 1>;
    using First = std::integral_constant<bool, fresh && s == 0>;
    using Early = std::integral_constant<bool, fresh>;
    using Late = std::integral_constant<bool, fresh && s == 0>;
    advance(std::integral_constant<bool, s == 0>{});
    lb.issue(l, f, unit_b(F{}, S{}));
    read_features<kAA>(l, unit_a(Z{}, S{}), fa);
    work(Z{}, F{}, DoF{}, First{}, Early{});

    la.issue(l, 0, unit_a(Z{}, S{}));
    read_rows<kBA>(l, unit_b(G{}, S{}), fb[f ^ 1]);
    work(Z{}, G{}, DoG{}, First{}, Early{});

    lb.issue(l, f ^ 1, unit_b(G{}, S{}));
    read_features<kAA>(l, unit_a(O{}, S{}), fa);
    work(O{}, G{}, DoG{}, First{}, Late{});

    la.issue(l, 1, unit_a(O{}, S{}));
    read_rows<kBA>(l, unit_b(G{}, N{}), fb[f ^ 1]);
    work(O{}, F{}, DoF{}, First{}, Late{});
  };
  // the block of zeros (slot 1) that makes an odd number even: its refills and the read of the
  // next block's Bf, which was loaded a block before, three units ago
  auto hollow = [&]() __attribute__((always_inline)) {
    wait_vm<6>();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    barrier();
    advance(std::false_type{});
    lb.issue(l, 1, u.b11);
    la.issue(l, 0, u.a01);
    lb.issue(l, 0, u.b01);
    la.issue(l, 1, u.a11);
    read_rows<kBA>(l, u.b00, fb[0]);
    wait_vm<12>();
    wait_lgkm0();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    barrier();
  };
  using Yes = std::true_type;
  using No = std::false_type;
  auto work_item = [&](int n, auto two) __attribute__((always_inline)) {
    block(Z{}, two, Yes{});
    int b = 2;
    if (n > 1) {
      block(O{}, two, Yes{});
      for (; b + 1 < n; b += 2) {
        block(Z{}, two, No{});
        block(O{}, two, No{});
      }
      if (b < n) block(Z{}, two, No{});
    }
    if (n & 1) hollow();
  };

  for (int it = job.first(); it != Job::kEnd; it = job.next(it)) {
    const typename Job::Item x = job.item(it);
    const int n = job.blocks(x);
    const bool two = job.two(x);
    const typename Job::Claim later = job.claim(l, x);
    if (n == 0 || !two) {
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) acc[tm][tn] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (n > 0) {
      if (l.wm == 1) barrier();   // a turn behind
      if (two) work_item(n, Yes{});
      else work_item(n, No{});
      if (l.wm == 0) barrier();   // in step again, to store together
    }
    // what is in flight lands before the stores, so that an item's first phases wait for neither
    wait_vm<0>();
    job.claimed(l, it, later);
    if (Job::kEmptyLast && n == 0) {   // what is claimed is seen two items later
      wait_lgkm0();
      barrier();
    }
    job.store(l.again(), x, acc, later);
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vm<0>();   // no load into LDS outlives the workgroup
}

// ------------------------------------------------------------------ storing

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// two values as bf16, rounded to nearest even, in one instruction
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__device__ __forceinline__ u32x4 bf16x8_of(const float* v) {
  return u32x4{bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]),
               bf16x2_of(v[6], v[7])};
}

// The whole offset in the lane's register, none in a scalar one: after a 16-byte store with a
// scalar offset the next instruction may overwrite the data before its last lanes are read
// (seen as wrong values in lanes 12 .. 15 of 16), and the compiler keeps them apart without one.
__device__ __forceinline__ void store16(Rsrc r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, 0);
}

// A lane's 8 sums of a pair of tiles, in the order of their features, at byte off
__device__ __forceinline__ void store_pair(Rsrc r, uint32_t off, uint32_t d, bool odd, f32x4 a,
                                           f32x4 b, const uint16_t*) {
  const uint32_t a0 = bf16x2_of(a.x, a.y), a1 = bf16x2_of(a.z, a.w);
  const uint32_t b0 = bf16x2_of(b.x, b.y), b1 = bf16x2_of(b.z, b.w);
  store16(r, off + d, odd ? u32x4{b0, b1, a0, a1} : u32x4{a0, a1, b0, b1});
}
__device__ __forceinline__ void store_pair(Rsrc r, uint32_t off, uint32_t d, bool odd, f32x4 a,
                                           f32x4 b, const float*) {
  store16(r, off + d + (odd ? 16 : 0), __builtin_bit_cast(u32x4, a));
  store16(r, off + d + (odd ? 0 : 16), __builtin_bit_cast(u32x4, b));
}

// The tile at out, of rows of F values: `rows` of its rows and `cols` of its columns are there.
// Stores go through descriptors: a lane's own offset for all of them, and rows past the last
// refused by range.
template <class T>
__device__ __forceinline__ void store_tile(const Lane& l, const f32x4 (&acc)[TM][TN], T* out, int F,
                                           int rows, int cols) {
  constexpr uint32_t e = sizeof(T);
  const uint32_t row_bytes = (uint32_t)F * e;
  const uint32_t off = (uint32_t)(l.wn * 16 + l.m) * row_bytes + (uint32_t)(64 * l.wm + 8 * l.g) * e;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(out);
  // up to the end of the last row
  const uint32_t all = (uint32_t)(rows - 1) * row_bytes + (uint32_t)min(cols, kTile) * e;
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    if (64 * tn >= rows) break;   // few rows: the rest of the code is not even fetched
#pragma unroll
    for (int p = 0; p < TM / 2; ++p) {
      const int f = kHalf * (p >> 1) + 32 * (p & 1);
      const Rsrc r = make_rsrc(base, f + 64 * l.wm < cols ? all : 0);
      store_pair(r, off + (uint32_t)f * e, (uint32_t)(64 * tn) * row_bytes, l.g & 1,
                 acc[2 * p][tn], acc[2 * p + 1][tn], out);
    }
  }
}

// The sums of a gate/up tile in fp32, out of rows of 2I values (its first column of gate), 64
// columns in each half of the tile, up's I further
__device__ __forceinline__ void store_gate_up(const Lane& l, const f32x4 (&acc)[TM][TN], float* out,
                                              int I, int rows, int cols) {
  const uint32_t row_bytes = (uint32_t)I * 8;
  const uint32_t off = (uint32_t)(l.wn * 16 + l.m) * row_bytes + (uint32_t)(32 * l.wm + 8 * l.g) * 4;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(out);
  const uint32_t all = (uint32_t)(rows - 1) * row_bytes + (uint32_t)(I + min(cols, kHalf)) * 4;
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    if (64 * tn >= rows) break;
#pragma unroll
    for (int p = 0; p < TM / 2; ++p) {   // gate, up, gate, up
      const Rsrc r = make_rsrc(base, 64 * (p >> 1) + 32 * l.wm < cols ? all : 0);
      store_pair(r, off + (uint32_t)(64 * (p >> 1) + (p & 1 ? I : 0)) * 4,
                 (uint32_t)(64 * tn) * row_bytes, l.g & 1, acc[2 * p][tn], acc[2 * p + 1][tn], out);
    }
  }
}

// The same of either tile by pair: out, of rows of F values, one for each pair, at column f0.  pair:
// that of this lane's rows; all: bytes of the rows together, at most half of kPartBytes.
constexpr uint32_t kNowhere = 0x80000000u;   // past any of them, and so are a row's columns after it
template <bool kGateUp>
__device__ __forceinline__ void store_by_pair(const Lane& l, const f32x4 (&acc)[TM][TN], float* out,
                                              uint32_t all, int F, int I, int f0, int rows,
                                              const int (&pair)[TN]) {
  constexpr int kWide = kGateUp ? 32 : 64;   // columns of a wavefront row in a half
  const int cols = (kGateUp ? I : F) - f0;
  const uint32_t row_bytes = (uint32_t)F * 4, col = (uint32_t)(kWide * l.wm + 8 * l.g) * 4;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(out + f0);
  all -= (uint32_t)f0 * 4;
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) {
    if (64 * tn >= rows) break;
    const uint32_t off = tile_row(l, tn) < rows ? (uint32_t)pair[tn] * row_bytes + col : kNowhere;
#pragma unroll
    for (int p = 0; p < TM / 2; ++p) {
      const int f = kGateUp ? 64 * (p >> 1) : kHalf * (p >> 1) + 32 * (p & 1);
      const Rsrc r = make_rsrc(base, f + kWide * l.wm < cols ? all : 0);
      store_pair(r, off, (uint32_t)(f + (kGateUp && (p & 1) ? I : 0)) * 4, l.g & 1, acc[2 * p][tn],
                 acc[2 * p + 1][tn], out);
    }
  }
}

__device__ __forceinline__ void bf16x8_to(u32x4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// a, and the gradients of g and u, from that of a
__device__ __forceinline__ void gradients(const float* da, const float* g, const float* u, float* a,
                                          float* dg, float* du) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float s = sigmoid(g[q]), gs = g[q] * s;
    a[q] = gs * u[q];
    dg[q] = da[q] * u[q] * (s * (1.0f + g[q] * (1.0f - s)));
    du[q] = da[q] * gs;
  }
}

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
  float* part;          // partial sums [splits][part_rows][features], where the contraction is split
  int splits;
  bool by_pair;         // part_rows: a row for each pair; else the rows of the buffers
  int64_t part_rows;
  int* counters;        // kDAct: of 8, cleared
};

// A row buffer from a span's first row on, of `cols` values a row, as a lane sees it: byte
// offsets of its row and columns in one descriptor, rows past the span's last refused by range.
template <class T>
struct Rows {
  const uint8_t* base;
  uint32_t row_bytes, all, off;
  // row, col: this lane's first; n: the span's rows
  __device__ __forceinline__ Rows(const T* p, size_t row0, int cols, int n, int row, int col) {
    row_bytes = (uint32_t)cols * (uint32_t)sizeof(T);
    base = reinterpret_cast<const uint8_t*>(p + row0 * cols);
    all = (uint32_t)n * row_bytes;
    off = (uint32_t)row * row_bytes + (uint32_t)col * (uint32_t)sizeof(T);
  }
  // `there`: the columns are no further than the edge (the same for the wavefront)
  __device__ __forceinline__ Rsrc rsrc(bool there) const { return make_rsrc(base, there ? all : 0); }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The gate and up values kept: two Rows of them, and of their scales
template <bool kFp8>
struct Kept {
  typedef typename std::conditional<kFp8, uint8_t, uint16_t>::type Code;
  Rows<Code> h;
  Rows<uint8_t> s;
  uint32_t up, up_s;   // from gate to up
  __device__ __forceinline__ Kept(const void* values, const uint8_t* scales, size_t row0, int I,
                                  int n, int row, int col)
      : h(static_cast<const Code*>(values), row0, 2 * I, n, row, col),
        s(scales, row0, 2 * I / 32, n, row, col / 32) {
    up = (uint32_t)I * (uint32_t)sizeof(Code);
    up_s = (uint32_t)I / 32;
  }
  // 8 neighbours of row + 64 tn, col + add (a multiple of 32), of gate (which 0) or up (1)
  __device__ __forceinline__ uint32_t at(int tn, int which) const {
    return (uint32_t)(64 * tn) * h.row_bytes + (which ? up : 0);
  }
  __device__ __forceinline__ uint32_t at_s(int tn, int which) const {
    return (uint32_t)(64 * tn) * s.row_bytes + (which ? up_s : 0);
  }
  __device__ __forceinline__ void keep(const Lane& l, bool there, int tn, int add, int which,
                                       const float* v) const {
    if constexpr (kFp8) {
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = abs_max(most, v[j]);
      const int byte = scale_byte(column_max(most));   // every lane takes part
      const uint2 c = pack_e4m3x8(v, inverse_scale(byte));
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{c.x, c.y}, h.rsrc(there), (int)(h.off + add),
                                            (int)uniform(at(tn, which)), 0);
      // one lane of the four that share a block has its offset, the others none
      __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, s.rsrc(there),
                                           (int)(l.g == 0 ? s.off + add / 32 : kOutside),
                                           (int)uniform(at_s(tn, which)), 0);
    } else {
      store16(h.rsrc(there), h.off + add * 2 + at(tn, which), bf16x8_of(v));
    }
  }
  struct Raw {
    u32x4 q;
    int byte;
  };
  __device__ __forceinline__ Raw read(bool there, int tn, int add, int which) const {
    Raw r;
    if constexpr (kFp8) {
      const u32x2 c = __builtin_amdgcn_raw_buffer_load_b64(h.rsrc(there), (int)(h.off + add),
                                                           (int)uniform(at(tn, which)), 0);
      r.q = u32x4{c.x, c.y, 0, 0};
      r.byte = __builtin_amdgcn_raw_buffer_load_b8(s.rsrc(there), (int)(s.off + add / 32),
                                                   (int)uniform(at_s(tn, which)), 0);
    } else {
      r.q = __builtin_amdgcn_raw_buffer_load_b128(h.rsrc(there), (int)(h.off + add * 2),
                                                  (int)uniform(at(tn, which)), 0);
      r.byte = 0;
    }
    return r;
  }
  __device__ __forceinline__ void values(const Raw& r, float* v) const {
    if constexpr (kFp8) unpack_e4m3x8(uint2{r.q.x, r.q.y}, scale_of(r.byte & 255), v);
    else bf16x8_to(r.q, v);
  }
};

// the rows of expert e, inside the row buffers whatever the plan says
__device__ __forceinline__ int expert_rows(const TrainRows& r, int e, int* row0) {
  *row0 = 0;
  if (!r.counts || r.tokens == 0) return (int)r.tokens;   // without tokens the plan holds nothing
  const int64_t off = r.offsets[e];
  const int64_t n = r.counts[e];
  if (off < 0 || off >= r.rows) return 0;
  *row0 = (int)off;
  return (int)(n < 0 ? 0 : n < r.rows - off ? n : r.rows - off);
}

// exclusive sums of u and of v over the threads, in pre_u[0 ..] and pre_v[0 ..], `values` of them
__device__ __forceinline__ void prefix(const Lane& l, int u, int v, int values, int* pre_u,
                                       int* pre_v, int (*wsum)[kWaves]) {
  int su = u, sv = v;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {   // both side by side: each step is a trip through LDS
    const int a = __shfl_up(su, d, kWave), b = __shfl_up(sv, d, kWave);
    if (l.lane >= d) {
      su += a;
      sv += b;
    }
  }
  if (l.lane == kWave - 1) {
    wsum[0][l.wave] = su;
    wsum[1][l.wave] = sv;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    if (w < l.wave) {
      su += wsum[0][w];
      sv += wsum[1][w];
    }
  if (l.tid < values) {
    pre_u[l.tid + 1] = su;
    pre_v[l.tid + 1] = sv;
  }
  if (l.tid == 0) pre_u[0] = pre_v[0] = 0;
  __syncthreads();
}

// the last i < n with pre[i] <= at (pre[0] is): a lane looks at four of them, all at once
__device__ __forceinline__ int last_at_most(const int* pre, int n, int at) {
  const int lane = threadIdx.x & (kWave - 1);
  int below = 0;
#pragma unroll
  for (int k = 0; k < kMaxE / kWave; ++k) {
    const int i = lane + k * kWave;
    below += __popcll(__ballot(i < n && pre[i] <= at));
  }
  return below - 1;
}

// One of the products over rows.  Items: (expert, feature tile, span of up to 256 rows), spans
// fastest, one run of them per XCD (workgroup b runs on XCD b % 8) that its workgroups take in
// turn, so that the spans that share a weight tile run side by side on one L2.  Experts of up to
// 128 rows come after all others, whose items take twice as long (Qwen2-shaped da and dx of 3001
// tokens with skewed routing: 517 -> 472 and 817 -> 742 us).  Where a run's last round would leave
// half the workgroups or more without an item, its items are cut into two of 128 rows (kCut; not
// where other work fills the round: a dense backward of 1024 rows of 4096 x 1024 104 -> 90 us).
//
// An item of up to 128 rows takes 0.8 of a whole one's time, of 32 rows hardly less (Mixtral-shaped
// dx: 540 and 520 against 670 us): its features come from memory and out of LDS all the same.  So
// 1056 rows an expert cost almost what 1280 do (dx of 8 experts 1.80 and 1.87 ms, of 1024 rows 1.38).
//
// kSplit: the contraction of every item is cut into a.splits parts, items of their own, whose sums
// go to a.part and are added by the finish kernels.
template <Op kOp, bool kFp8, Split kSplit, bool kCut = kSplit == kWhole>
struct RowsJob {
  static constexpr bool kAAcross = kOp == kDAct || kOp == kDX, kBAcross = false;
  static constexpr bool kEmptyLast = false;
  using A = typename std::conditional<kAAcross, Across, Along>::type;
  using B = typename std::conditional<kOp == kGateUp, Gathered, Along>::type;
  static constexpr int kEnd = -1;
  static constexpr int kFeatures = kOp == kGateUp ? kTile / 2 : kTile;   // of the result
  const Args& a;
  const Smem& sm;
  int nexp, step, xcd;
  int full0, full, cut, light0;   // this XCD's items: its first, whole, in two; its first short one
  int hi;

  struct Item {
    int e, f0, n, part, block0, blocks;   // blocks block0 .. of the contraction
    int64_t row0;
  };

  __device__ __forceinline__ RowsJob(const Args& args, const Lane& l, Smem& m) : a(args), sm(m) {
    nexp = a.r.counts ? a.r.E : 1;
    const int F = kOp == kGateUp || kOp == kDAct ? a.r.I : a.r.H;
    const int ntiles = (F + kFeatures - 1) / kFeatures;
    int n = 0, row0 = 0;
    if (l.tid < nexp) {
      n = expert_rows(a.r, l.tid, &row0);
      m.first[l.tid] = row0;
      m.rows[l.tid] = n;
    }
    prefix(l, n > kHalf ? ntiles * spans(n) : 0, n > 0 && n <= kHalf ? ntiles : 0, nexp, m.pre,
           m.pre_light, m.wsum);
    const int all = uniform(m.pre[nexp]), lights = uniform(m.pre_light[nexp]);
    step = (int)gridDim.x / 8;
    xcd = (int)blockIdx.x % 8;
    const int per = (all + 7) / 8, per_light = (lights + 7) / 8;
    full0 = xcd * per;
    light0 = xcd * per_light;
    full = max(0, min(per, all - full0));
    const int over = uniform(full % step);
    cut = kCut && 2 * over <= step ? over : 0;
    full -= cut;
    hi = full + 2 * cut + max(0, min(per_light, lights - light0));
    if (kSplit != kWhole) hi *= a.splits;
  }
  static __device__ __forceinline__ int spans(int n) { return (n + kTile - 1) / kTile; }

  __device__ __forceinline__ int first() const {
    const int it = (int)blockIdx.x / 8;
    return it < hi ? it : kEnd;
  }
  __device__ __forceinline__ int next(int it) const { return it + step < hi ? it + step : kEnd; }

  __device__ __forceinline__ Item item(int it) const {
    Item x;
    x.part = 0;
    if (kSplit != kWhole) {
      const int whole = uniform(it / a.splits);
      x.part = it - whole * a.splits;
      it = whole;
    }
    int tile, skip;
    if (it < full + 2 * cut) {
      const int half = it < full ? 0 : (it - full) & 1;
      const int q = full0 + (it < full ? it : full + ((it - full) >> 1));
      x.e = uniform(last_at_most(sm.pre, nexp, q));
      const int n = uniform(sm.rows[x.e]), each = spans(n);
      const int at = q - uniform(sm.pre[x.e]);
      tile = uniform(at / each);
      skip = (at - tile * each) * kTile + half * kHalf;
      x.n = max(0, min(it < full ? kTile : kHalf, n - skip));
    } else {
      const int q = light0 + it - full - 2 * cut;
      x.e = uniform(last_at_most(sm.pre_light, nexp, q));
      const int n = uniform(sm.rows[x.e]);
      tile = q - uniform(sm.pre_light[x.e]);
      x.n = n;
      skip = 0;
    }
    x.f0 = tile * kFeatures;
    x.row0 = uniform(sm.first[x.e]) + (int64_t)skip;
    const int all = x.n > 0 ? contraction() / kBlock : 0;
    x.block0 = 0;
    x.blocks = all;
    if (kSplit != kWhole) {
      const int each = uniform((all + a.splits - 1) / a.splits);
      x.block0 = min(all, x.part * each);
      x.blocks = min(each, all - x.block0);
    }
    return x;
  }

  // kByPair: the pairs of this lane's rows, loaded at the start of an item, used at its end (loaded
  // there, between the stores, each load waits for the stores before it)
  struct Claim {
    int pair[TN];
  };
  __device__ __forceinline__ Claim claim(const Lane& l, const Item& x) const {
    Claim c{};
    if constexpr (kSplit == kByPair) {
      const Rsrc ids = make_rsrc(a.r.sorted_ids + x.row0, (uint32_t)x.n * 4);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        c.pair[tn] = __builtin_amdgcn_raw_buffer_load_b32(ids, tile_row(l, tn) * 4, 0, 0);
    }
    return c;
  }
  __device__ __forceinline__ void claimed(const Lane&, int, const Claim&) const {}

  __device__ __forceinline__ int contraction() const {
    return kOp == kGateUp || kOp == kDAct ? a.r.H : kOp == kDown ? a.r.I : 2 * a.r.I;
  }
  __device__ __forceinline__ int blocks(const Item& x) const { return x.blocks; }
  __device__ __forceinline__ bool two(const Item& x) const { return x.n > kHalf; }

  __device__ __forceinline__ void load(const Lane& l, const Item& x, A& la, B& lb) const {
    const int H = a.r.H, I = a.r.I, K = contraction(), k0 = x.block0 * kBlock;
    const uint32_t row_bytes = (uint32_t)K * 2, k0_bytes = (uint32_t)k0 * 2;
    if constexpr (kOp == kGateUp) {
      if (a.r.counts) {
        lb.set(l, a.in + k0, (uint32_t)a.r.tokens * row_bytes - k0_bytes, [&](int j) -> uint32_t {
          const int p = j < x.n ? a.r.sorted_ids[x.row0 + j] : -1;
          const uint32_t t = divided(a.div, (uint32_t)p & 0x7fffffffu);
          return p >= 0 && t < (uint64_t)a.r.tokens ? t * row_bytes : kOutside;
        });
      } else {
        lb.set(l, a.in + (size_t)x.row0 * K + k0, (uint32_t)x.n * row_bytes - k0_bytes,
               [&](int j) -> uint32_t { return (uint32_t)j * row_bytes; });
      }
    } else {
      lb.set(l, a.in + (size_t)x.row0 * K + k0, (uint32_t)x.n * row_bytes - k0_bytes,
             kHalf * row_bytes, [&](int j) -> uint32_t { return (uint32_t)j * row_bytes; });
    }
    if constexpr (kAAcross) {
      const int F = kOp == kDAct ? I : H;
      la.set(l, a.w + ((size_t)x.e * K + k0) * F, (uint32_t)F * 2, K - k0, x.f0);
    } else {
      const size_t mat = (kOp == kGateUp ? (size_t)2 : (size_t)1) * I * H;
      const size_t before = (size_t)x.f0 * K + k0;
      // of a half's four MFMA tiles (gate/up) two are gate's and two up's, of the same 32 columns
      la.set(l, a.w + (size_t)x.e * mat + before, (uint32_t)((mat - before) * 2),
             kFeatures / 2 * row_bytes, [&](int r) -> uint32_t {
               const int wm = r >> 6, t = (r >> 4) & 3, c = (r >> 2) & 3, j = r & 3;
               const int f = kOp == kGateUp ? 32 * wm + feature(t & 1, c, j) + (t & 2 ? I : 0)
                                            : 64 * wm + feature(t, c, j);
               return (uint32_t)f * row_bytes;
             });
    }
  }

  __device__ __forceinline__ void store(const Lane& l, const Item& x, f32x4 (&acc)[TM][TN],
                                        const Claim& c) const {
    const int H = a.r.H, I = a.r.I;
    if (x.n == 0) return;
    if constexpr (kSplit == kByPair) {
      const int F = kOp == kGateUp ? 2 * I : kOp == kDAct ? I : H;
      store_by_pair<kOp == kGateUp>(l, acc, a.part + (size_t)x.part * a.part_rows * F,
                                    (uint32_t)a.part_rows * (uint32_t)F * 4, F, I, x.f0, x.n, c.pair);
      return;
    }
    if constexpr (kSplit == kByRow) {
      const int F = kOp == kGateUp ? 2 * I : kOp == kDAct ? I : H;
      float* part = a.part + ((size_t)x.part * a.r.rows + x.row0) * F + x.f0;
      if constexpr (kOp == kGateUp)
        store_gate_up(l, acc, part, I, x.n, I - x.f0);
      else
        store_tile(l, acc, part, F, x.n, F - x.f0);
      return;
    }
    if constexpr (kOp == kDown || kOp == kDX) {
      store_tile(l, acc, a.out + (size_t)x.row0 * H + x.f0, H, x.n, H - x.f0);
      return;
    }
    const int row = tile_row(l, 0);
    if constexpr (kOp == kGateUp) {
      const int i = x.f0 + 32 * l.wm + 8 * l.g;   // + 64 in the second half
      const Kept<kFp8> kept(a.h, a.scales, (size_t)x.row0, I, x.n, row, i);
      const Rows<uint16_t> act(a.act, (size_t)x.row0, I, x.n, row, i);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        if (64 * tn >= x.n) break;   // few rows: the rest of the code is not even fetched
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool there = x.f0 + 64 * h + 32 * l.wm < I;
          float gv[8], uv[8], av[8];
          in_order(l.g, acc[4 * h][tn], acc[4 * h + 1][tn], gv);
          in_order(l.g, acc[4 * h + 2][tn], acc[4 * h + 3][tn], uv);
#pragma unroll
          for (int q = 0; q < 8; ++q) av[q] = silu(gv[q]) * uv[q];
          kept.keep(l, there, tn, 64 * h, 0, gv);
          kept.keep(l, there, tn, 64 * h, 1, uv);
          store16(act.rsrc(there), act.off + 128 * h + (uint32_t)(64 * tn) * act.row_bytes,
                  bf16x8_of(av));
        }
      }
    } else if constexpr (kOp == kDAct) {
      const int f = x.f0 + 64 * l.wm + 8 * l.g;   // + 128 in the second half, + 32 in odd pairs
      const Kept<kFp8> kept(a.h, a.scales, (size_t)x.row0, I, x.n, row, f);
      const Rows<uint16_t> act(a.act, (size_t)x.row0, I, x.n, row, f);
      const Rows<uint16_t> dh(a.dh, (size_t)x.row0, 2 * I, x.n, row, f);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        if (64 * tn >= x.n) break;
        typename Kept<kFp8>::Raw gr[TM / 2], ur[TM / 2];
#pragma unroll
        for (int p = 0; p < TM / 2; ++p) {   // all of them in flight
          const int add = kHalf * (p >> 1) + 32 * (p & 1);
          const bool there = x.f0 + 64 * l.wm + add < I;
          gr[p] = kept.read(there, tn, add, 0);
          ur[p] = kept.read(there, tn, add, 1);
        }
#pragma unroll
        for (int p = 0; p < TM / 2; ++p) {
          const int add = kHalf * (p >> 1) + 32 * (p & 1);
          const bool there = x.f0 + 64 * l.wm + add < I;
          float v[8], gv[8], uv[8], av[8], dg[8], du[8];
          in_order(l.g, acc[2 * p][tn], acc[2 * p + 1][tn], v);
          kept.values(gr[p], gv);
          kept.values(ur[p], uv);
          gradients(v, gv, uv, av, dg, du);
          const uint32_t d = (uint32_t)(64 * tn) * act.row_bytes;
          store16(act.rsrc(there), act.off + 2 * add + d, bf16x8_of(av));
          store16(dh.rsrc(there), dh.off + 2 * add + 2 * d, bf16x8_of(dg));
          store16(dh.rsrc(there), dh.off + 2 * add + 2 * d + act.row_bytes, bf16x8_of(du));
        }
      }
    }
  }
};

template <Op kOp, bool kFp8, Split kSplit>
__global__ __launch_bounds__(kThreads, 1) void rows_kernel(Args a) {
  TRAIN_UNITS;
  __shared__ Smem sm;
  const Lane l(threadIdx.x);
  if (kOp == kDAct && blockIdx.x == 0 && l.tid < 8) a.counters[l.tid] = 0;   // see WeightsJob
  RowsJob<kOp, kFp8, kSplit> job(a, l, sm);
  stream(l, job, units);
}

// Gradients of the weights: [E][N][M] from rows of M features (the side along memory of the
// result) and rows of N.  An item is one 256 x 256 tile of one expert's matrix, its
// contraction the expert's rows; an expert without rows gets zeros.
//
// Experts come by falling numbers of rows, those without any last, the tiles of each dealt to the
// 8 XCDs in runs of equal length, so that skewed routing leaves no XCD with the busy experts and
// the short items fill in at the end (contiguous experts per XCD: Qwen2-shaped dW13 of 3001 tokens
// with skewed routing 2.4 ms).
// Both matrices' gradients are one launch, with one end: per expert dW13's tiles, then dW2's.
struct WeightArgs {
  TrainRows r;
  struct Product {
    const uint16_t* m_rows;
    const uint16_t* n_rows;
    void* out;
    int M, N;
    int64_t part;   // values of the result; splits > 1: out is [splits][that]
  } p[2];   // M 0: none
  int splits;
  int* counters;   // of 8, zeros before the launch (kClaims)
};

// kClaims: a workgroup's first three items are given, the others claimed in order from a counter,
// three items ahead, so that workgroups that come later or slower take fewer of them.  Whoever
// works on a tile, its sums are the same.  Without: splits > 1, or counters that nobody cleared.
// (Behind dx, with every item given: Qwen2-shaped gradients of 3001 tokens, skewed, 2.73 ms, claimed
// 2.38; of 200 rows of 1024 x 512 54 and 44 us; dense, 1024 rows of 4096 x 1024, 99 and 104.  With
// one item given instead of three a dense backward of 4096 x 7168 x 2048 643 -> 695 us.)
template <class TOut, bool kClaims>
struct WeightsJob {
  static constexpr bool kAAcross = true, kBAcross = true, kEmptyLast = kClaims;
  using A = Across;
  using B = Across;
  static constexpr int kEnd = -1;
  const WeightArgs& a;
  Smem& sm;   // pre: the experts by rank
  int each0, each1, run0, run, hi, start, step, xcd;

  struct Item {
    int e, k, m0, n0, n, part;   // k: the product
    int64_t row0;
  };

  static __device__ __forceinline__ int tiles(int n) { return (n + kTile - 1) / kTile; }

  __device__ __forceinline__ WeightsJob(const WeightArgs& args, const Lane& l, Smem& m)
      : a(args), sm(m) {
    const int E = a.r.counts ? a.r.E : 1;
    int n = 0, row0 = 0;
    if (l.tid < E) {
      n = expert_rows(a.r, l.tid, &row0);
      m.first[l.tid] = row0;
      m.rows[l.tid] = n;
    }
    __syncthreads();
    if (l.tid < E) {
      int rank = 0;
#pragma unroll 8
      for (int e = 0; e < E; ++e) rank += m.rows[e] > n || (m.rows[e] == n && e < l.tid);
      m.pre[rank] = l.tid;
    }
    __syncthreads();
    // the parts of a tile's contraction are tiles of their own
    each0 = tiles(a.p[0].M) * tiles(a.p[0].N) * a.splits;
    each1 = tiles(a.p[1].M) * tiles(a.p[1].N) * a.splits;
    // an item a workgroup, or few that share their operands
    if (E * (int64_t)(each0 + each1) <= (int64_t)gridDim.x || (kClaims && each0 + each1 < 64)) {
      run0 = each0;
      run = each0 + each1;
      xcd = -1;
      start = (int)blockIdx.x;
      step = (int)gridDim.x;
    } else {
      run0 = (each0 + 7) / 8;
      run = run0 + (each1 + 7) / 8;
      xcd = (int)blockIdx.x % 8;
      start = (int)blockIdx.x / 8;
      step = (int)gridDim.x / 8;
    }
    hi = E * run;
    if constexpr (kClaims) {
      // from the last workgroup on: the first ones may come from other work
      if (l.tid == 0) {
        int n = 0;
        for (int k = 0; k < 3; ++k) {
          const int it = step - 1 - start + k * step;
          if (present(it)) m.claim[n++] = it;
        }
        while (n < 3) m.claim[n++] = next_claim();   // in the order of the list, as all are
      }
      __syncthreads();
    }
  }
  __device__ __forceinline__ bool present(int it) const {
    int e, k, tile;
    return it < hi && tile_of(it, &e, &k, &tile);
  }
  // one lane: an item nobody has, or hi
  __device__ __forceinline__ int next_claim() const {
    int it;
    do {
      it = 3 * step + __hip_atomic_fetch_add(a.counters + max(xcd, 0), 1, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
    } while (it < hi && !present(it));
    return it;
  }
  // at the start of item number it of this workgroup: the item three further on, claimed; and at
  // the end of it, where it has come, kept
  typedef int Claim;
  __device__ __forceinline__ int claim(const Lane& l, const Item&) const {
    int taken = 0;
    if constexpr (kClaims)
      if (l.tid == 0) {
        int at = max(xcd, 0);
        asm volatile("" : "+v"(at));   // a lane's own address: what it adds is not waited for here
        taken = __hip_atomic_fetch_add(a.counters + at, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    return taken;
  }
  __device__ __forceinline__ void claimed(const Lane& l, int number, int taken) const {
    if constexpr (kClaims)
      if (l.tid == 0) {
        const int it = 3 * step + taken;
        sm.claim[(number + 3) & 3] = it < hi && !present(it) ? next_claim() : it;
      }
  }
  // the expert, product and tile of place it in this XCD's order; false: none
  __device__ __forceinline__ bool tile_of(int it, int* e, int* k, int* tile) const {
    const int rank = uniform(it / run);
    *e = uniform(sm.pre[rank]);
    int at = it - rank * run;
    *k = at >= run0;
    const int part = *k ? run - run0 : run0;
    if (*k) at -= run0;
    *tile = xcd < 0 ? at : ((xcd + *e) & 7) * part + at;
    return *tile < (*k ? each1 : each0);
  }
  __device__ __forceinline__ int held(int it) const {
    int e, k, tile;
    while (it < hi && !tile_of(it, &e, &k, &tile)) it += step;
    return it < hi ? it : kEnd;
  }
  // kClaims: the number of an item of this workgroup
  __device__ __forceinline__ int first() const { return kClaims ? next(-1) : held(start); }
  __device__ __forceinline__ int next(int it) const {
    if (kClaims) return uniform(sm.claim[(it + 1) & 3]) < hi ? it + 1 : kEnd;
    return held(it + step);
  }

  __device__ __forceinline__ Item item(int it) const {
    if (kClaims) it = uniform(sm.claim[it & 3]);
    Item x;
    int at;
    tile_of(it, &x.e, &x.k, &at);
    x.part = 0;
    if (a.splits > 1) {
      const int tile = uniform(at / a.splits);
      x.part = at - tile * a.splits;
      at = tile;
    }
    const int tm_n = tiles(a.p[x.k].M), tn_n = tiles(a.p[x.k].N);
    // tiles in bands of 4 along N, so that those at work together share their operands
    const int band = uniform(at / (4 * tm_n)), in_band = at - band * 4 * tm_n;
    const int width = min(4, tn_n - 4 * band);
    const int tm = uniform(in_band / width);
    x.m0 = tm * kTile;
    x.n0 = (4 * band + in_band - tm * width) * kTile;
    x.n = uniform(sm.rows[x.e]);
    x.row0 = uniform(sm.first[x.e]);
    if (a.splits > 1) {   // whole blocks of rows
      const int blocks = (x.n + kBlock - 1) / kBlock;
      const int rows = uniform((blocks + a.splits - 1) / a.splits) * kBlock;
      const int before = min(x.n, x.part * rows);
      x.row0 += before;
      x.n = min(rows, x.n - before);
    }
    return x;
  }
  __device__ __forceinline__ int blocks(const Item& x) const {
    return (x.n + kBlock - 1) / kBlock;
  }
  __device__ __forceinline__ bool two(const Item&) const { return true; }
  __device__ __forceinline__ void load(const Lane& l, const Item& x, Across& la, Across& lb) const {
    const WeightArgs::Product& p = a.p[x.k];
    la.set(l, p.m_rows + (size_t)x.row0 * p.M, (uint32_t)p.M * 2, x.n, x.m0);
    lb.set(l, p.n_rows + (size_t)x.row0 * p.N, (uint32_t)p.N * 2, x.n, x.n0);
  }
  __device__ __forceinline__ void store(const Lane& l, const Item& x, f32x4 (&acc)[TM][TN],
                                        int) const {
    const WeightArgs::Product& p = a.p[x.k];
    store_tile(l, acc, static_cast<TOut*>(p.out) + (size_t)x.part * p.part +
                           ((size_t)x.e * p.N + x.n0) * p.M + x.m0, p.M,
               min(kTile, p.N - x.n0), p.M - x.m0);
  }
};

template <class TOut, bool kClaims>
__global__ __launch_bounds__(kThreads, 1) void weights_kernel(WeightArgs a) {
  TRAIN_UNITS;
  __shared__ Smem sm;
  const Lane l(threadIdx.x);
  WeightsJob<TOut, kClaims> job(a, l, sm);
  stream(l, job, units);
}

// dx, then the weights' gradients, by workgroups as they come: the tiles of the latter fill the
// rounds that dx leaves part empty.  (In two launches and in one, a backward: tiny layer 36 and
// 29 us; 64 experts of 3584 x 2560, 128 tokens, 1522 and 1470, 3001 tokens 2430 and 2378; 8 of
// 4096 x 14336, 4096 tokens, 5622 and 5526; dense, 200 rows of 1024 x 512 57 and 44, 1003 of
// 2048 x 1024 98 and 73, 512 of 2048 x 2048 87 and 83, 2000 of 1024 x 1024 107 both.)
template <Split kSplit, class TOut>
__global__ __launch_bounds__(kThreads, 1) void grads_kernel(Args a, WeightArgs w) {
  TRAIN_UNITS;
  __shared__ Smem sm;
  const Lane l(threadIdx.x);
  {
    RowsJob<kDX, false, kSplit, false> job(a, l, sm);
    stream(l, job, units);
  }
  __syncthreads();   // the experts' lists are read to the end
  WeightsJob<TOut, true> job(w, l, sm);
  stream(l, job, units);
}

// ------------------------------------------------------------------ adding partial sums
//
// Where a launch has few items, parts of their contraction run on the other compute units, and
// their sums are added here in the order of the parts: bound by those sums' bytes, at most
// kPartBytes.  Where padding leaves no room for them by row they are kept by pair, so that it
// changes neither the parts nor a sum.
// A lane has 8 neighbours of a row that holds a pair, as the products' epilogues do.
constexpr int kFinishThreads = 256;

__device__ __forceinline__ void add_parts(const float* p, int64_t stride, int parts, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  for (int s = 0; s < parts; ++s) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p + s * stride)[0];
    const f32x4 b = reinterpret_cast<const f32x4*>(p + s * stride)[1];
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
}

template <Op kOp, bool kFp8, bool kPair>
__global__ __launch_bounds__(kFinishThreads) void finish_rows_kernel(Args a) {
  const int H = a.r.H, I = a.r.I;
  const int width = kOp == kGateUp || kOp == kDAct ? I : H, groups = width / 8;
  const int64_t at = (int64_t)blockIdx.x * kFinishThreads + threadIdx.x;
  const int64_t row = at / groups;
  if (row >= a.r.rows) return;
  const int c = (int)(at - row * groups) * 8;   // 4 lanes share a block of 32, and a row
  int64_t from = row;
  if (a.r.counts) {
    const int p = a.r.sorted_ids[row];
    if (p < 0 || p >= a.r.tokens * a.r.K) return;
    if (kPair) from = p;
  }
  const int F = kOp == kGateUp ? 2 * I : width;
  const int64_t stride = a.part_rows * F;
  float v[8];
  add_parts(a.part + from * F + c, stride, a.splits, v);
  if constexpr (kOp == kGateUp) {
    float u[8], av[8];
    add_parts(a.part + from * F + I + c, stride, a.splits, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) av[q] = silu(v[q]) * u[q];
    *reinterpret_cast<u32x4*>(a.act + row * I + c) = bf16x8_of(av);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* w = k ? u : v;
      const int64_t to = row * 2 * I + (k ? I : 0) + c;
      if constexpr (kFp8) {
        float most = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) most = abs_max(most, w[q]);
        const int byte = scale_byte(quad_max(most));
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.h) + to) =
            pack_e4m3x8(w, inverse_scale(byte));
        if ((c & 31) == 0) a.scales[to / 32] = (uint8_t)byte;
      } else {
        *reinterpret_cast<u32x4*>(a.h + to) = bf16x8_of(w);
      }
    }
  } else if constexpr (kOp == kDAct) {
    float kept[2][8], av[8], dg[8], du[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t from = row * 2 * I + (k ? I : 0) + c;
      if constexpr (kFp8)
        unpack_e4m3x8(*reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.h) + from),
                      scale_of(a.scales[from / 32]), kept[k]);
      else
        bf16x8_to(*reinterpret_cast<const u32x4*>(a.h + from), kept[k]);
    }
    gradients(v, kept[0], kept[1], av, dg, du);
    *reinterpret_cast<u32x4*>(a.act + row * I + c) = bf16x8_of(av);
    *reinterpret_cast<u32x4*>(a.dh + row * 2 * I + c) = bf16x8_of(dg);
    *reinterpret_cast<u32x4*>(a.dh + row * 2 * I + I + c) = bf16x8_of(du);
  } else {
    *reinterpret_cast<u32x4*>(a.out + row * H + c) = bf16x8_of(v);
  }
}

// values: a multiple of 8
template <class TOut>
__global__ __launch_bounds__(kFinishThreads) void finish_weights_kernel(const float* part,
                                                                        int64_t values, int parts,
                                                                        TOut* out) {
  const int64_t at = ((int64_t)blockIdx.x * kFinishThreads + threadIdx.x) * 8;
  if (at >= values) return;
  float v[8];
  add_parts(part + at, values, parts, v);
  if constexpr (sizeof(TOut) == 2) {
    *reinterpret_cast<u32x4*>(out + at) = bf16x8_of(v);
  } else {
    reinterpret_cast<f32x4*>(out + at)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(out + at)[1] = f32x4{v[4], v[5], v[6], v[7]};
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

// Parts of the contraction of a launch of `items` items (at most) of `blocks` blocks, whose sums
// are `values` in all: as many as the compute units take in one round (`xcds`: of runs that each
// XCD has of its own) where the items would leave three quarters of them idle, 16 blocks or more,
// and as `room` bytes hold; up to 8 of 4 blocks or more, more of 8.
// Measured, whole and in parts: one token of a Mixtral-shaped down product 219 and 51 us; the da
// and dx of 200 rows of 1024 x 512 48 us in parts of 8 blocks or more, 42 of 4 (128 rows of
// 4096 x 4096, 16 parts of 4 and 8 of 8: 69 and 65); 300 rows of 512 x 512 forward, of 8 blocks,
// 33 whole and 42.
// others: items of the same launch, of other_blocks.  Where they fit, they have compute units of
// their own and leave fewer parts, unless that makes a part longer by more than 8 blocks and by
// more than two of the others, which a workgroup then does after it.  Measured, a dense backward
// with such fewer parts of dx and with all: 1003 rows of 1088 x 1856 (5 parts or 8) 74 and 95 us,
// 900 of 2048 x 1536 (3, 8) 79 and 100, 768 of 2048 x 2048 (2, 8; as long as two others) 97 and 99,
// 640 94 and 90, 512 91 and 84, 232 of 1472 x 3584 (whole, 14) 183 and 79.
int parts_of(int64_t items, int64_t blocks, int64_t values, int64_t room, bool xcds,
             int64_t others = 0, int64_t other_blocks = 0) {
  if (items < 1 || 4 * items > workgroups() || blocks < 16 || values < 1) return 1;
  const auto fit = [&](int64_t units) { return xcds ? units / 8 / ((items + 7) / 8) : units / items; };
  int64_t n = fit(workgroups());
  const int64_t most = blocks / 4 < 8 ? blocks / 4 : blocks / 8 > 8 ? blocks / 8 : 8;
  if (n > kMaxParts) n = kMaxParts;
  if (n > most) n = most;
  if (n > room / (4 * values)) n = room / (4 * values);
  if (others > 0 && others < workgroups()) {
    int64_t own = fit(workgroups() - others);
    if (own < 1) own = 1;
    if (own < n) {
      const int64_t longer = (blocks + own - 1) / own - (blocks + n - 1) / n;
      if (longer <= 8 || longer <= 2 * other_blocks) n = own;
    }
  }
  return n < 2 ? 1 : (int)n;
}

// The parts of a product over rows, and the grid for the most items it can have
template <Op kOp>
hipError_t plan_rows(Args& a, const PartSpace& space, int64_t others, unsigned* grid) {
  const int per_tile = kOp == kGateUp ? kTile / 2 : kTile;
  const int F = kOp == kGateUp || kOp == kDAct ? a.r.I : a.r.H;
  const int K = kOp == kGateUp || kOp == kDAct ? a.r.H : kOp == kDown ? a.r.I : 2 * a.r.I;
  // spans: one for each 256 rows, and a short one an expert
  const int64_t pairs = a.r.counts ? a.r.tokens * a.r.K : a.r.tokens;
  const int64_t experts = a.r.counts ? (a.r.E < pairs ? a.r.E : pairs) : 1;
  const int64_t spans = pairs / kTile + experts;
  const int64_t items = spans * ((F + per_tile - 1) / per_tile);
  if (items >= (int64_t)1 << 30) return hipErrorInvalidValue;
  const int64_t width = kOp == kGateUp ? 2 * (int64_t)F : F;
  a.part = space.part;
  // blocks of a weights' tile: an expert's rows, of the busier ones twice the mean
  const int64_t tile_blocks = ((experts > 1 ? 2 : 1) * pairs / experts + kBlock - 1) / kBlock;
  a.splits = parts_of(items, K / kBlock, pairs * width, space.bytes, true, others, tile_blocks);
  // By row where there is room for the padding too: by pair, whose rows a tile scatters, da and dx of
  // 300 rows of 1024 x 2048 for two experts take 61 us for 59.  In the parts that have room by row,
  // and by pair: one token of a Mixtral-shaped layer forward 153 and 139 us with its rows 128 apart,
  // 304 and 141 with 1024.
  a.by_pair = a.r.counts && a.splits > 1 && a.splits > space.bytes / (4 * a.r.rows * width);
  a.part_rows = a.by_pair ? pairs : a.r.rows;
  // whole: twice the items, as they may be cut in two; in parts: an XCD's run, and its run of
  // short experts, in one round (without: dx of 1003 rows of 1088 x 1856 48 us, with 30)
  *grid = grid_of(a.splits == 1 ? 2 * items : 8 * ((items + 7) / 8 + 1) * a.splits);
  return hipSuccess;
}

template <Op kOp, bool kFp8>
hipError_t finish_rows(const Args& a, hipStream_t s) {
  const int64_t lanes = a.r.rows * ((kOp == kGateUp || kOp == kDAct ? a.r.I : a.r.H) / 8);
  const dim3 grid((unsigned)((lanes + kFinishThreads - 1) / kFinishThreads)), block(kFinishThreads);
  if (a.by_pair) hipLaunchKernelGGL((finish_rows_kernel<kOp, kFp8, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((finish_rows_kernel<kOp, kFp8, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <Op kOp, bool kFp8>
hipError_t launch_planned(const Args& a, unsigned grid, hipStream_t s) {
  if (a.splits == 1)
    hipLaunchKernelGGL((rows_kernel<kOp, kFp8, kWhole>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (!a.by_pair)
    hipLaunchKernelGGL((rows_kernel<kOp, false, kByRow>), dim3(grid), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((rows_kernel<kOp, false, kByPair>), dim3(grid), dim3(kThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && a.splits > 1 ? finish_rows<kOp, kFp8>(a, s) : e;
}

template <Op kOp, bool kFp8>
hipError_t launch_rows(Args a, const PartSpace& space, hipStream_t s) {
  if (a.r.tokens == 0) return hipSuccess;
  unsigned grid;
  const hipError_t e = plan_rows<kOp>(a, space, 0, &grid);
  return e == hipSuccess ? launch_planned<kOp, kFp8>(a, grid, s) : e;
}

template <class TOut>
hipError_t launch_joined(const Args& a, const WeightArgs& w, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(kThreads);
  if (a.splits == 1) hipLaunchKernelGGL((grads_kernel<kWhole, TOut>), g, b, 0, s, a, w);
  else if (!a.by_pair) hipLaunchKernelGGL((grads_kernel<kByRow, TOut>), g, b, 0, s, a, w);
  else hipLaunchKernelGGL((grads_kernel<kByPair, TOut>), g, b, 0, s, a, w);
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
                                const SavedRows& saved, uint16_t* act, const PartSpace& space,
                                hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w13);
  a.in = static_cast<const uint16_t*>(x);
  a.act = act;
  a.h = static_cast<uint16_t*>(saved.h);
  a.scales = saved.scales;
  return saved.fp8 ? launch_rows<kGateUp, true>(a, space, s) : launch_rows<kGateUp, false>(a, space, s);
}

hipError_t launch_train_down(const TrainRows& r, const void* w2, const uint16_t* act, void* y,
                             const PartSpace& space, hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w2);
  a.in = act;
  a.out = static_cast<uint16_t*>(y);
  return launch_rows<kDown, false>(a, space, s);
}

hipError_t launch_train_dact(const TrainRows& r, const void* w2, const void* dy,
                             const SavedRows& saved, uint16_t* act, uint16_t* dh, int* counters,
                             const PartSpace& space, hipStream_t s) {
  Args a = args_of(r);
  a.w = static_cast<const uint16_t*>(w2);
  a.in = static_cast<const uint16_t*>(dy);
  a.act = act;
  a.dh = dh;
  a.counters = counters;
  a.h = static_cast<uint16_t*>(saved.h);
  a.scales = saved.scales;
  return saved.fp8 ? launch_rows<kDAct, true>(a, space, s) : launch_rows<kDAct, false>(a, space, s);
}

hipError_t launch_train_grads(const TrainRows& r, const void* w13, const uint16_t* dh, void* dx,
                              const uint16_t* x_rows, void* dw13, const uint16_t* act,
                              const void* dy, void* dw2, bool f32, const PartSpace& space,
                              int* counters, hipStream_t s) {
  const int64_t matrices = r.counts ? r.E : 1;
  const int64_t n13 = dw13 ? matrices * 2 * r.I * r.H : 0, n2 = dw2 ? matrices * r.H * r.I : 0;
  WeightArgs w{r,
               {{x_rows, dh, dw13, dw13 ? r.H : 0, 2 * r.I, n13},
                {act, static_cast<const uint16_t*>(dy), dw2, dw2 ? r.I : 0, r.H, n2}},
               1,
               counters};
  int64_t items = 0;
  for (const WeightArgs::Product& p : w.p)
    items += matrices * ((p.M + kTile - 1) / kTile) * ((p.N + kTile - 1) / kTile);
  if (items >= (int64_t)1 << 30) return hipErrorInvalidValue;
  // the most rows an expert may have
  const int64_t rows = r.tokens < r.rows ? r.tokens : r.rows;
  w.splits = parts_of(items, rows / kBlock, n13 + n2, space.bytes, false);
  const dim3 block(kThreads);
  hipError_t e = hipSuccess;
  if (dx && r.tokens > 0) {
    Args a = args_of(r);
    a.w = static_cast<const uint16_t*>(w13);
    a.in = dh;
    a.out = static_cast<uint16_t*>(dx);
    const int64_t beside = w.splits == 1 ? items : 0;
    unsigned rows_grid;
    e = plan_rows<kDX>(a, space, beside, &rows_grid);
    if (e != hipSuccess) return e;
    if (beside > 0) {
      const unsigned grid = grid_of(rows_grid + items);
      e = f32 ? launch_joined<float>(a, w, grid, s) : launch_joined<uint16_t>(a, w, grid, s);
      return e == hipSuccess && a.splits > 1 ? finish_rows<kDX, false>(a, s) : e;
    }
    e = launch_planned<kDX, false>(a, rows_grid, s);
  }
  if (e != hipSuccess || items == 0) return e;
  const dim3 grid(grid_of(items * w.splits));
  if (w.splits > 1) {
    w.p[0].out = space.part;
    w.p[1].out = space.part + w.splits * n13;
    hipLaunchKernelGGL((weights_kernel<float, false>), grid, block, 0, s, w);
  } else if (r.tokens == 0) {
    if (f32) hipLaunchKernelGGL((weights_kernel<float, false>), grid, block, 0, s, w);
    else hipLaunchKernelGGL((weights_kernel<uint16_t, false>), grid, block, 0, s, w);
  } else {
    if (f32) hipLaunchKernelGGL((weights_kernel<float, true>), grid, block, 0, s, w);
    else hipLaunchKernelGGL((weights_kernel<uint16_t, true>), grid, block, 0, s, w);
  }
  e = hipGetLastError();
  void* const outs[2] = {dw13, dw2};
  for (int k = 0; k < 2 && w.splits > 1 && e == hipSuccess; ++k) {
    const int64_t n = w.p[k].part;
    if (n == 0) continue;
    const dim3 g((unsigned)((n / 8 + kFinishThreads - 1) / kFinishThreads)), b(kFinishThreads);
    const float* part = static_cast<const float*>(w.p[k].out);
    if (f32)
      hipLaunchKernelGGL(finish_weights_kernel<float>, g, b, 0, s, part, n, w.splits,
                         static_cast<float*>(outs[k]));
    else
      hipLaunchKernelGGL(finish_weights_kernel<uint16_t>, g, b, 0, s, part, n, w.splits,
                         static_cast<uint16_t*>(outs[k]));
    e = hipGetLastError();
  }
  return e;
}

}  // namespace moe
