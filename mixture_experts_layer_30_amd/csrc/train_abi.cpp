// C ABI of the experts' training step and of activations kept in 8 bits.  What each call
// computes is documented in include/moe_layer.h.
#include <stdint.h>

#include <initializer_list>

#include "block_checks.h"
#include "train_kernels.h"

namespace {

using namespace moe_checks;

constexpr int kMaxWidth = 1 << 20;   // of H and I: a span's rows are counted in 32 bits

// the FFN's sizes; every matrix of an expert is read through 32-bit offsets
moe_status check_ffn(const char* what, int64_t T, int H, int I) {
  if (T < 0) return fail(MOE_EINVAL, "%s: T = %lld < 0", what, (long long)T);
  if (T >= ((int64_t)1 << 31) - 256)   // rows up to a tile's end are counted in 32 bits
    return fail(MOE_EUNSUPPORTED, "%s: T must be < 2^31 - 256", what);
  if (H < 64 || H % 64 != 0 || H > kMaxWidth || I < 64 || I % 64 != 0 || I > kMaxWidth)
    return fail(MOE_EUNSUPPORTED, "%s: H = %d and I = %d must be multiples of 64 up to 2^20", what,
                H, I);
  if ((int64_t)4 * I * H >= (int64_t)1 << 32)
    return fail(MOE_EUNSUPPORTED, "%s: an expert's gate and up weights must be below 4 GB", what);
  return MOE_OK;
}

moe_status check_grouped(const char* what, int64_t T, int H, int I, int E, int K,
                         const moe_plan* plan) {
  moe_status st = check_ffn(what, T, H, I);
  if (st) return st;
  st = check_routing(what, T, E, K);
  if (st) return st;
  if (T * H * 2 >= (int64_t)1 << 32)
    return fail(MOE_EUNSUPPORTED, "%s: x must be below 4 GB", what);
  return check_plan(what, plan, T, K, E);
}

moe_status check_saved(const char* what, const moe_saved* saved, int64_t rows,
                       moe::SavedRows* out) {
  if (!saved) return fail(MOE_EINVAL, "%s: saved is NULL", what);
  if (saved->format != MOE_SAVE_BF16 && saved->format != MOE_SAVE_FP8)
    return fail(MOE_EINVAL, "%s: saved->format = %d", what, (int)saved->format);
  const bool fp8 = saved->format == MOE_SAVE_FP8;
  if (rows > 0 && (!good(saved->h, 16) || (fp8 && !saved->scales)))
    return fail(MOE_EINVAL, "%s: saved has a NULL or misaligned pointer", what);
  *out = moe::SavedRows{saved->h, saved->scales, fp8};
  return MOE_OK;
}

moe_status check_space(const char* what, int64_t rows, const void* workspace, int64_t bytes,
                       int64_t need) {
  if (bytes < need)
    return fail(MOE_ECAPACITY, "%s: workspace %lld bytes < %lld required", what, (long long)bytes,
                (long long)need);
  if (rows > 0 && !good(workspace, 16)) return null_pointer(what);
  return MOE_OK;
}

// A buffer of a call; bytes 0 or p NULL: none
struct Buffer {
  const char* name;
  const void* p;
  int64_t bytes;
};

// what a call writes (each of `written`) overlaps neither the others of them nor what it reads
moe_status check_apart(const char* what, std::initializer_list<Buffer> written,
                       std::initializer_list<Buffer> read) {
  auto meet = [](const Buffer& a, const Buffer& b) {
    const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p;
    return p && q && a.bytes > 0 && b.bytes > 0 && p < q + (uintptr_t)b.bytes &&
           q < p + (uintptr_t)a.bytes;
  };
  for (const Buffer* a = written.begin(); a != written.end(); ++a) {
    for (const Buffer* b = a + 1; b != written.end(); ++b)
      if (meet(*a, *b)) return fail(MOE_EINVAL, "%s: %s and %s overlap", what, a->name, b->name);
    for (const Buffer& b : read)
      if (meet(*a, b)) return fail(MOE_EINVAL, "%s: %s overwrites %s", what, a->name, b.name);
  }
  return MOE_OK;
}

moe::TrainRows planned(const moe_plan* plan, int64_t T, int E, int K, int H, int I) {
  return moe::TrainRows{plan->expert_counts, plan->expert_offsets, plan->sorted_ids, T, plan->cap,
                        K, E, H, I};
}

moe::TrainRows dense(int64_t T, int H, int I) {
  return moe::TrainRows{nullptr, nullptr, nullptr, T, T, 1, 1, H, I};
}

// bytes of partial sums, past the others: no more than all rows' in every part
int64_t part_bytes(int64_t rows, int H, int I) {
  const int64_t most = rows * (2 * I > H ? 2 * I : H) * 4 * moe::kMaxParts;
  return most < moe::kPartBytes ? most : moe::kPartBytes;
}

int64_t rounded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

Buffer saved_values(const moe::SavedRows& s, const moe::TrainRows& r) {
  return {"the kept values", s.h, r.rows * r.I * (s.fp8 ? 2 : 4)};
}
Buffer saved_scales(const moe::SavedRows& s, const moe::TrainRows& r) {
  return {"the kept scales", s.fp8 ? s.scales : nullptr, r.rows * r.I / 16};
}

moe_status forward(const char* what, const moe::TrainRows& r, const void* x, const void* w13,
                   const void* w2, const moe_saved* kept, void* workspace,
                   int64_t workspace_bytes, void* y, void* stream) {
  moe::SavedRows saved;
  moe_status st = check_saved(what, kept, r.tokens, &saved);
  if (st) return st;
  st = check_space(what, r.tokens, workspace, workspace_bytes,
                   moe_ffn_train_workspace_bytes(r.rows, r.H, r.I));
  if (st) return st;
  if (r.tokens == 0) return ok();
  if (!good(x, 16) || !good(w13, 16) || !good(w2, 16) || !good(y, 16)) return null_pointer(what);
  const int64_t matrix = (int64_t)(r.counts ? r.E : 1) * r.H * r.I * 2;
  const Buffer in{"x", x, r.tokens * r.H * 2}, up{"w13", w13, 2 * matrix}, down{"w2", w2, matrix};
  const Buffer room{"the workspace", workspace, moe_ffn_train_workspace_bytes(r.rows, r.H, r.I)};
  const Buffer rows{"rows", y, r.rows * r.H * 2};   // written last, when x and w13 have been read
  st = check_apart(what, {saved_values(saved, r), saved_scales(saved, r), room}, {in, up, down, rows});
  if (!st) st = check_apart(what, {rows}, {down});
  if (st) return st;
  uint16_t* act = static_cast<uint16_t*>(workspace);
  const hipStream_t s = (hipStream_t)stream;
  const moe::PartSpace space{(float*)(act + rounded(r.rows * r.I * 2) / 2),
                             part_bytes(r.rows, r.H, r.I)};
  hipError_t e = moe::launch_train_gate_up(r, x, w13, saved, act, space, s);
  if (e == hipSuccess) e = moe::launch_train_down(r, w2, act, y, space, s);
  return hip_status(e, what);
}

moe_status backward(const char* what, const moe::TrainRows& r, const moe_plan* plan, const void* dy,
                    const void* x, const void* w13, const void* w2, const moe_saved* kept, void* workspace,
                    int64_t workspace_bytes, void* dx, void* dw13, void* dw2, int dwdt,
                    void* stream) {
  if (dwdt != MOE_F32 && dwdt != MOE_BF16) return fail(MOE_EUNSUPPORTED, "%s: dwdt", what);
  moe::SavedRows saved;
  moe_status st = check_saved(what, kept, r.tokens, &saved);
  if (st) return st;
  st = check_space(what, r.tokens, workspace, workspace_bytes,
                   moe_ffn_backward_workspace_bytes(r.rows, r.H, r.I));
  if (st) return st;
  if (!optional(dw13, 16) || !optional(dw2, 16) || !optional(dx, 16)) return null_pointer(what);
  if (!dx && !dw13 && !dw2) return fail(MOE_EINVAL, "%s: no gradient is asked for", what);
  if (r.tokens > 0) {
    if (!good(dy, 16) || !good(w2, 16) || (dx ? !good(w13, 16) : !optional(w13, 16)) ||
        (dw13 ? !good(x, 16) : !optional(x, 16)))
      return null_pointer(what);
  }
  // The gradients of the rows and of the weights are written by workgroups in no order, which
  // still read dy, x and w13; w2 and the kept values have been read by then.
  const int64_t matrix = (int64_t)(r.counts ? r.E : 1) * r.H * r.I;
  const int64_t row_bytes = r.tokens > 0 ? r.rows * r.H * 2 : 0, x_bytes = r.tokens * r.H * 2;
  const int64_t dw_bytes = dwdt == MOE_F32 ? 4 : 2;
  const Buffer room{"the workspace", r.tokens > 0 ? workspace : nullptr,
                    moe_ffn_backward_workspace_bytes(r.rows, r.H, r.I)};
  const Buffer rows{"the rows' gradient", dx, row_bytes};
  st = check_apart(what,
                   {rows,
                    {"dw13", dw13, 2 * matrix * dw_bytes},
                    {"dw2", dw2, matrix * dw_bytes},
                    room},
                   {{"the output's gradient", dy, row_bytes},
                    {"x", dw13 ? x : nullptr, x_bytes},
                    {"w13", dx && r.tokens > 0 ? w13 : nullptr, 4 * matrix}});
  if (!st) st = check_apart(what, {rows}, {{"x", x, x_bytes}});
  if (!st && r.tokens > 0)
    st = check_apart(what, {room},
                     {{"w2", w2, 2 * matrix}, saved_values(saved, r), saved_scales(saved, r)});
  if (st) return st;
  uint16_t* act = static_cast<uint16_t*>(workspace);
  uint16_t* dh = act + rounded(r.rows * r.I * 2) / 2;
  uint16_t* x_rows = dh + rounded(r.rows * r.I * 4) / 2;
  const moe::PartSpace space{(float*)(x_rows + rounded(r.rows * r.H * 2) / 2),
                             part_bytes(r.rows, r.H, r.I)};
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  int* counters = (int*)((char*)space.part + rounded(space.bytes));
  if (r.tokens > 0) e = moe::launch_train_dact(r, w2, dy, saved, act, dh, counters, space, s);
  const uint16_t* xr = static_cast<const uint16_t*>(x);
  if (e == hipSuccess && dw13 && plan && r.tokens > 0) {
    // x by row: the contraction over rows then reads whole lines in order (gathering in it
    // took the registers that hide its loads; the copy is 1% of a Mixtral-shaped backward).  The
    // product reads no padding rows.
    e = moe::launch_permute(x, moe::kDtBF16, r.tokens, r.K, r.H, plan_rows(plan, r.K), r.E, r.rows,
                            x_rows, false, s);
    xr = x_rows;
  }
  if (e == hipSuccess)
    e = moe::launch_train_grads(r, w13, dh, dx, xr, dw13, act, dy, dw2, dwdt == MOE_F32, space,
                                counters, s);
  return hip_status(e, what);
}

moe_status check_pack(const char* what, int64_t T, int H, int dt) {
  moe_status st = check_rows(what, T, H);
  if (st) return st;
  if (H % 32 != 0) return fail(MOE_EUNSUPPORTED, "%s: H = %d must be a multiple of 32", what, H);
  if (!valid_dtype(dt)) return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_ffn_train_workspace_bytes(int64_t rows, int H, int I) {
  if (rows < 0 || rows >= (int64_t)1 << 31 || H < 64 || H % 64 != 0 || H > kMaxWidth || I < 64 ||
      I % 64 != 0 || I > kMaxWidth)
    return -1;
  return rounded(rows * I * 2) + part_bytes(rows, H, I);
}

int64_t moe_ffn_backward_workspace_bytes(int64_t rows, int H, int I) {
  const int64_t act = moe_ffn_train_workspace_bytes(rows, H, I);   // a, and partial sums
  // dh of every row, and x by row
  return act < 0 ? -1
                 : rounded(act) + rounded(rows * I * 4) + rounded(rows * H * 2) +
                       (rows > 0 ? moe::kCounterBytes : 0);
}

moe_status moe_grouped_ffn_train(const void* x, int64_t T, int H, int I, int E, int K,
                                 const void* w13, const void* w2, const moe_plan* plan,
                                 const moe_saved* saved, void* workspace, int64_t workspace_bytes,
                                 void* rows, void* stream) {
  const char* what = "moe_grouped_ffn_train";
  moe_status st = check_grouped(what, T, H, I, E, K, plan);
  if (st) return st;
  return forward(what, planned(plan, T, E, K, H, I), x, w13, w2, saved, workspace, workspace_bytes,
                 rows, stream);
}

moe_status moe_grouped_ffn_backward(const void* drows, const void* x, int64_t T, int H, int I,
                                    int E, int K, const void* w13, const void* w2,
                                    const moe_plan* plan, const moe_saved* saved, void* workspace,
                                    int64_t workspace_bytes, void* dxrows, void* dw13, void* dw2,
                                    moe_dtype dwdt, void* stream) {
  const char* what = "moe_grouped_ffn_backward";
  moe_status st = check_grouped(what, T, H, I, E, K, plan);
  if (st) return st;
  return backward(what, planned(plan, T, E, K, H, I), plan, drows, x, w13, w2, saved, workspace,
                  workspace_bytes, dxrows, dw13, dw2, dwdt, stream);
}

moe_status dense_ffn_train(const void* x, int64_t T, int H, int I, const void* w13, const void* w2,
                           const moe_saved* saved, void* workspace, int64_t workspace_bytes,
                           void* out, void* stream) {
  const char* what = "dense_ffn_train";
  moe_status st = check_ffn(what, T, H, I);
  if (st) return st;
  return forward(what, dense(T, H, I), x, w13, w2, saved, workspace, workspace_bytes, out, stream);
}

moe_status dense_ffn_backward(const void* dout, const void* x, int64_t T, int H, int I,
                              const void* w13, const void* w2, const moe_saved* saved,
                              void* workspace, int64_t workspace_bytes, void* dx, void* dw13,
                              void* dw2, moe_dtype dwdt, void* stream) {
  const char* what = "dense_ffn_backward";
  moe_status st = check_ffn(what, T, H, I);
  if (st) return st;
  return backward(what, dense(T, H, I), nullptr, dout, x, w13, w2, saved, workspace, workspace_bytes, dx,
                  dw13, dw2, dwdt, stream);
}

moe_status moe_pack_fp8(const void* x, moe_dtype dt, int64_t T, int H, uint8_t* codes,
                        uint8_t* scales, void* stream) {
  const char* what = "moe_pack_fp8";
  moe_status st = check_pack(what, T, H, dt);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(x, 16) || !good(codes, 16) || !scales) return null_pointer(what);
  st = check_apart(what, {{"codes", codes, T * H}, {"scales", scales, T * (H / 32)}},
                   {{"x", x, T * H * (dt == MOE_F32 ? 4 : 2)}});
  if (st) return st;
  return hip_status(moe::launch_pack_fp8(x, dt, T, H, codes, scales, (hipStream_t)stream), what);
}

moe_status moe_unpack_fp8(const uint8_t* codes, const uint8_t* scales, int64_t T, int H, void* x,
                          moe_dtype dt, void* stream) {
  const char* what = "moe_unpack_fp8";
  moe_status st = check_pack(what, T, H, dt);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(codes, 16) || !scales || !good(x, 16)) return null_pointer(what);
  st = check_apart(what, {{"x", x, T * H * (dt == MOE_F32 ? 4 : 2)}},
                   {{"codes", codes, T * H}, {"scales", scales, T * (H / 32)}});
  if (st) return st;
  return hip_status(moe::launch_unpack_fp8(codes, scales, T, H, x, dt, (hipStream_t)stream), what);
}

}  // extern "C"
