// C ABI of the operators around the layer pass: rows in the alignment's order
// and their gradients, and the norms, gate and residual sum of the block.  What
// each call computes is documented in include/moe_layer.h.
#include <math.h>
#include <stdint.h>

#include "block_checks.h"

namespace {

using namespace moe_checks;

constexpr int kMaxNormH = 16384;   // a workgroup's 1024 lanes hold 16 elements each

moe_status check_sorted(const char* what, int64_t T, int H, int E, int K, const moe_plan* plan) {
  moe_status st = check_rows(what, T, H);
  if (st) return st;
  st = check_routing(what, T, E, K);
  if (st) return st;
  return check_plan(what, plan, T, K, E);
}

moe_status check_norm(const char* what, const char* name, const moe_norm_params* n, bool none_ok,
                      moe::NormSpec* out) {
  if (!n) return fail(MOE_EINVAL, "%s: %s is NULL", what, name);
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER &&
      !(none_ok && n->kind == MOE_NORM_NONE))
    return fail(MOE_EINVAL, "%s: %s->kind = %d", what, name, (int)n->kind);
  if (!(n->eps >= 0.0f) || isinf(n->eps))
    return fail(MOE_EINVAL, "%s: %s->eps must be finite and >= 0", what, name);
  if (n->kind == MOE_NORM_NONE && (n->weight || n->bias))
    return fail(MOE_EINVAL, "%s: %s has a weight or bias but no norm", what, name);
  if (!optional(n->weight, 16) || !optional(n->bias, 16))
    return fail(MOE_EINVAL, "%s: %s has a misaligned weight or bias", what, name);
  *out = moe::NormSpec{n->kind, n->eps, n->weight, n->bias};
  return MOE_OK;
}

moe_status check_gate(const char* what, const moe_gate_params* g, moe::GateSpec* out) {
  if (!g) return fail(MOE_EINVAL, "%s: gate is NULL", what);
  if (!isfinite(g->alpha)) return fail(MOE_EINVAL, "%s: gate->alpha must be finite", what);
  if (!optional(g->channel, 16) || !optional(g->token, 4))
    return fail(MOE_EINVAL, "%s: gate has a misaligned pointer", what);
  *out = moe::GateSpec{g->alpha, g->channel, g->token};
  return MOE_OK;
}

moe_status check_norm_rows(const char* what, int64_t T, int H, int dt_a, int dt_b, int pdt) {
  moe_status st = check_rows(what, T, H);
  if (st) return st;
  if (H > kMaxNormH) return fail(MOE_EUNSUPPORTED, "%s: H = %d > %d", what, H, kMaxNormH);
  if (!valid_dtype(dt_a) || !valid_dtype(dt_b) || !valid_dtype(pdt))
    return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  return MOE_OK;
}

moe_status check_workspace(const char* what, int64_t T, int H, const void* workspace,
                           int64_t bytes) {
  const int64_t need = moe_norm_workspace_bytes(T, H);
  if (bytes < need)
    return fail(MOE_ECAPACITY, "%s: workspace %lld bytes < %lld required", what, (long long)bytes,
                (long long)need);
  if (T > 0 && !good(workspace, 16)) return null_pointer(what);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_permute(const void* x, moe_dtype dt, int64_t T, int H, int E, int K,
                       const moe_plan* plan, void* rows, void* stream) {
  const char* what = "moe_permute";
  moe_status st = check_sorted(what, T, H, E, K, plan);
  if (st) return st;
  if (!valid_dtype(dt)) return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  if (T == 0) return ok();
  if (!good(x, 16) || !good(rows, 16)) return null_pointer(what);
  return hip_status(moe::launch_permute(x, dt, T, K, H, plan_rows(plan, K), E, plan->cap, rows,
                                        true, (hipStream_t)stream),
                    what);
}

moe_status moe_permute_backward(const void* drows, moe_dtype dt, int64_t T, int H, int E, int K,
                                const moe_plan* plan, void* dx, void* stream) {
  const char* what = "moe_permute_backward";
  moe_status st = check_sorted(what, T, H, E, K, plan);
  if (st) return st;
  if (!valid_dtype(dt)) return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  if (T == 0) return ok();
  if (!good(drows, 16) || !good(dx, 16)) return null_pointer(what);
  return hip_status(moe::launch_unpermute(drows, dt, nullptr, nullptr, dt, T, K, H, plan->inv_pos,
                                          plan->cap, dx, dt, (hipStream_t)stream),
                    what);
}

moe_status moe_unpermute(const void* rows, moe_dtype rdt, const float* topk_w, const void* shared,
                         moe_dtype sdt, int64_t T, int H, int E, int K, const moe_plan* plan,
                         void* out, moe_dtype odt, void* stream) {
  const char* what = "moe_unpermute";
  moe_status st = check_sorted(what, T, H, E, K, plan);
  if (st) return st;
  if (!valid_dtype(rdt) || !valid_dtype(sdt) || !valid_dtype(odt))
    return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  if (T == 0) return ok();
  if (!good(rows, 16) || !good(out, 16) || !optional(topk_w, 4) || !optional(shared, 16))
    return null_pointer(what);
  return hip_status(moe::launch_unpermute(rows, rdt, topk_w, shared, sdt, T, K, H, plan->inv_pos,
                                          plan->cap, out, odt, (hipStream_t)stream),
                    what);
}

moe_status moe_unpermute_backward(const void* dout, const void* rows, moe_dtype dt,
                                  const float* topk_w, int64_t T, int H, int E, int K,
                                  const moe_plan* plan, void* drows, float* dw, void* stream) {
  const char* what = "moe_unpermute_backward";
  moe_status st = check_sorted(what, T, H, E, K, plan);
  if (st) return st;
  if (!valid_dtype(dt)) return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  if (T == 0) return ok();
  if (!drows && !dw) return fail(MOE_EINVAL, "%s: drows and dw are both NULL", what);
  if (dw && !topk_w) return fail(MOE_EINVAL, "%s: dw without topk_w", what);
  if (!good(dout, 16) || (dw ? !good(rows, 16) : !optional(rows, 16)) || !optional(topk_w, 4) ||
      !optional(drows, 16) || !optional(dw, 4))
    return null_pointer(what);
  return hip_status(moe::launch_unpermute_backward(dout, rows, dt, topk_w, T, K, H,
                                                   plan_rows(plan, K), E, plan->cap, drows, dw,
                                                   (hipStream_t)stream),
                    what);
}

moe_status moe_route_backward(const int32_t* topk_ids, const float* topk_w, const float* dw,
                              int64_t T, int E, int K, float* dlogits, void* stream) {
  const char* what = "moe_route_backward";
  moe_status st = check_routing(what, T, E, K);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(topk_ids, 4) || !good(topk_w, 4) || !good(dw, 4) || !good(dlogits, 4))
    return null_pointer(what);
  return hip_status(moe::launch_route_backward(topk_ids, topk_w, dw, T, E, K, dlogits,
                                               (hipStream_t)stream),
                    what);
}

int64_t moe_norm_workspace_bytes(int64_t T, int H) {
  if (T < 0 || T >= (int64_t)1 << 31 || H < 8 || H % 8 != 0 || H > kMaxNormH) return -1;
  return moe::norm_workspace_floats(T, H) * 4;
}

moe_status moe_norm(const void* x, moe_dtype xdt, int64_t T, int H, const moe_norm_params* norm,
                    moe_dtype pdt, void* n, moe_dtype odt, void* stream) {
  const char* what = "moe_norm";
  moe_status st = check_norm_rows(what, T, H, xdt, odt, pdt);
  if (st) return st;
  moe::NormSpec spec;
  st = check_norm(what, "norm", norm, false, &spec);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(x, 16) || !good(n, 16)) return null_pointer(what);
  return hip_status(moe::launch_norm(x, xdt, T, H, spec, pdt, n, odt, (hipStream_t)stream), what);
}

moe_status moe_norm_backward(const void* dn, moe_dtype odt, const void* x, moe_dtype xdt,
                             const void* dres, int64_t T, int H, const moe_norm_params* norm,
                             moe_dtype pdt, void* dx, float* dweight, float* dbias,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const char* what = "moe_norm_backward";
  moe_status st = check_norm_rows(what, T, H, odt, xdt, pdt);
  if (st) return st;
  moe::NormSpec spec;
  st = check_norm(what, "norm", norm, false, &spec);
  if (st) return st;
  if (!optional(dweight, 16) || !optional(dbias, 16)) return null_pointer(what);
  if (dweight || dbias) {
    st = check_workspace(what, T, H, workspace, workspace_bytes);
    if (st) return st;
  }
  if (T > 0 && (!good(dn, 16) || !good(x, 16) || !good(dx, 16) || !optional(dres, 16)))
    return null_pointer(what);
  const moe::GateSpec none{1.0f, nullptr, nullptr};
  return hip_status(moe::launch_norm_backward(dn, odt, x, xdt, dres, T, H, spec, none, pdt, dx,
                                              dweight, dbias, nullptr, nullptr, (float*)workspace,
                                              (hipStream_t)stream),
                    what);
}

// post, gate and, where n is asked for, pre (an empty batch's n may be NULL)
static moe_status check_residual(const char* what, int64_t T, const moe_norm_params* post,
                                 const moe_gate_params* gate, const moe_norm_params* pre,
                                 const void* n, moe::NormSpec* post_spec, moe::GateSpec* gate_spec,
                                 moe::NormSpec* pre_spec) {
  moe_status st = check_norm(what, "post", post, true, post_spec);
  if (st) return st;
  st = check_gate(what, gate, gate_spec);
  if (st) return st;
  *pre_spec = moe::NormSpec{MOE_NORM_NONE, 0.0f, nullptr, nullptr};
  if (n && !pre) return fail(MOE_EINVAL, "%s: n without pre", what);
  if (pre && !n && T > 0) return fail(MOE_EINVAL, "%s: pre without n", what);
  return pre ? check_norm(what, "pre", pre, false, pre_spec) : MOE_OK;
}

moe_status moe_norm_residual(const void* y, moe_dtype ydt, const void* x, moe_dtype xdt, int64_t T,
                             int H, const moe_norm_params* post, const moe_gate_params* gate,
                             moe_dtype pdt, void* r, const moe_norm_params* pre, void* n,
                             void* stream) {
  const char* what = "moe_norm_residual";
  moe_status st = check_norm_rows(what, T, H, ydt, xdt, pdt);
  if (st) return st;
  moe::NormSpec a, b;
  moe::GateSpec g;
  st = check_residual(what, T, post, gate, pre, n, &a, &g, &b);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(y, 16) || !good(x, 16) || !good(r, 16) || !optional(n, 16)) return null_pointer(what);
  return hip_status(moe::launch_norm_residual(y, ydt, x, xdt, T, H, a, g, pdt, r, b, n,
                                              (hipStream_t)stream),
                    what);
}

moe_status moe_combine_norm_residual(const void* y_pairs, moe_dtype ydt, const float* topk_w,
                                     const void* shared, moe_dtype sdt, const void* x,
                                     moe_dtype xdt, int64_t T, int K, int H,
                                     const moe_norm_params* post, const moe_gate_params* gate,
                                     moe_dtype pdt, void* r, const moe_norm_params* pre, void* n,
                                     void* stream) {
  const char* what = "moe_combine_norm_residual";
  moe_status st = check_norm_rows(what, T, H, ydt, xdt, pdt);
  if (st) return st;
  if (!valid_dtype(sdt)) return fail(MOE_EUNSUPPORTED, "%s: dtype", what);
  if (K < 1) return fail(MOE_EINVAL, "%s: K = %d", what, K);
  if (T * K >= (int64_t)1 << 31) return fail(MOE_EUNSUPPORTED, "%s: T*K must be < 2^31", what);
  moe::NormSpec a, b;
  moe::GateSpec g;
  st = check_residual(what, T, post, gate, pre, n, &a, &g, &b);
  if (st) return st;
  if (T == 0) return ok();
  if (!good(y_pairs, 16) || !good(topk_w, 4) || !good(x, 16) || !good(r, 16) || !optional(n, 16) ||
      !optional(shared, 16))
    return null_pointer(what);
  return hip_status(moe::launch_combine_norm_residual(y_pairs, ydt, topk_w, K, shared, sdt, x, xdt,
                                                      T, H, a, g, pdt, r, b, n,
                                                      (hipStream_t)stream),
                    what);
}

moe_status moe_norm_residual_backward(const void* dr, moe_dtype xdt, const void* y, moe_dtype ydt,
                                      int64_t T, int H, const moe_norm_params* post,
                                      const moe_gate_params* gate, moe_dtype pdt, void* dy,
                                      float* dweight, float* dbias, float* dchannel, float* dtoken,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
  const char* what = "moe_norm_residual_backward";
  moe_status st = check_norm_rows(what, T, H, xdt, ydt, pdt);
  if (st) return st;
  moe::NormSpec a, b;
  moe::GateSpec g;
  st = check_residual(what, T, post, gate, nullptr, nullptr, &a, &g, &b);
  if (st) return st;
  if (a.kind == MOE_NORM_NONE && (dweight || dbias))
    return fail(MOE_EINVAL, "%s: dweight or dbias without a norm", what);
  if ((dchannel && !g.channel) || (dtoken && !g.token))
    return fail(MOE_EINVAL, "%s: the gradient of a gate that is not there", what);
  if (!optional(dweight, 16) || !optional(dbias, 16) || !optional(dchannel, 16) ||
      !optional(dtoken, 4))
    return null_pointer(what);
  if (dweight || dbias || dchannel) {
    st = check_workspace(what, T, H, workspace, workspace_bytes);
    if (st) return st;
  }
  if (T > 0 && (!good(dr, 16) || !good(y, 16) || !good(dy, 16))) return null_pointer(what);
  return hip_status(moe::launch_norm_backward(dr, xdt, y, ydt, nullptr, T, H, a, g, pdt, dy,
                                              dweight, dbias, dchannel, dtoken, (float*)workspace,
                                              (hipStream_t)stream),
                    what);
}

}  // extern "C"
