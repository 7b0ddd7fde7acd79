"""The operators around the experts where their arithmetic or their choice of kernel is
at its edge: rows far from zero, slots of weight zero, no tokens, norms without biases,
rows that the workgroups take in turn at every width, every subset of the gradients.

Tolerances are bounds on rounding as in test_gpu_block_ops.py, whose helpers are used;
e = 2^-24 is one fp32 rounding.
"""
import itertools

import numpy as np
import pytest
import torch

from mixture_experts_layer_30_amd import binding as B
from test_gpu_block_ops import (DEV, DT, E24, EPS, Ref, close, columns, gate_factors, gates, gen,
                                hchain, pairs_of, params, randn, reference, check_residual,
                                routed, softmax_grad, stream_rows, tchain)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def workspace(T, H):
    return torch.full((max(B.moe_norm_workspace_bytes(T, H), 16),), 255, dtype=torch.uint8, device=DEV)


def nans(*shape):
    return torch.full(shape, float("nan"), device=DEV)


# ------------------------------------------------------------ rows far from zero

# additions one after the other in a sum over a row: 16 products a lane, 4 across 16
# lanes, 2 + 4 across the wavefronts; and the product with 1 / H
C = 28


class Far(Ref):
    """A layer norm of rows whose mean is far larger than their deviation, with a bound on
    what two passes can do.  A mean m of fp32 sums is off by at most d0 = C e mean|x|.  The
    centred values x - m and their own mean, at most d0, leave an error of
    dm = (C + 1) e (mean|x - mean| + d0): what is left goes by the deviation and no longer
    by the mean, but for the second order C e d0."""

    def __init__(self, x, n):
        eps = float(np.float32(n.eps))
        super().__init__(x, n.kind, n.weight, n.bias, eps)
        x = x.double()
        c = x - x.mean(1, keepdim=True)
        d0 = C * E24 * x.abs().mean(1, keepdim=True)
        dm = (C + 1) * E24 * (c.abs().mean(1, keepdim=True) + d0)
        # x - m, then less the mean of that: a rounding each
        e_c = dm + 2 * E24 * (c.abs() + d0)
        var = (c * c).mean(1, keepdim=True)
        # the mean of (x - m)^2 is var + d0^2 at most, from which the square of its mean is taken
        e_var = (C + 6) * E24 * (var + d0 * d0) + 2 * (d0 + dm) * dm
        assert (e_var <= 0.01 * (var + eps)).all()   # (so the root's error is half of it, and 1%)
        e_r = 0.51 * e_var / (var + eps) + 4 * E24
        self.e_xh = self.rstd * e_c + self.xh.abs() * e_r * 1.02
        self.e_out = self.e_xh * self.w.abs() + 3 * E24 * ((self.xh * self.w).abs() + self.b.abs())
        # the dot products go over x - m, whose magnitude is that of c and d0
        self.xm, self.e_r = self.xh.abs() + d0 * self.rstd, e_r

    def backward(self, g, eg):
        xh = self.xh
        m = (g * xh).mean(1, keepdim=True)
        em = (eg * self.xm + g.abs() * self.e_xh).mean(1, keepdim=True) + \
            (C + 4) * E24 * (g.abs() * self.xm).mean(1, keepdim=True)
        mg = g.mean(1, keepdim=True)
        o = g - xh * m - mg
        e = eg + self.e_xh * m.abs() + self.xm * em + 6 * E24 * (g.abs() + self.xm * m.abs() + mg.abs())
        e = e + eg.mean(1, keepdim=True) + (C + 4) * E24 * g.abs().mean(1, keepdim=True)
        return o * self.rstd, self.rstd * (e + (self.e_r + 4 * E24) * o.abs())


def far_rows(g, H):
    """Constant rows, and rows whose mean is 300 to 100 thousand times their deviation."""
    x = torch.randn(14, H, generator=g, device=DEV)
    for i, v in enumerate((1000.0, 100.0, -333.3, 1e4, 0.1, 1.0)):
        x[i] = v
    for i, v in enumerate((300.0, 1e3, -1e3, 1e4, -3e4, 1e5)):
        x[6 + i] += v
    x[12] = x[12] * 1e-3 + 5.0
    return x


@pytest.mark.parametrize("H", [1000, 3584, 7168, 8200, 16384])
def test_layer_norm_of_rows_far_from_zero(H):
    g = gen(H + 51)
    x = far_rows(g, H)
    T = x.shape[0]
    for n in (params(g, H, "f32", B.NORM_LAYER), B.Norm(B.NORM_LAYER, EPS)):
        o = torch.empty_like(x)
        B.moe_norm(x, n, o)
        ref = Far(x, n)
        close(o, ref.out, ref.e_out)
        # after a block too: gate 1 on a stream of zeros, and before the next, block's output 0
        zero, r, o2 = torch.zeros_like(x), torch.empty_like(x), torch.empty_like(x)
        B.moe_norm_residual(x, zero, n, B.Gate(), r)
        close(r, ref.out, ref.e_out + E24 * ref.out.abs())
        B.moe_norm_residual(zero, x, B.Norm(B.NORM_NONE), B.Gate(), r, pre=n, n=o2)
        assert torch.equal(r, x)
        close(o2, ref.out, ref.e_out)
        one = torch.ones(T, 1, device=DEV)
        B.moe_combine_norm_residual(x, one, zero, n, B.Gate(), r)
        close(r, ref.out, ref.e_out + E24 * ref.out.abs())


@pytest.mark.parametrize("H", [1000, 3584, 7168, 8200, 16384])
def test_layer_norm_gradients_of_rows_far_from_zero(H):
    g = gen(H + 52)
    x = far_rows(g, H)
    T = x.shape[0]
    n, d = params(g, H, "f32", B.NORM_LAYER), randn(g, T, H)
    gate = gates(g, T, H, "f32", True, True, 0.5)
    ref = Far(x, n)
    dx, dw, db = torch.empty_like(x), nans(H), nans(H)
    B.moe_norm_backward(d, x, n, dx, workspace(T, H), dweight=dw, dbias=db)
    gw = d.double() * ref.w
    close(dx, *ref.backward(gw, E24 * gw.abs()))
    e1 = ref.e_xh + 4 * E24 * ref.xm
    close(dw, *columns(d.double() * ref.xh, d.double().abs() * e1))
    close(db, *columns(d.double(), 0 * gw))
    dc, dq = nans(H), nans(T)
    B.moe_norm_residual_backward(d, x, n, gate, dx, workspace(T, H), dw, db, dc, dq)
    a, c = gate_factors(gate, T)
    du = a * c * d.double()
    gw = du * ref.w
    close(dx, *ref.backward(gw, 4 * E24 * gw.abs()))
    close(dw, *columns(du * ref.xh, du.abs() * e1))
    close(db, *columns(du, 4 * E24 * du.abs()))
    # from two sums each, put together at the end
    mag = (ref.xm * ref.w).abs() + ref.b.abs()
    ad = (a * d.double())
    err = (ad.abs() * (ref.e_out + 4 * E24 * mag)).sum(0) + (tchain(T) + 2) * E24 * (ad.abs() * mag).sum(0)
    close(dc, (ad * ref.out).sum(0), err)
    v = 0.5 * c * d.double()
    close(dq, (v * ref.out).sum(1), (v.abs() * (ref.e_out + (C + 8) * E24 * mag)).sum(1))


@pytest.mark.parametrize("H", [264, 3584, 7168])
def test_layer_norm_of_constant_bf16_rows(H):
    """Constant rows have the bias for a norm, to half a step of the result."""
    g = gen(H + 53)
    x = torch.tensor([3.0, 300.0, -1000.0, 0.1, 0.0], device=DEV)[:, None].expand(5, H).bfloat16().contiguous()
    n = params(g, H, "bf16", B.NORM_LAYER)
    o = torch.empty(5, H, device=DEV)
    B.moe_norm(x, n, o)
    # Far's bound at no deviation: (C + 3) e d0 / sqrt(eps), d0 = C e 1000, below 4e-6 a weight
    close(o, n.bias.double()[None].expand(5, H), 4e-6 * n.weight.double().abs()[None])


# ----------------------------------------------------------- slots of weight zero


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,E,K", [(5, 4, 2), (33, 64, 8), (9, 256, 8), (3, 200, 100)])
def test_gradients_next_to_a_slot_of_weight_zero(T, E, K, bad):
    """A slot of weight 0 adds nothing to the tokens, whatever its row holds: the logits'
    gradient goes on without it, and its own is 0."""
    H = 64
    ids, w, plan = routed(T, E, K, 16, B.PAD_BLOCK, T + E)
    w[:, -1] = 0.0
    inv = pairs_of(plan, T, K)
    g = gen(T + E + 54)
    rows, dout = randn(g, plan.cap, H), randn(g, T, H)
    rows[inv[:, -1]] = bad
    out, drows = torch.empty(T, H, device=DEV), torch.empty_like(rows)
    B.moe_unpermute(rows, w, plan, out)
    assert torch.isfinite(out).all()
    dw, o = nans(T, K), nans(T, E)
    B.moe_unpermute_backward(dout, rows, w, plan, drows, dw)
    assert torch.isfinite(dw[:, :-1]).all() and (drows[inv[:, -1]] == 0).all()
    B.moe_route_backward(ids, w, dw, o)
    clean = dw.clone()
    clean[:, -1] = 0.0
    ref, mag = softmax_grad(ids, w, clean, E)
    # the mean is taken in 64 bits: a rounding for the product and one for the result
    close(o, ref, 2 * E24 * ref.abs() + K * 2.0 ** -52 * mag)
    assert (o.gather(1, ids[:, -1:].long()) == 0).all()


@pytest.mark.parametrize("T,E,K,budget", [(1, 256, 8, False), (37, 37, 5, True), (3, 256, 256, True),
                                          (2049, 8, 2, False), (5, 200, 100, True)])
def test_route_backward_to_its_last_rounding(T, E, K, budget):
    """The mean over the slots is summed in 64 bits: the result is off by its own rounding
    and what 64 bits leave."""
    ids, w, _ = routed(T, E, K, 16, B.PAD_BLOCK, T + E + 1, budget)
    dw, o = randn(gen(T + 55), T, K), nans(T, E)
    B.moe_route_backward(ids, w, dw, o)
    ref, mag = softmax_grad(ids, w, dw, E)
    close(o, ref, 2 * K * 2.0 ** -52 * mag)


# ------------------------------------------------------------------ empty batches


def test_gradients_of_no_tokens_are_zero_whatever_the_parameters():
    x, v = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    bad = v.clone()
    bad[3], bad[7], bad[11] = float("inf"), float("nan"), float("-inf")
    n, gate = B.Norm(B.NORM_RMS, EPS, bad, bad), B.Gate(1.0, bad)
    d = [nans(64) for _ in range(5)]
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)
    B.moe_norm_backward(x, x, n, x, dweight=d[0], dbias=d[1], workspace=ws)
    B.moe_norm_residual_backward(x, x, n, gate, x, ws, d[2], d[3], d[4])
    for t in d:
        assert (t == 0).all()


# ------------------------------------------------- norms without biases, rows in turn

# (T, H, y, x, parameters): one row a workgroup, then more rows than workgroups at each
# width of a lane -- 8 elements, 16 by width, and 16 of bf16 rows past 4096
TURNS = [(5, 72, "bf16", "bf16", "bf16"), (128, 7168, "bf16", "bf16", "bf16"),
         (4500, 264, "bf16", "f32", "f32"), (1300, 3584, "f32", "f32", "bf16"),
         (700, 4096, "bf16", "f32", "bf16"), (1200, 4104, "bf16", "bf16", "f32"),
         (1100, 7168, "bf16", "bf16", "bf16"), (530, 8200, "bf16", "bf16", "bf16"),
         (300, 8200, "f32", "f32", "f32"), (300, 16384, "bf16", "f32", "f32"),
         (270, 12288, "f32", "bf16", "f32"),
         (8200, 2568, "bf16", "f32", "bf16")]   # one workgroup a CU where there is a gate


@pytest.mark.parametrize("kind,pre_kind", [(B.NORM_RMS, B.NORM_RMS), (B.NORM_LAYER, None),
                                           (B.NORM_RMS, B.NORM_LAYER)])
@pytest.mark.parametrize("T,H,ydt,xdt,pdt", TURNS)
def test_residual_without_biases(T, H, ydt, xdt, pdt, kind, pre_kind):
    """From y and from pair rows, without a gate, with a token's, and with a channel's."""
    g = gen(T + H + 61)
    y, x = stream_rows(g, T, H, ydt, kind), stream_rows(g, T, H, xdt, pre_kind)
    post = params(g, H, pdt, kind, bias=False)
    pre = params(g, H, pdt, pre_kind, bias=False) if pre_kind is not None else None
    w = torch.rand(T, 2, generator=g, device=DEV)
    pairs = randn(g, 2 * T, H, dt=ydt)
    c = torch.empty(T, H, device=DEV)
    B.moe_combine(pairs, w, c)
    from_y, from_c = reference(y, post), reference(c, post)
    for channel, token in ((False, False), (False, True), (True, False)):
        gate = gates(g, T, H, pdt, channel, token, 0.7)
        for ref in (from_y, from_c):
            r = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
            n = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV) if pre else None
            if ref is from_y:
                B.moe_norm_residual(y, x, post, gate, r, pre=pre, n=n)
            else:
                B.moe_combine_norm_residual(pairs, w, x, post, gate, r, pre=pre, n=n)
            check_residual(r, n, ref, x, gate, pre, T)


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,H,ydt,xdt,pdt", [(800, 8200, "bf16", "bf16", "bf16"), (530, 16384, "f32", "bf16", "f32"),
                                             (560, 12288, "bf16", "f32", "bf16")])
def test_wide_rows_in_turn(T, H, ydt, xdt, pdt, kind, bias):
    """Norms wider than 8192: more rows than workgroups, forward and all the gradients."""
    g = gen(T + H + 62)
    y = stream_rows(g, T, H, ydt, kind)
    n = params(g, H, pdt, kind, bias=bias)
    ref = reference(y, n)
    o = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
    B.moe_norm(y, n, o)
    close(o, ref.out, ref.e_out)
    dr, dres = randn(g, T, H, dt=xdt), randn(g, T, H, dt=ydt)
    d = dr.double()
    dx, dw, db = torch.full_like(y, float("nan")), nans(H), nans(H) if bias else None
    B.moe_norm_backward(dr, y, n, dx, workspace(T, H), dres=dres, dweight=dw, dbias=db)
    gw = d * ref.w
    want, err = ref.backward(gw, E24 * gw.abs())
    close(dx, want + dres.double(), err + E24 * (want.abs() + dres.double().abs()))
    close(dw, *columns(d * ref.xh, d.abs() * (ref.e_xh + E24 * ref.xh.abs())))
    if bias:
        close(db, *columns(d, 0 * d))
    check_gradients(dr, y, n, gates(g, T, H, pdt, True, True, 0.6), ref, subsets=[(1, bias, 1, 1)])


# ----------------------------------------------------- every subset of the gradients


def check_gradients(dr, y, post, gate, ref, subsets):
    T, H = y.shape
    a, c = gate_factors(gate, T)
    d = dr.double()
    du, ad = a * c * d, a * d
    gw = du * ref.w
    dy_ref = ref.backward(gw, 4 * E24 * gw.abs())
    mag = (ref.xh * ref.w).abs() + ref.b.abs()
    v = torch.tensor(gate.alpha, dtype=torch.float32).double().item() * c * d
    refs = [columns(du * ref.xh, du.abs() * (ref.e_xh + 4 * E24 * ref.xh.abs())),
            columns(du, 4 * E24 * du.abs()),
            ((ad * ref.out).sum(0), (ad.abs() * (ref.e_out + 3 * E24 * mag)).sum(0) +
             (tchain(T) + 2) * E24 * (ad.abs() * mag).sum(0)),
            ((v * ref.out).sum(1), (v.abs() * (ref.e_out + (hchain(H) + 4) * E24 * mag)).sum(1))]
    ws = workspace(T, H)
    for asked in subsets:
        outs = [nans(n) if on else None for on, n in zip(asked, (H, H, H, T))]
        dy = torch.full_like(y, float("nan"))
        B.moe_norm_residual_backward(dr, y, post, gate, dy, ws if any(asked[:3]) else None, *outs)
        close(dy, *dy_ref)
        for o, r in zip(outs, refs):
            if o is not None:
                close(o, *r)


@pytest.mark.parametrize("kind,bias", [(B.NORM_RMS, True), (B.NORM_RMS, False), (B.NORM_LAYER, True),
                                       (B.NORM_LAYER, False), (B.NORM_NONE, False)])
@pytest.mark.parametrize("T,H,ydt,xdt", [(515, 520, "bf16", "bf16"), (300, 3584, "bf16", "f32"),
                                         (4099, 128, "f32", "f32"), (300, 8200, "bf16", "bf16"),
                                         (2, 16384, "f32", "bf16")])
def test_every_subset_of_the_gradients(T, H, ydt, xdt, kind, bias):
    g = gen(T + H + 71)
    y, dr = stream_rows(g, T, H, ydt, kind), randn(g, T, H, dt=xdt)
    post, gate = params(g, H, "f32", kind, bias=bias), gates(g, T, H, "f32", True, True, 0.6)
    norm = (False, True) if kind != B.NORM_NONE else (False,)
    subsets = list(itertools.product(norm, norm, (False, True), (False, True)))
    check_gradients(dr, y, post, gate, reference(y, post), subsets)


# --------------------------------------------------------------- past 32-bit offsets


def test_gates_gradients_past_32_bit_offsets():
    """A token buffer of more than 2^32 bytes and 2^31 elements, whose last 40 rows carry
    nearly all of the sums over the tokens: one of them lost would show."""
    T, H = 300007, 7168
    g = gen(81)
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    n, gate = params(g, H, "f32", B.NORM_RMS), gates(g, T, H, "f32", True, True, 0.5)
    gate.token[-40:] += 1e5
    ws = workspace(T, H)
    dw, db, dc, dq = nans(H), nans(H), nans(H), nans(T)
    dy = torch.empty_like(y)
    B.moe_norm_residual_backward(y, y, n, gate, dy, ws, dw, db, dc, dq)   # y for the gradient too
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).to(DEV)
    ref, part = reference(y[some], n), B.Gate(gate.alpha, gate.channel, gate.token[some])
    a, c = gate_factors(part, 80)
    d = y[some].double()
    gw = a * c * d * ref.w
    close(dy[some], *ref.backward(gw, 4 * E24 * gw.abs()))
    v, mag = 0.5 * c * d, (ref.xh * ref.w).abs() + ref.b.abs()
    close(dq[some], (v * ref.out).sum(1), (v.abs() * (ref.e_out + (hchain(H) + 4) * E24 * mag)).sum(1))
    sums, mags, last = (torch.zeros(2, H, dtype=torch.float64, device=DEV) for _ in range(3))
    for lo in range(0, T, 8192):
        ref = reference(y[lo:lo + 8192], n)
        ad = 0.5 * gate.token[lo:lo + 8192].double()[:, None] * y[lo:lo + 8192].double()
        for i, v in enumerate((ad * ref.xh, ad)):
            sums[i] += v.sum(0)
            mags[i] += v.abs().sum(0)
    for i, v in enumerate(((a * d * reference(y[some], n).xh)[40:], (a * d)[40:])):
        last[i] = v.abs().sum(0) / 40
    # rows one after the other in a sum: T / 512 in a workgroup, then 512 / 64 + 8 + 8 of their
    # sums; a row's own value is right to hchain(H) roundings
    err = (hchain(H) + T / 512 + 30) * E24 * mags
    assert (err * 100 < last).all()   # the bound is far below what a row of the last adds
    ch, w, b = gate.channel.double(), n.weight.double(), n.bias.double()
    close(dw, ch * sums[0], ch.abs() * err[0])
    close(db, ch * sums[1], ch.abs() * err[1])
    close(dc, w * sums[0] + b * sums[1], w.abs() * err[0] + b.abs() * err[1])
