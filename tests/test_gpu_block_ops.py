"""The operators around the experts against their definitions in 64 bits.

Tolerances are bounds on rounding, element by element.  u is half a step of the
output type (2^-24 fp32, 2^-8 bf16), e = 2^-24 one fp32 rounding.  A sum of n
products whose longest chain of additions is c is off by at most about
(c + 1) e sum|products|.  Chains: K + 1 for the sums over slots; H / 64 + 32 for
the sums over a row (a lane adds at most H / 64 products, the rest is a tree);
T / 256 + 300 for the sums over the tokens (more than they need: a lane adds at most
T / 256 + 1 rows, 15 sums of the rows beside, then those of up to 512 workgroups in 64
chains of 8, and 14 more).
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_30_amd import binding as B
from mixture_experts_layer_30_amd import synth
from mixture_experts_layer_30_amd.configs import LayerShape
from mixture_experts_layer_30_amd.layer import MoEBlock, MoELayer

pytestmark = pytest.mark.gpu
DEV = "cuda"
E24 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dt="f32", std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(DT[dt])


def close(got, ref, err):
    """|got - ref| <= half a step of got's type + err, element by element."""
    u = U[got.dtype]
    off = (got.double() - ref).abs()
    tol = u * (ref.abs() + err) + err + 1e-37
    bad = off > tol
    assert not bad.any(), (int(bad.sum()), float((off / tol).max()))
    assert torch.isfinite(got).all()


def hchain(H):
    return H / 64 + 32


def tchain(T):
    return T / 256 + 300


# ------------------------------------------------------------- rows by expert


def routed(T, E, K, block, pad, seed, budget=False, one_expert=False):
    """(ids, weights, plan), by the library's routing and alignment."""
    logits = synth.router_logits(T, E, "zipf", seed=seed, device=DEV)
    if one_expert:
        logits[:, 0] += 100.0
    ids = torch.empty(T, K, dtype=torch.int32, device=DEV)
    w = torch.empty(T, K, device=DEV)
    plan = B.Plan(T, K, E, block, DEV, pad=pad)
    k_tok = synth.budgets(T, range(K + 1), seed=seed).to(DEV) if budget else None
    B.moe_route_align(logits, K, ids, w, plan, pad=pad, k_tok=k_tok)
    return ids, w, plan


# T, H, E, K, block, padding, type, budgets, all tokens on one expert
SORTED = [
    (1, 8, 1, 1, 1, B.PAD_BLOCK, "bf16", False, False),
    (1, 7168, 256, 8, 16, B.PAD_BLOCK, "bf16", False, False),
    (3, 64, 4, 4, 128, B.PAD_BLOCK, "f32", False, False),
    (37, 1000, 37, 5, 16, B.PAD_MAX, "f32", False, False),
    (64, 264, 8, 2, 64, B.PAD_BLOCK, "bf16", True, False),
    (129, 520, 16, 16, 7, B.PAD_BLOCK, "bf16", True, False),
    (200, 2056, 8, 2, 128, B.PAD_BLOCK, "bf16", False, True),
    (257, 3584, 64, 8, 1, B.PAD_BLOCK, "f32", True, False),
    (300, 1032, 256, 13, 1000, B.PAD_BLOCK, "bf16", False, False),
    (33, 16392, 5, 3, 16, B.PAD_MAX, "bf16", True, False),
    (70, 136, 9, 2, 1, B.PAD_MAX, "bf16", False, False),     # blocks of one row, and padding all the same
    (900, 1024, 4, 1, 128, B.PAD_MAX, "f32", False, True),   # one expert's rows, three slots of padding
]


def pairs_of(plan, T, K):
    return plan.inv_pos[:T * K].view(T, K).long()


@pytest.mark.parametrize("T,H,E,K,block,pad,dt,budget,one", SORTED)
def test_permute(T, H, E, K, block, pad, dt, budget, one):
    _, _, plan = routed(T, E, K, block, pad, T + H, budget, one)
    x = randn(gen(1), T, H, dt=dt)
    rows = torch.full((plan.cap + 2, H), -7.0, dtype=DT[dt], device=DEV)
    B.moe_permute(x, plan, rows)
    sid = plan.sorted_ids[:plan.cap].long()
    padded = int(plan.expert_offsets[E])
    want = torch.full((plan.cap + 2, H), -7.0, dtype=DT[dt], device=DEV)
    want[:padded] = 0
    held = torch.nonzero(sid < T * K)[:, 0]
    want[held] = x[sid[held] // K]
    assert torch.equal(rows, want)   # copies, zeros, and rows past the end as they were


@pytest.mark.parametrize("T,H,E,K,block,pad,dt,budget,one", SORTED)
def test_permute_backward(T, H, E, K, block, pad, dt, budget, one):
    _, _, plan = routed(T, E, K, block, pad, T + H, budget, one)
    drows = randn(gen(2), plan.cap, H, dt=dt)
    held = plan.sorted_ids[:plan.cap] < T * K
    drows[~held] = float("nan")   # padding rows take no part
    dx = torch.full((T, H), float("nan"), dtype=DT[dt], device=DEV)
    B.moe_permute_backward(drows, plan, dx)
    inv = pairs_of(plan, T, K)
    v = drows[inv.clamp(min=0)].double().masked_fill((inv < 0)[:, :, None], 0.0)
    close(dx, v.sum(1), (K + 2) * E24 * v.abs().sum(1))


@pytest.mark.parametrize("shared,out", [(None, "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,H,E,K,block,pad,dt,budget,one", SORTED)
def test_unpermute(T, H, E, K, block, pad, dt, budget, one, shared, out):
    _, w, plan = routed(T, E, K, block, pad, T + H, budget, one)
    rows = randn(gen(3), plan.cap, H, dt=dt)
    rows[plan.sorted_ids[:plan.cap] >= T * K] = float("nan")
    sh = randn(gen(4), T, H, dt=shared) if shared else None
    o = torch.full((T, H), float("nan"), dtype=DT[out], device=DEV)
    B.moe_unpermute(rows, w, plan, o, shared=sh)
    inv = pairs_of(plan, T, K)
    y = rows[inv.clamp(min=0)].masked_fill((inv < 0)[:, :, None], 0.0)
    v = y.double() * w.double()[:, :, None]
    ref, mag = v.sum(1), v.abs().sum(1)
    if sh is not None:
        ref, mag = ref + sh.double(), mag + sh.double().abs()
    close(o, ref, (K + 2) * E24 * mag)
    # the same sums as the combine's over pair rows, bit for bit
    c = torch.empty_like(o)
    B.moe_combine(y.view(T * K, H).contiguous(), w, c, shared=sh)
    assert torch.equal(o, c)


def test_unpermute_skips_rows_of_weight_zero():
    T, H, E, K = 5, 64, 4, 2
    _, w, plan = routed(T, E, K, 16, B.PAD_BLOCK, 5)
    rows = randn(gen(5), plan.cap, H)
    w[:, 1] = 0.0
    rows[pairs_of(plan, T, K)[:, 1]] = float("inf")
    o = torch.empty(T, H, device=DEV)
    B.moe_unpermute(rows, w, plan, o)
    v = rows[pairs_of(plan, T, K)[:, 0]].double() * w[:, :1].double()
    close(o, v, E24 * v.abs())


@pytest.mark.parametrize("T,H,E,K,block,pad,dt,budget,one", SORTED)
def test_unpermute_backward(T, H, E, K, block, pad, dt, budget, one):
    _, w, plan = routed(T, E, K, block, pad, T + H, budget, one)
    rows = randn(gen(6), plan.cap, H, dt=dt)
    rows[plan.sorted_ids[:plan.cap] >= T * K] = float("nan")
    dout = randn(gen(7), T, H, dt=dt)
    drows = torch.full((plan.cap + 1, H), -7.0, dtype=DT[dt], device=DEV)
    dw = torch.full((T, K), float("nan"), device=DEV)
    B.moe_unpermute_backward(dout, rows, w, plan, drows, dw)
    inv = pairs_of(plan, T, K)
    y = rows[inv.clamp(min=0)].double().masked_fill((inv < 0)[:, :, None], 0.0)
    p = y * dout.double()[:, None]
    close(dw, p.sum(2), hchain(H) * E24 * p.abs().sum(2))
    used = inv >= 0
    g = (dout.double()[:, None] * w.double()[:, :, None])[used]
    close(drows[inv[used]], g, E24 * g.abs())
    pad_rows = torch.nonzero(plan.sorted_ids[:plan.cap] >= T * K)[:, 0]
    padded = int(plan.expert_offsets[E])
    assert (drows[pad_rows[pad_rows < padded]] == 0).all()
    assert (drows[pad_rows[pad_rows >= padded]] == -7).all() and (drows[plan.cap:] == -7).all()
    # each gradient on its own, and the rows' in place: the same bits
    one_r, one_w = torch.full_like(drows, -7.0), torch.empty_like(dw)
    B.moe_unpermute_backward(dout, None, w, plan, one_r)
    B.moe_unpermute_backward(dout, rows, w, plan, dw=one_w)
    assert torch.equal(one_r, drows) and torch.equal(one_w, dw)
    buf = torch.full_like(drows, -7.0)
    buf[:padded] = rows[:padded]
    B.moe_unpermute_backward(dout, buf, w, plan, buf, one_w)
    assert torch.equal(buf, drows) and torch.equal(one_w, dw)
    # unit weights: the rows' gradient is the tokens' copy
    B.moe_unpermute_backward(dout, None, None, plan, one_r)
    B.moe_permute(dout, plan, drows)
    assert torch.equal(one_r, drows)


def softmax_grad(ids, w, dw, E):
    """dlogits in 64 bits, and the sum of the magnitudes behind each"""
    w, dw = w.double(), dw.double()
    used = (ids >= 0) & (ids < E)
    w, dw = w.masked_fill(~used, 0.0), dw.masked_fill(~used, 0.0)
    s, m = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    at = torch.where(used, ids.long(), E)
    z = torch.zeros(ids.shape[0], E + 1, dtype=torch.float64, device=DEV)
    return (z.scatter_add(1, at, w * (dw - s))[:, :E],
            z.scatter_add(1, at, w * (dw.abs() + m))[:, :E])


@pytest.mark.parametrize("T,E,K,budget", [(1, 1, 1, False), (1, 256, 8, False), (37, 37, 5, True),
                                          (300, 64, 8, True), (3, 256, 256, True), (65, 65, 65, False),
                                          (2049, 8, 2, False), (5, 200, 100, True)])
def test_route_backward(T, E, K, budget):
    ids, w, _ = routed(T, E, K, 16, B.PAD_BLOCK, T + E, budget)
    dw = randn(gen(8), T, K)
    dw[ids < 0] = float("nan")   # unused slots take no part
    o = torch.full((T, E), float("nan"), device=DEV)
    B.moe_route_backward(ids, w, dw, o)
    ref, mag = softmax_grad(ids, w, dw.nan_to_num(0.0), E)
    close(o, ref, (K / 64 + 10) * E24 * mag)   # (the mean is summed in 64 bits: more than it needs)
    if K == 1:
        assert (o == 0).all()


def test_route_backward_sums_an_expert_listed_twice():
    ids = torch.tensor([[3, 3, 1], [0, -1, 9]], dtype=torch.int32, device=DEV)   # 9: past E
    w = torch.tensor([[0.5, 0.25, 0.25], [0.75, 0.0, 0.25]], device=DEV)
    dw = torch.tensor([[1.0, 2.0, -3.0], [1.5, 7.0, 8.0]], device=DEV)
    o = torch.empty(2, 5, device=DEV)
    B.moe_route_backward(ids, w, dw, o)
    ref, mag = softmax_grad(ids, w, dw, 5)
    close(o, ref, 12 * E24 * mag)


def test_route_backward_next_to_a_weight_of_one():
    """One expert's weight 1 - 2^-20: its gradient is the small rest of two near-equal numbers,
    right to its own rounding and not to that of the numbers."""
    ids = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1 - 2.0 ** -20, 2.0 ** -20]], device=DEV)
    dw = torch.tensor([[1.2345678, -0.7654321]], device=DEV)
    o = torch.empty(1, 3, device=DEV)
    B.moe_route_backward(ids, w, dw, o)
    ref, _ = softmax_grad(ids, w, dw, 3)
    close(o, ref, 2 * 2.0 ** -52 * (w * dw).double().abs().sum())


def test_route_backward_against_differences():
    """The gradient of sum(c * weights) along a direction, against the central
    difference of the routing weights' definition (fixed experts) in 64 bits."""
    T, E, K = 40, 16, 4
    logits = synth.router_logits(T, E, "uniform", seed=3, device=DEV)
    ids = torch.empty(T, K, dtype=torch.int32, device=DEV)
    w = torch.empty(T, K, device=DEV)
    B.moe_route(logits, K, ids, w)
    c, d = randn(gen(9), T, K), randn(gen(10), T, E)
    o = torch.empty(T, E, device=DEV)
    B.moe_route_backward(ids, w, c, o)

    def f(l):
        return (torch.softmax(l.gather(1, ids.long()), 1) * c.double()).sum()
    h = 1e-5
    diff = (f(logits.double() + h * d.double()) - f(logits.double() - h * d.double())) / (2 * h)
    # weights are right to 1e-5 (the routing's own bar), the difference to about h^2
    assert abs(float((o.double() * d.double()).sum() - diff)) <= 4e-5 * float(c.abs().sum())


def test_rows_past_32_bit_offsets():
    """A row buffer of more than 2^32 bytes and 2^31 elements."""
    T, H, E, K = 40001, 7168, 8, 8
    ids, w, plan = routed(T, E, K, 128, B.PAD_BLOCK, 11)
    assert plan.cap * H > 2 ** 31
    x = randn(gen(11), T, H, dt="bf16")
    rows = torch.empty(plan.cap, H, dtype=torch.bfloat16, device=DEV)
    B.moe_permute(x, plan, rows)
    padded = int(plan.expert_offsets[E])
    sid = plan.sorted_ids[:padded].long()
    for a in range(0, padded, 32768):
        s = sid[a:min(a + 32768, padded)]
        want = x[(s // K).clamp(max=T - 1)].masked_fill((s >= T * K)[:, None], 0.0)
        assert torch.equal(rows[a:a + s.numel()], want), a
    o = torch.empty_like(x)
    B.moe_unpermute(rows, w, plan, o)   # K copies of x with weights that sum to one
    ref = x.double() * w.double().sum(1, keepdim=True)
    close(o, ref, (K + 2) * E24 * ref.abs())
    dw = torch.empty_like(w)
    B.moe_unpermute_backward(x, rows, w, plan, rows, dw)   # in place
    sq = (x.double() ** 2).sum(1, keepdim=True).expand(T, K)
    close(dw, sq, hchain(H) * E24 * sq)
    for k in (0, K - 1):
        t = torch.arange(T - 500, T, device=DEV)
        g = x[t].double() * w[t, k].double()[:, None]
        close(rows[pairs_of(plan, T, K)[t, k]], g, E24 * g.abs())


# ---------------------------------------------------------------- norms, gates

EPS = 1e-6


class Ref:
    """A norm of rows in 64 bits, with a bound on the error of its normalised rows."""

    def __init__(self, x, kind, w, b, eps=EPS):
        x = x.double()
        H = x.shape[1]
        c = hchain(H)
        self.kind, self.H, self.c = kind, H, c
        one = torch.ones(H, dtype=torch.float64, device=DEV)
        self.w = one if w is None else w.double()
        self.b = 0 * one if b is None else b.double()
        if kind == B.NORM_NONE:
            self.rstd = torch.ones(x.shape[0], 1, dtype=torch.float64, device=DEV)
            self.xh, self.e_xh = x, torch.zeros_like(x)
        else:
            mean = x.mean(1, keepdim=True) if kind == B.NORM_LAYER else 0.0
            d = x - mean
            self.rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
            self.xh = d * self.rstd
            # the mean is off by c e mean|x|; the sum of squares relatively by (c + 2) e,
            # so rstd by half of it, the quotient and root a few more
            dm = (c + 2) * E24 * x.abs().mean(1, keepdim=True) if kind == B.NORM_LAYER else 0.0
            self.e_xh = E24 * (c / 2 + 8) * self.xh.abs() + dm * self.rstd
        self.out = self.xh * self.w + self.b
        self.e_out = self.e_xh * self.w.abs() + 3 * E24 * ((self.xh * self.w).abs() + self.b.abs())

    def backward(self, g, eg):
        """Gradient of the row from g = d out * weight, known to eg; and its error."""
        if self.kind == B.NORM_NONE:
            return g, eg
        c, xh = self.c, self.xh
        m = (g * xh).mean(1, keepdim=True)
        em = (eg * xh.abs() + g.abs() * self.e_xh).mean(1, keepdim=True) + \
            (c + 2) * E24 * (g * xh).abs().mean(1, keepdim=True)
        o = g - xh * m
        e = eg + self.e_xh * m.abs() + xh.abs() * em + 4 * E24 * (g.abs() + (xh * m).abs())
        if self.kind == B.NORM_LAYER:
            mg = g.mean(1, keepdim=True)
            o = o - mg
            e = e + eg.mean(1, keepdim=True) + (c + 2) * E24 * g.abs().mean(1, keepdim=True) + \
                4 * E24 * mg.abs()
        return o * self.rstd, self.rstd * (e + (c / 2 + 8) * E24 * o.abs())


def columns(v, ev):
    """Sum down the tokens of v (known to ev) and its error"""
    return v.sum(0), ev.sum(0) + tchain(v.shape[0]) * E24 * v.abs().sum(0)


def stream_rows(g, T, H, dt, kind):
    """Rows of differing scales, one of zeros; layer norms also get rows far from zero."""
    x = torch.randn(T, H, generator=g, device=DEV) * (0.1 + 3 * torch.rand(T, 1, generator=g, device=DEV))
    if T > 2:
        x[1] = 0.0
        if kind == B.NORM_LAYER:
            x[2] += 300.0
    return x.to(DT[dt])


def params(g, H, dt, kind, weight=True, bias=True):
    if kind == B.NORM_NONE:
        return B.Norm(kind, EPS)
    return B.Norm(kind, EPS, randn(g, H, dt=dt, std=0.3, mean=1.0) if weight else None,
                  randn(g, H, dt=dt, std=0.3) if bias else None)


def reference(x, n):
    return Ref(x, n.kind, n.weight, n.bias, float(np.float32(n.eps)))


# T, H, x, out, parameters, weight, bias
NORMS = [
    (1, 8, "bf16", "bf16", "bf16", True, True),
    (1, 7168, "bf16", "bf16", "f32", True, False),
    (3, 64, "f32", "f32", "f32", False, False),
    (5, 520, "bf16", "f32", "bf16", False, True),
    (33, 1000, "f32", "bf16", "f32", True, True),
    (700, 264, "bf16", "bf16", "bf16", True, False),
    (300, 3584, "f32", "f32", "bf16", True, True),
    (5000, 128, "bf16", "bf16", "f32", True, True),
    (7, 8200, "bf16", "bf16", "bf16", True, True),
    (4, 16384, "f32", "bf16", "f32", True, True),
]


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER])
@pytest.mark.parametrize("T,H,xdt,odt,pdt,weight,bias", NORMS)
def test_norm(T, H, xdt, odt, pdt, weight, bias, kind):
    g = gen(T + H)
    x = stream_rows(g, T, H, xdt, kind)
    n = params(g, H, pdt, kind, weight, bias)
    o = torch.full((T, H), float("nan"), dtype=DT[odt], device=DEV)
    B.moe_norm(x, n, o)
    ref = reference(x, n)
    close(o, ref.out, ref.e_out)
    if xdt == odt:   # in place
        B.moe_norm(x, n, x)
        assert torch.equal(x, o)


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER])
@pytest.mark.parametrize("T,H,xdt,odt,pdt,weight,bias", NORMS)
def test_norm_backward(T, H, xdt, odt, pdt, weight, bias, kind):
    g = gen(T + H + 1)
    x = stream_rows(g, T, H, xdt, kind)
    n = params(g, H, pdt, kind, weight, bias)
    dn, dres = randn(g, T, H, dt=odt), randn(g, T, H, dt=xdt)
    ws = torch.full((B.moe_norm_workspace_bytes(T, H),), 255, dtype=torch.uint8, device=DEV)
    ref = reference(x, n)
    d = dn.double()
    gw = d * ref.w
    dx, ex = ref.backward(gw, E24 * gw.abs())

    def run(**k):
        o = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
        dw, db = (torch.full((H,), float("nan"), device=DEV) for _ in range(2))
        B.moe_norm_backward(dn, x, n, o, ws, dweight=dw, dbias=db, **k)
        return o, dw, db
    o, dw, db = run()
    close(o, dx, ex)
    w_ref, w_err = columns(d * ref.xh, d.abs() * (ref.e_xh + E24 * ref.xh.abs()))
    close(dw, w_ref, w_err)
    close(db, *columns(d, 0 * d))
    o2, dw2, db2 = run(dres=dres)
    close(o2, dx + dres.double(), ex + E24 * (dx.abs() + dres.double().abs()))
    assert torch.equal(dw, dw2) and torch.equal(db, db2)
    # in place over the gradient that passes by, and without parameter gradients or workspace
    inplace = dres.clone()
    B.moe_norm_backward(dn, x, n, inplace, dres=inplace)
    assert torch.equal(inplace, o2)
    if xdt == odt:
        inplace = dn.clone()
        B.moe_norm_backward(inplace, x, n, inplace, dres=dres)
        assert torch.equal(inplace, o2)


# T, H, y, x, parameters, post norm, channel gate, token gate, alpha, next norm
RESIDUALS = [
    (1, 8, "bf16", "bf16", "bf16", B.NORM_RMS, True, True, 1.0, B.NORM_RMS),
    (1, 7168, "bf16", "bf16", "bf16", B.NORM_RMS, False, False, 1.0, B.NORM_RMS),
    (3, 64, "f32", "f32", "f32", B.NORM_NONE, False, False, 0.25, None),
    (6, 520, "bf16", "f32", "f32", B.NORM_LAYER, True, False, -0.5, B.NORM_LAYER),
    (33, 1000, "f32", "bf16", "bf16", B.NORM_LAYER, False, True, 1.7, B.NORM_RMS),
    (301, 264, "bf16", "bf16", "bf16", B.NORM_NONE, True, True, 0.1, B.NORM_LAYER),
    (300, 3584, "bf16", "f32", "bf16", B.NORM_RMS, True, False, 0.0, B.NORM_RMS),
    (4099, 72, "f32", "f32", "f32", B.NORM_RMS, False, True, 1.0, None),
    (7, 8200, "bf16", "bf16", "f32", B.NORM_RMS, True, True, 0.3, B.NORM_LAYER),
    (4, 16384, "f32", "f32", "bf16", B.NORM_LAYER, True, True, 1.0, B.NORM_RMS),
]


def gates(g, T, H, pdt, channel, token, alpha):
    return B.Gate(alpha, randn(g, H, dt=pdt, std=0.4, mean=0.5) if channel else None,
                  torch.rand(T, generator=g, device=DEV) if token else None)


def gate_factors(gate, T):
    """(alpha * token [T,1], channel [H] or 1) in 64 bits"""
    a = torch.full((T, 1), float(np.float32(gate.alpha)), dtype=torch.float64, device=DEV)
    if gate.token is not None:
        a = a * gate.token.double()[:, None]
    return a, 1.0 if gate.channel is None else gate.channel.double()


def residual_ref(ref, x, gate, T):
    a, c = gate_factors(gate, T)
    u = a * c * ref.out
    r = x.double() + u
    return r, (a * c).abs() * ref.e_out + 4 * E24 * u.abs() + E24 * r.abs()


def check_residual(r, n, ref, x, gate, pre, T):
    want, err = residual_ref(ref, x, gate, T)
    close(r, want, err)
    if pre is not None:
        nxt = reference(want, pre)
        # an error of err in the row moves the norm by rstd * (err + what it moves the
        # statistics by), at most rstd * (err + (1 + |xh|) * its root mean square) and the mean's
        rms = (err * err).mean(1, keepdim=True).sqrt()
        more = nxt.rstd * (err + (1 + nxt.xh.abs()) * rms) * nxt.w.abs()
        close(n, nxt.out, nxt.e_out + 1.01 * more)


@pytest.mark.parametrize("T,H,ydt,xdt,pdt,kind,channel,token,alpha,pre_kind", RESIDUALS)
def test_norm_residual(T, H, ydt, xdt, pdt, kind, channel, token, alpha, pre_kind):
    g = gen(T + H + 2)
    y, x = stream_rows(g, T, H, ydt, kind), stream_rows(g, T, H, xdt, pre_kind)
    post, gate = params(g, H, pdt, kind), gates(g, T, H, pdt, channel, token, alpha)
    pre = params(g, H, pdt, pre_kind) if pre_kind is not None else None
    r = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
    n = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV) if pre else None
    B.moe_norm_residual(y, x, post, gate, r, pre=pre, n=n)
    check_residual(r, n, reference(y, post), x, gate, pre, T)
    # in place: r over x, n over y
    x2, y2 = x.clone(), y.clone()
    B.moe_norm_residual(y2, x2, post, gate, x2, pre=pre, n=y2 if pre else None)
    assert torch.equal(x2, r) and (pre is None or torch.equal(y2, n))


@pytest.mark.parametrize("K,shared", [(1, None), (2, "f32"), (5, "bf16"), (8, "f32")])
@pytest.mark.parametrize("T,H,ydt,xdt,pdt,kind,channel,token,alpha,pre_kind", RESIDUALS)
def test_combine_norm_residual(T, H, ydt, xdt, pdt, kind, channel, token, alpha, pre_kind, K, shared):
    if T * K > 5000:
        T = 5000 // K
    g = gen(T + H + K)
    y, x = randn(g, T * K, H, dt=ydt), stream_rows(g, T, H, xdt, pre_kind)
    w = torch.softmax(torch.randn(T, K, generator=g, device=DEV), 1)
    if K > 1:
        w[0, -1] = 0.0
        y[K - 1] = float("nan")   # a slot of weight zero: its row is not read
    if T > 4:   # a token without experts
        w[3] = 0.0
    sh = randn(g, T, H, dt=shared) if shared else None
    post, gate = params(g, H, pdt, kind), gates(g, T, H, pdt, channel, token, alpha)
    pre = params(g, H, pdt, pre_kind) if pre_kind is not None else None
    r = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
    n = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV) if pre else None
    B.moe_combine_norm_residual(y, w, x, post, gate, r, pre=pre, n=n, shared=sh)
    # the combine in fp32 (the same sums bit for bit), then the norm and residual sum from it
    c = torch.empty(T, H, device=DEV)
    B.moe_combine(y, w, c, shared=sh)
    ref = reference(c, post)
    check_residual(r, n, ref, x, gate, pre, T)
    # the two calls one after the other, to the same bound: the statistics are sums over the
    # row in an order that goes by the types (a lane holds 8 neighbours of bf16 rows, 4 of
    # fp32 ones), so the bits agree only where y is fp32 in both
    r2 = torch.empty_like(r)
    B.moe_norm_residual(c, x, post, gate, r2)
    check_residual(r2, None, ref, x, gate, None, T)
    if ydt == "f32":
        assert torch.equal(r, r2)


@pytest.mark.parametrize("T,H,ydt,xdt,pdt,kind,channel,token,alpha,pre_kind", RESIDUALS)
def test_norm_residual_backward(T, H, ydt, xdt, pdt, kind, channel, token, alpha, pre_kind):
    g = gen(T + H + 3)
    y, dr = stream_rows(g, T, H, ydt, kind), randn(g, T, H, dt=xdt)
    post, gate = params(g, H, pdt, kind), gates(g, T, H, pdt, channel, token, alpha)
    if token and T > 4:
        gate.token[4] = 0.0   # a gate that is shut still has a gradient
    ws = torch.full((B.moe_norm_workspace_bytes(T, H),), 255, dtype=torch.uint8, device=DEV)
    norm = kind != B.NORM_NONE
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    dy = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV)
    dw, db = (nan(H), nan(H)) if norm else (None, None)
    dc, dq = nan(H) if channel else None, nan(T) if token else None
    B.moe_norm_residual_backward(dr, y, post, gate, dy, ws, dweight=dw, dbias=db, dchannel=dc,
                                 dtoken=dq)
    ref = reference(y, post)
    a, c = gate_factors(gate, T)
    d = dr.double()
    du = a * c * d
    gw = du * ref.w
    want, err = ref.backward(gw, 4 * E24 * gw.abs())
    close(dy, want, err)
    if norm:
        close(dw, *columns(du * ref.xh, du.abs() * (ref.e_xh + 4 * E24 * ref.xh.abs())))
        close(db, *columns(du, 4 * E24 * du.abs()))
    # u = xh w + b: both sums are taken of the two terms apart and put together at the end
    # (w sum(..xh) + b sum(..)), so their roundings go by the terms' magnitudes
    u, eu = ref.out, ref.e_out
    mag = (ref.xh * ref.w).abs() + ref.b.abs()
    if channel:
        ad = a * d
        err = (ad.abs() * (eu + 3 * E24 * mag)).sum(0) + (tchain(T) + 2) * E24 * (ad.abs() * mag).sum(0)
        close(dc, (ad * u).sum(0), err)
    if token:
        v = float(np.float32(alpha)) * c * d
        close(dq, (v * u).sum(1), (v.abs() * (eu + (hchain(H) + 4) * E24 * mag)).sum(1))
    # without parameter gradients, in place
    if norm or not (channel or token):
        y2 = y.clone()
        B.moe_norm_residual_backward(dr, y2, post, gate, y2)
        assert torch.equal(y2, dy)
    if xdt == ydt:
        d2 = dr.clone()
        B.moe_norm_residual_backward(d2, y, post, gate, d2)
        assert torch.equal(d2, dy)


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER])
def test_rows_of_tiny_values_without_eps(kind):
    """Rows of 1e-15: their deviation's reciprocal cubed is past fp32."""
    T, H = 3, 264
    g = gen(23)
    x, dn = randn(g, T, H) * 1e-15, randn(g, T, H) * 1e-15
    n = B.Norm(kind, 0.0, randn(g, H, mean=1.0))
    o, dx = torch.empty_like(x), torch.empty_like(x)
    B.moe_norm(x, n, o)
    ref = Ref(x, kind, n.weight, None, 0.0)
    close(o, ref.out, ref.e_out)
    B.moe_norm_backward(dn, x, n, dx)
    gw = dn.double() * ref.w
    close(dx, *ref.backward(gw, E24 * gw.abs()))


def test_norms_past_32_bit_offsets():
    """Token buffers of more than 2^32 bytes and 2^31 elements: the rows at both ends, and
    the sums over all of them."""
    T, H = 300007, 7168
    assert T * H > 2 ** 31
    g = gen(24)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    n, gate = params(g, H, "f32", B.NORM_RMS), gates(g, T, H, "f32", True, True, 0.5)
    o, r = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(B.moe_norm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    dw, db, dc = (torch.empty(H, device=DEV) for _ in range(3))
    dq = torch.empty(T, device=DEV)
    B.moe_norm(x, n, o)
    B.moe_norm_residual(o, x, n, gate, r)
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).to(DEV)
    ref = reference(x[some], n)
    close(o[some], ref.out, ref.e_out)
    part = B.Gate(gate.alpha, gate.channel, gate.token[some])
    check_residual(r[some], None, reference(o[some], n), x[some], part, None, some.numel())
    B.moe_norm_residual_backward(x, o, n, gate, r, ws, dw, db, dc, dq)   # x for the gradient
    ref = reference(o[some], n)
    a, c = gate_factors(part, some.numel())
    gw = a * c * x[some].double() * ref.w
    close(r[some], *ref.backward(gw, 4 * E24 * gw.abs()))
    sums = torch.zeros(2, H, dtype=torch.float64, device=DEV)
    mags = torch.zeros(2, H, dtype=torch.float64, device=DEV)
    for lo in range(0, T, 8192):
        ref = reference(o[lo:lo + 8192], n)
        ad = gate_factors(B.Gate(gate.alpha, None, gate.token[lo:lo + 8192]), ref.xh.shape[0])[0] * x[lo:lo + 8192].double()
        for i, v in enumerate((ad * ref.xh, ad)):
            sums[i] += v.sum(0)
            mags[i] += v.abs().sum(0)
    # a row's xh is right to hchain(H) roundings, a sum over the tokens to tchain(T) more
    err = (hchain(H) + tchain(T)) * E24 * mags
    ch, w, b = gate.channel.double(), n.weight.double(), n.bias.double()
    close(dw, ch * sums[0], ch.abs() * err[0])
    close(db, ch * sums[1], ch.abs() * err[1])
    close(dc, w * sums[0] + b * sums[1], w.abs() * err[0] + b.abs() * err[1])


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER])
def test_gradients_against_differences(kind):
    """Gradients of sum(c r) along a direction of every input, against central
    differences of the definition in 64 bits."""
    T, H = 9, 136
    g = gen(21)
    y, x, c = randn(g, T, H), randn(g, T, H), randn(g, T, H)
    post, gate = params(g, H, "f32", kind), gates(g, T, H, "f32", True, True, 0.7)
    leaves = [y, x, post.weight, post.bias, gate.channel, gate.token]

    def f(y, x, w, b, ch, tok):
        n = Ref(y, kind, w, b, float(np.float32(EPS)))
        return ((x + float(np.float32(0.7)) * ch * tok[:, None] * n.out) * c.double()).sum()
    ws = torch.empty(B.moe_norm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    dy = torch.empty_like(y)
    dw, db, dc, dq = (torch.empty(n, device=DEV) for n in (H, H, H, T))
    B.moe_norm_residual_backward(c, y, post, gate, dy, ws, dw, db, dc, dq)
    h = 1e-5
    for i, grad in enumerate([dy, c, dw, db, dc, dq]):
        d = torch.randn(leaves[i].shape, generator=g, device=DEV, dtype=torch.float64)

        def at(s):
            return f(*[l.double() + s * d if j == i else l.double() for j, l in enumerate(leaves)])
        diff = float((at(h) - at(-h)) / (2 * h))
        got = (grad.double() * d)
        # fp32 gradients: about 60 roundings' worth of the terms; the difference itself
        # h^2 times a third derivative and 1e-16 / h
        assert abs(float(got.sum()) - diff) <= 1e-5 * float(got.abs().sum()) + 1e-7 * float(c.abs().sum())


def test_values_that_are_not_finite_stay_in_their_row():
    T, H = 6, 264
    g = gen(22)
    x, y = randn(g, T, H, dt="bf16"), randn(g, T, H, dt="bf16")
    n, gate = params(g, H, "bf16", B.NORM_RMS), B.Gate(0.5)
    r, o = torch.empty_like(x), torch.empty_like(x)
    B.moe_norm_residual(y, x, n, gate, r, pre=n, n=o)
    y2 = y.clone()
    y2[2, 5], y2[4, 0] = float("nan"), float("inf")
    r2, o2 = torch.empty_like(x), torch.empty_like(x)
    B.moe_norm_residual(y2, x, n, gate, r2, pre=n, n=o2)
    keep = [0, 1, 3, 5]
    assert torch.equal(r[keep], r2[keep]) and torch.equal(o[keep], o2[keep])
    assert torch.isnan(r2[2]).all() and torch.isnan(r2[4, 0])


def test_a_missing_norm_or_gate_is_refused():
    x = torch.zeros(2, 64, device=DEV)
    for f in (lambda: B.moe_norm(x, None, x), lambda: B.moe_norm_backward(x, x, None, x),
              lambda: B.moe_norm_residual(x, x, None, B.Gate(), x),
              lambda: B.moe_norm_residual(x, x, B.Norm(), None, x),
              lambda: B.moe_norm(x, B.Norm(), torch.zeros(2, 64)),
              lambda: B.moe_norm(x, B.Norm(weight=torch.ones(64)), x)):
        with pytest.raises(B.MoEError) as e:
            f()
        assert e.value.status == B.MOE_EINVAL
    assert (x == 0).all()


def test_empty_batches():
    p = B.Plan(0, 2, 4, 16, DEV)
    B.moe_align(torch.empty(0, 2, dtype=torch.int32, device=DEV), 4, p)
    x = torch.empty(0, 64, device=DEV)
    rows = torch.full((8, 64), 7.0, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    B.moe_permute(x, p, rows)
    B.moe_permute_backward(rows, p, x)
    B.moe_unpermute(rows, w, p, x)
    B.moe_unpermute_backward(x, rows, w, p, rows, w)
    B.moe_route_backward(torch.empty(0, 2, dtype=torch.int32, device=DEV), w, w,
                         torch.empty(0, 4, device=DEV))
    assert (rows == 7).all()
    v = torch.ones(64, device=DEV)
    n, gate = B.Norm(B.NORM_RMS, EPS, v, v), B.Gate(1.0, v, torch.empty(0, device=DEV))
    B.moe_norm(x, n, x)
    B.moe_norm_residual(x, x, n, gate, x, pre=n, n=x)
    d = [torch.full((64,), 7.0, device=DEV) for _ in range(5)]
    B.moe_norm_backward(x, x, n, x, dweight=d[0], dbias=d[1],
                        workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    B.moe_norm_residual_backward(x, x, n, gate, x, torch.empty(0, dtype=torch.uint8, device=DEV),
                                 d[2], d[3], d[4])
    for t in d:   # a sum over no tokens
        assert (t == 0).all()


# ------------------------------------------------------------ a run of them all


class Step:
    """One training step of an MoE block on a residual stream x: norm, routing, rows,
    each expert's own product (a torch one), the way back, norm, gate and residual sum;
    then every gradient, from dr."""

    def __init__(self, T, H, E, K, block, dt, seed):
        g = gen(seed)
        self.T, self.H, self.E, self.K = T, H, E, K
        new = lambda *s, dtype=DT[dt]: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
        f32 = torch.float32
        self.x, self.dr = randn(g, T, H, dt=dt, std=2.0), randn(g, T, H, dt=dt)
        self.wr = randn(g, E, H, std=H ** -0.5)
        self.we = randn(g, E, H, H, std=H ** -0.5, dt=dt)
        self.pre, self.post = params(g, H, "f32", B.NORM_RMS, bias=False), params(g, H, "f32", B.NORM_RMS)
        self.gate = gates(g, T, H, "f32", True, True, 0.6)
        self.plan = B.Plan(T, K, E, block, DEV)
        cap = self.plan.cap
        self.n, self.y, self.r, self.dy, self.dn, self.dx = (new(T, H) for _ in range(6))
        self.rows, self.out_rows, self.drows = (torch.zeros(cap, H, dtype=DT[dt], device=DEV) for _ in range(3))
        self.ids, self.w, self.dw = new(T, K, dtype=torch.int32), new(T, K, dtype=f32), new(T, K, dtype=f32)
        self.logits, self.dlogits = new(T, E, dtype=f32), new(T, E, dtype=f32)
        self.grads = [new(H, dtype=f32) for _ in range(4)] + [new(T, dtype=f32)]
        self.ws = new(B.moe_norm_workspace_bytes(T, H), dtype=torch.uint8)

    def products(self, a, w, o):
        """o[rows of e] = a[rows of e] w[e], for every expert's full slot"""
        for e in range(self.E):
            lo, hi = self.bounds[e], self.bounds[e + 1]
            if hi > lo:
                o[lo:hi] = (a[lo:hi].float() @ w[e].float()).to(o.dtype)

    def routing(self):
        B.moe_norm(self.x, self.pre, self.n)
        self.logits.copy_(self.n.float() @ self.wr.t())
        B.moe_route_align(self.logits, self.K, self.ids, self.w, self.plan)

    def run(self):
        B.moe_permute(self.n, self.plan, self.rows)
        self.products(self.rows, self.we, self.out_rows)
        B.moe_unpermute(self.out_rows, self.w, self.plan, self.y)
        B.moe_norm_residual(self.y, self.x, self.post, self.gate, self.r)
        g = self.grads
        B.moe_norm_residual_backward(self.dr, self.y, self.post, self.gate, self.dy, self.ws, g[0],
                                     g[1], g[2], g[4])
        B.moe_unpermute_backward(self.dy, self.out_rows, self.w, self.plan, self.drows, self.dw)
        B.moe_route_backward(self.ids, self.w, self.dw, self.dlogits)
        self.products(self.drows, self.wet, self.rows)
        B.moe_permute_backward(self.rows, self.plan, self.dn)
        self.dn.add_((self.dlogits @ self.wr).to(self.dn.dtype))
        B.moe_norm_backward(self.dn, self.x, self.pre, self.dx, self.ws, dres=self.dr, dweight=g[3])
        return [self.r, self.dx, self.dw, self.dlogits] + g

    def prepare(self):
        self.routing()
        self.bounds = self.plan.expert_offsets.tolist()
        self.wet = self.we.transpose(1, 2).contiguous()

    def reference(self):
        """The same from the definitions, differentiated by torch in 64 bits on the CPU."""
        d = lambda t: t.detach().double().cpu()  # noqa: E731
        x, w0 = d(self.x).requires_grad_(), d(self.pre.weight).requires_grad_()
        w1, b1 = d(self.post.weight).requires_grad_(), d(self.post.bias).requires_grad_()
        ch, tok = d(self.gate.channel).requires_grad_(), d(self.gate.token).requires_grad_()
        ids = self.ids.cpu().long()

        def rms(v):
            return v / torch.sqrt((v * v).mean(1, keepdim=True) + float(np.float32(EPS)))
        n = rms(x) * w0
        logits = n @ d(self.wr).t()
        logits.retain_grad()
        w = torch.softmax(logits.gather(1, ids), 1)
        w.retain_grad()
        we = d(self.we)
        out = torch.stack([torch.stack([n[t] @ we[e] for e in ids[t]]) for t in range(self.T)])
        y = (out * w[:, :, None]).sum(1)
        r = x + float(np.float32(0.6)) * ch * tok[:, None] * (rms(y) * w1 + b1)
        r.backward(d(self.dr))
        return [r.detach(), x.grad, w.grad, logits.grad, w1.grad, b1.grad, ch.grad, w0.grad, tok.grad]


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


def test_training_step_in_fp32():
    s = Step(29, 72, 6, 3, 16, "f32", 31)
    s.prepare()
    # fp32 throughout; the longest chains hold a few hundred roundings, the norm of dy's
    # small rows magnifies the error of y's by under 100: below 1e-4 of each result
    for got, want in zip(s.run(), s.reference()):
        assert rel(got, want) <= 1e-4


def test_training_step_in_bf16():
    s = Step(40, 64, 4, 2, 16, "bf16", 32)
    s.prepare()
    # every tensor between the operators is rounded to 2^-8 of an element; up to ten such
    # roundings follow one another, each at most doubled by the next norm or weight
    for got, want in zip(s.run(), s.reference()):
        assert rel(got, want) <= 10 * 2 * 2.0 ** -8


def test_training_step_captured_in_a_graph():
    """Forward and backward captured once and replayed, with eager passes on other data in
    between and on another stream: every replay as the eager pass."""
    s = Step(33, 136, 4, 2, 16, "bf16", 33)
    s.prepare()
    other = Step(21, 264, 6, 3, 16, "f32", 34)
    other.prepare()
    want = [t.clone() for t in s.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = s.run()
    for _ in range(3):
        for t in outs:
            t.zero_()
        with torch.cuda.stream(side):   # a step of its own buffers beside the replay
            other.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_given_stream_and_its_order():
    """Calls take the stream they are given, in order with the work on it."""
    T, H = 64, 4096
    g = gen(35)
    x, n = randn(g, T, H, dt="bf16"), params(g, H, "bf16", B.NORM_RMS)
    want, out, src = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(x)
    B.moe_norm(x, n, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(8):
            big = big @ big * 1e-2
        src.copy_(x)
    B.moe_norm(src, n, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,shared,stream_dtype", [(1, 128, torch.bfloat16), (48, 0, torch.float32),
                                                   (300, 128, torch.float32)])
def test_block_pass(T, shared, stream_dtype):
    """MoEBlock: two blocks in a row, the first one's next norm feeding the second, against
    the layer's own pass and the operators one by one."""
    shape = LayerShape("block", hidden=256, inter=192, experts=16, topk=4, shared_inter=shared,
                       dtype="bf16", tokens=(T,), routing=("zipf",))
    g = gen(36)
    H = shape.hidden
    x = torch.randn(T, H, generator=g, device=DEV).to(stream_dtype)
    norms = [params(g, H, "bf16", k) for k in (B.NORM_RMS, B.NORM_RMS, B.NORM_LAYER, B.NORM_RMS)]
    gate = gates(g, T, H, "bf16", True, False, 0.5)
    wr = randn(g, shape.experts, H, dt="bf16")
    layers = [MoELayer(shape, synth.layer_inputs(shape, T, seed=s, device=DEV, dense=False)) for s in (1, 2)]

    def router(n, logits):
        logits.copy_(n.float() @ wr.float().t())
    first = MoEBlock(layers[0], norms[0], norms[1], gate, next_norm=norms[2], router=router,
                     stream_dtype=stream_dtype)
    second = MoEBlock(layers[1], norms[2], norms[3], router=router, stream_dtype=stream_dtype)
    first.n = layers[1].inputs["x"]
    r1, n1 = first.forward(x)
    r2, n2 = second.normed(r1)
    assert n2 is None and n1 is layers[1].inputs["x"]

    for layer, pre, post, gt, xin, r, nxt, n in (
            (layers[0], norms[0], norms[1], gate, x, r1, norms[2], n1),
            (layers[1], None, norms[3], B.Gate(), r1, r2, None, None)):
        if pre is not None:
            want = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            B.moe_norm(xin, pre, want)
            assert torch.equal(layer.inputs["x"], want)
        layer.forward()   # the layer's own pass on the tokens and logits the block left
        c = torch.empty(T, H, device=DEV)
        B.moe_combine(layer.y_pairs, layer.topk_w, c, layer.shared_out if layer.has_shared else None)
        check_residual(r, n, reference(c, post), xin, gt, nxt, T)


def test_block_pass_captured_in_a_graph():
    """A block with shared experts (a second stream inside the layer), captured and replayed
    on new tokens, eager passes of another block between the replays."""
    shape = LayerShape("block", hidden=256, inter=192, experts=16, topk=4, shared_inter=128,
                       dtype="bf16", tokens=(20,), routing=("uniform",))
    g = gen(37)
    T, H = 20, shape.hidden

    def block(seed):
        layer = MoELayer(shape, synth.layer_inputs(shape, T, seed=seed, device=DEV, dense=False))
        return MoEBlock(layer, params(g, H, "f32", B.NORM_RMS), params(g, H, "f32", B.NORM_LAYER),
                        gates(g, T, H, "f32", True, True, 0.5), next_norm=params(g, H, "f32", B.NORM_RMS))
    one, other = block(1), block(2)
    xs = [randn(g, T, H, dt="bf16") for _ in range(4)]
    want = [tuple(t.clone() for t in one.forward(x)) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one.forward(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n = one.forward(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        r.zero_()
        n.zero_()
        graph.replay()
        other.forward(xs[0])
        torch.cuda.synchronize()
        assert torch.equal(r, want[i][0]) and torch.equal(n, want[i][1]), i


@pytest.mark.parametrize("kind", [B.NORM_RMS, B.NORM_LAYER, B.NORM_NONE])
@pytest.mark.parametrize("T,H", [(257, 8), (515, 520), (4099, 512), (769, 1032), (1025, 2048),
                                 (300, 3584), (4100, 128), (641, 4096)])
def test_gradients_of_rows_taken_together(T, H, kind):
    """Several rows to a workgroup, and a last turn that has too few: without eps, so that a
    row that is not there would turn up in the sums as a NaN."""
    g = gen(T + H + 31)
    y, dr, dres = (randn(g, T, H, dt="bf16") for _ in range(3))
    w, b, c = (randn(g, H, mean=1.0) for _ in range(3))
    none = kind == B.NORM_NONE
    post = B.Norm(kind, 0.0, None if none else w, None if none else b)
    gate = B.Gate(0.75, c, randn(g, T))
    dy = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((B.moe_norm_workspace_bytes(T, H),), 255, dtype=torch.uint8, device=DEV)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    dw, db = (None, None) if none else (nan(H), nan(H))
    dc, dq = nan(H), nan(T)
    B.moe_norm_residual_backward(dr, y, post, gate, dy, ws, dw, db, dc, dq)
    ref = reference(y, post)
    a, ch = gate_factors(gate, T)
    du = a * ch * dr.double()
    gw = du * ref.w
    close(dy, *ref.backward(gw, 4 * E24 * gw.abs()))
    mag = (ref.xh * ref.w).abs() + ref.b.abs()
    if not none:
        close(dw, *columns(du * ref.xh, du.abs() * (ref.e_xh + 4 * E24 * ref.xh.abs())))
        close(db, *columns(du, 4 * E24 * du.abs()))
    ad = a * dr.double()
    err = (ad.abs() * (ref.e_out + 3 * E24 * mag)).sum(0)
    close(dc, (ad * ref.out).sum(0), err + (tchain(T) + 2) * E24 * (ad.abs() * mag).sum(0))
    v = 0.75 * ch * dr.double()
    close(dq, (v * ref.out).sum(1), (v.abs() * (ref.e_out + (hchain(H) + 4) * E24 * mag)).sum(1))
    if none:
        return
    # the norm before a block: its gradient onto the residual's, without a bias
    pre = B.Norm(kind, 0.0, w)
    dx, dw2 = torch.empty_like(dy), nan(H)
    B.moe_norm_backward(dr, y, pre, dx, ws, dweight=dw2, dres=dres)
    ref = reference(y, pre)
    d = dr.double()
    gw = d * ref.w
    want, err = ref.backward(gw, 4 * E24 * gw.abs())
    close(dx, want + dres.double(), err + E24 * (want.abs() + dres.double().abs()))
    close(dw2, *columns(d * ref.xh, d.abs() * (ref.e_xh + 4 * E24 * ref.xh.abs())))


@pytest.mark.parametrize("kind,pre_kind", [(B.NORM_RMS, B.NORM_RMS), (B.NORM_RMS, B.NORM_LAYER),
                                           (B.NORM_LAYER, B.NORM_RMS)])
@pytest.mark.parametrize("T,H,ydt,xdt,pdt", [
    (4500, 264, "bf16", "bf16", "f32"), (1100, 2048, "bf16", "bf16", "bf16"),
    (700, 3584, "bf16", "f32", "f32"), (530, 4096, "f32", "f32", "bf16"),
    (600, 5000, "bf16", "bf16", "f32"), (2050, 5000, "bf16", "bf16", "bf16")])
def test_gates_and_biases_of_rows_in_turn(T, H, ydt, xdt, pdt, kind, pre_kind):
    """More rows than workgroups, each with its own gate, from pair rows too."""
    g = gen(T + H + 41)
    y, x = stream_rows(g, T, H, ydt, kind), stream_rows(g, T, H, xdt, pre_kind)
    post, pre = params(g, H, pdt, kind), params(g, H, pdt, pre_kind)
    gate = gates(g, T, H, pdt, True, True, 0.6)
    r = torch.full((T, H), float("nan"), dtype=DT[xdt], device=DEV)
    n = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV)
    B.moe_norm_residual(y, x, post, gate, r, pre=pre, n=n)
    check_residual(r, n, reference(y, post), x, gate, pre, T)
    w = torch.rand(T, 2, generator=g, device=DEV)
    pairs = randn(g, 2 * T, H, dt=ydt)
    c = torch.empty(T, H, device=DEV)
    B.moe_combine(pairs, w, c)
    B.moe_combine_norm_residual(pairs, w, x, post, gate, r, pre=pre, n=n)
    check_residual(r, n, reference(c, post), x, gate, pre, T)
    o = torch.full((T, H), float("nan"), dtype=DT[ydt], device=DEV)
    B.moe_norm(x, pre, o)
    ref = reference(x, pre)
    close(o, ref.out, ref.e_out)
