"""Training the experts where sums are cut into parts, buffers end and offsets pass 2 GB: subsets of
the gradients, padding of every width, an expert in both slots of a token, what lies around each
buffer, and operands close to 4 GB."""
import pytest
import torch

import test_gpu_train_ops as O
import train_reference as R
from mixture_experts_layer_30_amd import binding as B
from test_gpu_train_ops import (BF, DEV, HALF_STEP, check_kept, expert_rows, gen, given, held,
                                new_saved, randn, routed, space, weights, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


SUBSETS = [("dx", "dw13", "dw2"), ("dx",), ("dw13",), ("dw2",), ("dx", "dw2"), ("dx", "dw13"),
           ("dw13", "dw2")]


def each_subset(run, buffers, refs):
    """Whichever gradients are asked for, each is within its bound, element by element, and the same
    on a second run.  (Not the same as in another subset: sums may be taken in other parts.)"""
    for want in SUBSETS:
        first, again = (run({k: v for k, v in buffers().items() if k in want}) for _ in range(2))
        for k in want:
            for at, ref, err in refs[k]:
                within(first[k][at], ref, err, (want, k))
            assert torch.equal(first[k], again[k]), (want, k)


# dx in parts, fewer of them next to the weights' tiles; parts of few blocks; the weights'
# gradients in parts
@pytest.mark.parametrize("T,H,I", [(1003, 1088, 1856), (200, 1024, 512), (512, 2048, 2048),
                                   (232, 1472, 3584), (2100, 128, 192), (2100, 192, 1088)])
def test_dense_subsets_in_parts(T, H, I):
    g = gen(T)
    x, dout = randn(g, T, H), randn(g, T, H, std=0.1)
    w13, w2 = (w[0] for w in weights(g, 1, H, I))
    saved, h = given(T, I, B.SAVE_BF16, g)
    n = B.moe_ffn_backward_workspace_bytes(T, H, I)

    def run(out):
        B.dense_ffn_backward(dout, x, w13, w2, saved, space(n), **out)
        return out

    a = (dout.double(), x.double(), w13.double(), w2.double(), h)
    refs = {k: [(slice(None), ref, err)] for k, ref, err in
            zip(("dx", "dw13", "dw2"), R.backward(*a)[2:], R.backward_bounds(*a, HALF_STEP[BF]))}
    each_subset(run, lambda: dict(dx=torch.zeros_like(x), dw13=torch.zeros_like(w13),
                                  dw2=torch.zeros_like(w2)), refs)


@pytest.mark.parametrize("T,H,I,E,K", [(1500, 320, 1088, 2, 2), (1100, 256, 128, 4, 1),
                                       (256, 1024, 1024, 4, 2), (40, 1024, 1024, 3, 2)])
def test_grouped_subsets_in_parts(T, H, I, E, K):
    _, _, plan = routed(T, E, K, 16, B.PAD_BLOCK, T)
    g = gen(T + 1)
    x, drows = randn(g, T, H), randn(g, plan.cap, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    saved, h = given(plan.cap, I, B.SAVE_FP8, g)
    n = B.moe_ffn_backward_workspace_bytes(plan.cap, H, I)

    def run(out):
        names = {"dxrows" if k == "dx" else k: v for k, v in out.items()}
        B.moe_grouped_ffn_backward(drows, x, w13, w2, plan, saved, space(n), **names)
        return out

    refs = {"dx": [], "dw13": [], "dw2": []}
    for e in range(E):
        at, tok = expert_rows(plan, e)
        if len(tok) == 0:
            continue
        a = (drows[at].double(), x[tok].double(), w13[e].double(), w2[e].double(), h[at])
        for k, where, ref, err in zip(refs, (at, e, e), R.backward(*a)[2:],
                                      R.backward_bounds(*a, HALF_STEP[BF])):
            refs[k].append((where, ref, err))
    each_subset(run, lambda: dict(dx=torch.zeros_like(drows), dw13=torch.zeros_like(w13),
                                  dw2=torch.zeros_like(w2)), refs)


@pytest.mark.parametrize("dwdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [B.SAVE_BF16, B.SAVE_FP8])
@pytest.mark.parametrize("T,H,I,E,K", [(2, 1024, 2048, 4, 2), (1, 4096, 1024, 8, 2),
                                       (9, 1088, 1856, 3, 3), (200, 1024, 512, 2, 1)])
def test_padding_changes_no_value(T, H, I, E, K, fmt, dwdt):
    """Few rows of wide experts, whose contraction is cut into parts, are the same bits however
    far apart the alignment lays them, and within their bounds."""
    g = gen(12)
    x, dpairs = randn(g, T, H), randn(g, T * K, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    seen = []
    for block, pad in ((1, B.PAD_BLOCK), (16, B.PAD_BLOCK), (128, B.PAD_MAX), (1024, B.PAD_MAX)):
        _, _, plan = routed(T, E, K, block, pad, 12)
        at = plan.inv_pos[:T * K].long()
        drows = torch.full((plan.cap, H), float("nan"), dtype=BF, device=DEV)
        drows[at] = dpairs
        saved = new_saved(plan.cap, I, fmt)
        rows, dxrows = torch.zeros_like(drows), torch.zeros_like(drows)
        dw13, dw2 = (torch.full(w.shape, 9.0, dtype=dwdt, device=DEV) for w in (w13, w2))
        B.moe_grouped_ffn_train(x, w13, w2, plan, saved,
                                space(B.moe_ffn_train_workspace_bytes(plan.cap, H, I)), rows)
        B.moe_grouped_ffn_backward(drows, x, w13, w2, plan, saved,
                                   space(B.moe_ffn_backward_workspace_bytes(plan.cap, H, I)),
                                   dxrows=dxrows, dw13=dw13, dw2=dw2)
        kept = [saved.h[at].view(torch.uint8)] + ([saved.scales[at]] if fmt == B.SAVE_FP8 else [])
        seen.append([rows[at], dxrows[at], dw13, dw2] + kept)
        free = ~held(plan, T)
        assert not rows[free].any() and not dxrows[free].any()
        if block > 1:
            continue
        for e in range(E):
            here, tok = expert_rows(plan, e)
            if len(tok) == 0:
                assert not dw13[e].any() and not dw2[e].any()
                continue
            a = x[tok].double(), w13[e].double(), w2[e].double()
            err_h, err_y = R.forward_bounds(*a)
            h, _, y = R.forward(*a)
            h = check_kept(saved, here, h, err_h)
            within(rows[here], y, err_y, ("rows", e))
            a = (drows[here].double(),) + a + (h,)
            for got, ref, err in zip((dxrows[here], dw13[e], dw2[e]), R.backward(*a)[2:],
                                     R.backward_bounds(*a, HALF_STEP[dwdt])):
                within(got, ref, err, ("gradients", e))
    for other in seen[1:]:
        for a, b in zip(seen[0], other):
            assert torch.equal(a, b)


def step(b, x, drows, w13, w2, plan, stream=None):
    B.moe_grouped_ffn_train(x, w13, w2, plan, b["saved"], b["ws"], b["rows"], stream=stream)
    B.moe_grouped_ffn_backward(drows, x, w13, w2, plan, b["saved"], b["ws"], dxrows=b["dxrows"],
                               dw13=b["dw13"], dw2=b["dw2"], stream=stream)


def test_padded_parts_on_another_stream_and_in_a_graph():
    T, H, I, E, K = 9, 1088, 1856, 3, 2
    _, _, plan = routed(T, E, K, 1024, B.PAD_MAX, 5, budget=True)
    g = gen(5)
    x, drows = randn(g, T, H), randn(g, plan.cap, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    names = ("rows", "dxrows", "dw13", "dw2")

    def buffers():
        return dict(saved=new_saved(plan.cap, I, B.SAVE_FP8),
                    ws=space(B.moe_ffn_backward_workspace_bytes(plan.cap, H, I)),
                    rows=torch.zeros_like(drows), dxrows=torch.zeros_like(drows),
                    dw13=torch.zeros_like(w13), dw2=torch.zeros_like(w2))

    first, other, graphed = buffers(), buffers(), buffers()
    step(first, x, drows, w13, w2, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(other, x, drows, w13, w2, plan, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed, x, drows, w13, w2, plan)
    for _ in range(3):
        for k in names:
            graphed[k].zero_()
        graph.replay()
        step(other, x, drows, w13, w2, plan)   # eager work between the replays
        torch.cuda.synchronize()
        for k in names:
            assert torch.equal(first[k], other[k]) and torch.equal(first[k], graphed[k]), k


@pytest.mark.parametrize("T,block", [(300, 1), (5, 1024)])
def test_the_same_expert_twice(T, block):
    """An expert with more rows than there are tokens, as both slots of every token are its own."""
    H, I, E, K = 320, 1088, 3, 2
    plan = B.Plan(T, K, E, block, DEV)
    B.moe_align(torch.ones(T, K, dtype=torch.int32, device=DEV), E, plan)
    g = gen(T)
    x, drows = randn(g, T, H), randn(g, plan.cap, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    b = dict(saved=new_saved(plan.cap, I, B.SAVE_BF16),
             ws=space(B.moe_ffn_backward_workspace_bytes(plan.cap, H, I)),
             rows=torch.zeros_like(drows), dxrows=torch.zeros_like(drows),
             dw13=torch.ones_like(w13), dw2=torch.ones_like(w2))
    step(b, x, drows, w13, w2, plan)
    at, tok = expert_rows(plan, 1)
    assert len(tok) == 2 * T
    a = x[tok].double(), w13[1].double(), w2[1].double()
    h, _, y = R.forward(*a)
    err_h, err_y = R.forward_bounds(*a)
    within(b["rows"][at], y, err_y, "rows")
    a = (drows[at].double(),) + a + (check_kept(b["saved"], at, h, err_h),)
    for got, ref, err in zip((b["dxrows"][at], b["dw13"][1], b["dw2"][1]), R.backward(*a)[2:],
                             R.backward_bounds(*a, HALF_STEP[BF])):
        within(got, ref, err, "gradients")
    for e in (0, 2):
        assert not b["dw13"][e].any() and not b["dw2"][e].any()


# ------------------------------------------------------------------ what lies around the buffers

EDGE = 4096   # bytes of a pattern before and after each buffer


class Guarded:
    """Buffers of exactly their size, each between two runs of a pattern."""

    def __init__(self):
        self.all = []

    def new(self, shape, dt, fill):
        n = torch.empty(shape, dtype=dt, device="meta").numel() * dt.itemsize
        raw = torch.full((n + 2 * EDGE,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append(raw)
        t = raw[EDGE:EDGE + n].view(dt).view(shape)
        t.fill_(fill)
        return t

    def check(self, what):
        for k, raw in enumerate(self.all):
            for edge in (raw[:EDGE], raw[raw.numel() - EDGE:]):
                assert bool((edge == 0xA5).all()), (what, k)

    def saved(self, rows, I, fmt):
        s = B.Saved(rows, I, fmt, DEV)
        if fmt == B.SAVE_FP8:
            s.h = self.new(s.h.shape, torch.uint8, 127)
            s.scales = self.new(s.scales.shape, torch.uint8, 200)
        else:
            s.h = self.new(s.h.shape, BF, float("nan"))
        return s


@pytest.mark.parametrize("dwdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,I,E,K,block,pad,budget,one,fmt", O.CASES + [
    # parts whose sums are kept by pair
    (2, 1024, 2048, 4, 2, 1024, B.PAD_MAX, False, False, B.SAVE_FP8),
    (9, 1088, 1856, 3, 3, 1024, B.PAD_MAX, True, False, B.SAVE_BF16),
    (200, 1024, 512, 2, 1, 1024, B.PAD_MAX, False, True, B.SAVE_FP8)])
def test_nothing_outside_is_written(T, H, I, E, K, block, pad, budget, one, fmt, dwdt):
    """Neither around the buffers, the workspace among them, nor in rows that hold no pair."""
    _, _, plan = routed(T, E, K, block, pad, T + H, budget, one)
    g, m = gen(T + I), Guarded()
    x, drows = randn(g, T, H), randn(g, plan.cap, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    saved = m.saved(plan.cap, I, fmt)
    rows, dxrows = (m.new((plan.cap, H), BF, -7.0) for _ in range(2))
    dw13, dw2 = m.new((E, 2 * I, H), dwdt, 5.0), m.new((E, H, I), dwdt, 5.0)
    fws = m.new((B.moe_ffn_train_workspace_bytes(plan.cap, H, I),), torch.uint8, 255)
    bws = m.new((B.moe_ffn_backward_workspace_bytes(plan.cap, H, I),), torch.uint8, 255)
    free = ~held(plan, T)
    before = saved.h[free].view(torch.uint8).clone()
    B.moe_grouped_ffn_train(x, w13, w2, plan, saved, fws, rows)
    m.check("forward")
    kept = saved.h.view(torch.uint8).clone(), saved.scales.clone() if fmt == B.SAVE_FP8 else None
    assert torch.equal(saved.h[free].view(torch.uint8), before)
    if fmt == B.SAVE_FP8:
        assert bool((saved.scales[free] == 200).all())
        assert bool((saved.scales[~free] < 200).all())   # of values far below 2^73
    assert bool((rows[free] == -7).all())
    B.moe_grouped_ffn_backward(drows, x, w13, w2, plan, saved, bws, dxrows=dxrows, dw13=dw13, dw2=dw2)
    m.check("backward")
    assert bool((dxrows[free] == -7).all())
    assert torch.equal(saved.h.view(torch.uint8), kept[0])
    if fmt == B.SAVE_FP8:
        assert torch.equal(saved.scales, kept[1])


@pytest.mark.parametrize("T,H,I,fmt", O.DENSE + [(1003, 1088, 1856, B.SAVE_FP8),
                                                (200, 1024, 512, B.SAVE_BF16)])
def test_nothing_outside_is_written_dense(T, H, I, fmt):
    g, m = gen(T + I), Guarded()
    x, dout = randn(g, T, H), randn(g, T, H, std=0.1)
    w13, w2 = (w[0] for w in weights(g, 1, H, I))
    saved = m.saved(T, I, fmt)
    out, dx = (m.new((T, H), BF, -7.0) for _ in range(2))
    dw13, dw2 = m.new((2 * I, H), BF, 5.0), m.new((H, I), BF, 5.0)
    fws = m.new((B.moe_ffn_train_workspace_bytes(T, H, I),), torch.uint8, 255)
    bws = m.new((B.moe_ffn_backward_workspace_bytes(T, H, I),), torch.uint8, 255)
    B.dense_ffn_train(x, w13, w2, saved, fws, out)
    m.check("forward")
    B.dense_ffn_backward(dout, x, w13, w2, saved, bws, dx=dx, dw13=dw13, dw2=dw2)
    m.check("backward")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 32), (7, 96), (129, 1056)])
def test_nothing_outside_is_packed(T, H, dt):
    m = Guarded()
    x = randn(gen(T), T, H, dt=dt)
    codes, scales = m.new((T, H), torch.uint8, 1), m.new((T, H // 32), torch.uint8, 1)
    B.moe_pack_fp8(x, codes, scales)
    m.check("pack")
    y = m.new((T, H), dt, 1.0)
    B.moe_unpack_fp8(codes, scales, y)
    m.check("unpack")


# ------------------------------------------------------------------ operands close to 4 GB


def test_tokens_close_to_4_gb():
    """Every expert's rows of an x of 4.29 GB: gathered from offsets on both sides of 2^31, row
    buffers past 2^32 bytes."""
    T, H, I, E, K = (1 << 18) - 1, 8192, 64, 4, 1
    assert T * H * 2 < 1 << 32 <= (T + 1) * H * 2
    _, _, plan = routed(T, E, K, 128, B.PAD_BLOCK, 9)
    g = gen(9)
    x, drows = randn(g, T, H), randn(g, plan.cap, H, std=0.1)
    w13, w2 = weights(g, E, H, I)
    saved = new_saved(plan.cap, I, B.SAVE_BF16)
    rows, dxrows = torch.empty_like(drows), torch.empty_like(drows)
    dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
    ws = space(B.moe_ffn_backward_workspace_bytes(plan.cap, H, I))
    B.moe_grouped_ffn_train(x, w13, w2, plan, saved, ws, rows)
    B.moe_grouped_ffn_backward(drows, x, w13, w2, plan, saved, ws, dxrows=dxrows, dw13=dw13, dw2=dw2)
    seen = 0
    for e in range(E):
        at, tok = expert_rows(plan, e)
        if len(tok) == 0:
            assert not dw13[e].any() and not dw2[e].any()
            continue
        w = w13[e].double(), w2[e].double()
        # rows of their own, some thousand at a time; the weights' sums over all of them
        s13, s2, e13, e2 = 0, 0, 0, 0
        for part in torch.arange(len(tok), device=DEV).split(16384):
            r, n = at.start + part, len(part)
            xe, dy = x[tok[part]].double(), drows[r].double()
            h, _, y = R.forward(xe, *w)
            err_h, err_y = R.forward_bounds(xe, *w)
            kept = check_kept(saved, r, h, err_h)
            within(rows[r], y, err_y, ("rows", e))
            _, _, rx, r13, r2 = R.backward(dy, xe, *w, kept)
            ex, b13, b2 = R.backward_bounds(dy, xe, *w, kept, 0.0)
            within(dxrows[r], rx, ex, ("dxrows", e))
            # the bounds count n + 1 roundings of a part's n terms; a sum over all has len(tok) + 1
            more = (len(tok) - n) * R.E24
            dh, a, *_ = R.backward(dy, xe, *w, kept)
            s13, s2 = s13 + r13, s2 + r2
            e13 = e13 + b13 + 1.01 * more * (dh.abs().T @ xe.abs())
            e2 = e2 + b2 + 1.01 * more * (dy.abs().T @ a.abs())
            seen += n
        within(dw13[e], s13, e13 + HALF_STEP[BF] * (s13.abs() + e13), ("dw13", e))
        within(dw2[e], s2, e2 + HALF_STEP[BF] * (s2.abs() + e2), ("dw2", e))
    assert seen == T


def test_weights_close_to_4_gb():
    """Gate and up weights of 4.28 GB: tiles on both sides of offset 2^31 and at their end."""
    T, H, I = 70, 16384, 65344
    assert 4 * I * H < 1 << 32 <= 4 * (I + 256) * H
    g = gen(10)
    x, dout = randn(g, T, H), randn(g, T, H, std=0.1)
    w13 = torch.empty(2 * I, H, dtype=BF, device=DEV)
    for part in w13.split(8192):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * H ** -0.5)
    w2 = randn(g, H, I, std=I ** -0.5)
    saved = new_saved(T, I, B.SAVE_BF16)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
    ws = space(B.moe_ffn_backward_workspace_bytes(T, H, I))
    B.dense_ffn_train(x, w13, w2, saved, ws, out)
    B.dense_ffn_backward(dout, x, w13, w2, saved, ws, dx=dx, dw13=dw13, dw2=dw2)
    # by runs of gate, up and down columns: h, dw13 and dw2 of their own, y and dx summed
    xd, dy = x.double(), dout.double()
    y = err_y = rx = ex = 0

    def before_rounding(err, v):   # err = e + 2^-8 (|v| + e)
        return (err - HALF_STEP[BF] * v.abs()) / (1 + HALF_STEP[BF])

    for c in torch.arange(I, device=DEV).split(4096):
        rows = torch.cat([c, I + c])
        w = w13[rows].double(), w2[:, c].double()
        h, a, part = R.forward(xd, *w)
        err_h, err = R.forward_bounds(xd, *w)
        got = saved.h[:, rows].double()
        within(got, h, err_h + HALF_STEP[BF] * (h.abs() + err_h), "saved")
        # a run's bound counts the roundings of a sum of its own columns: the whole sum has those
        # of the other columns as well (a and dh themselves are off by less than 1% more)
        more = 1.01 * (I - len(c)) * R.E24
        y = y + part
        err_y = err_y + before_rounding(err, part) + more * (a.abs() @ w[1].abs().T)
        dh, _, part, r13, r2 = R.backward(dy, xd, *w, got)
        err, e13, e2 = R.backward_bounds(dy, xd, *w, got, HALF_STEP[BF])
        rx = rx + part
        ex = ex + before_rounding(err, part) + 2 * more * (dh.abs() @ w[0].abs())
        within(dw13[rows], r13, e13, "dw13")
        within(dw2[:, c], r2, e2, "dw2")
    within(out, y, err_y + HALF_STEP[BF] * (y.abs() + err_y), "out")
    within(dx, rx, ex + HALF_STEP[BF] * (rx.abs() + ex), "dx")
