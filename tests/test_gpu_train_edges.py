"""Training the experts where buffers end, sums are cut into parts and offsets pass 2 GB: what
the order of the sums depends on, what lies behind each buffer, and operands close to 4 GB."""
import pytest
import torch

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
