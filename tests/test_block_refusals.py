"""The operators around the experts without a GPU: the C entry points refuse bad
arguments before launching anything, and the binding refuses tensors of the wrong
shape, type, layout or device before calling the library."""
import ctypes
import os

import pytest
import torch

from mixture_experts_layer_30_amd import binding as B

FAKE = 0x10000  # an aligned, never dereferenced address
INV, UNS, CAP = B.MOE_EINVAL, B.MOE_EUNSUPPORTED, B.MOE_ECAPACITY
BF, F32 = B.MOE_BF16, B.MOE_F32
T, H, E, K = 128, 7168, 256, 8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_layer_30_amd import build
        build.build()
    return B.lib()


def plan(cap=4864, block_m=16, ptr=FAKE):
    return ctypes.byref(B.moe_plan(ptr, ptr, ptr, ptr, ptr, block_m, cap))


def call(fn, good, **bad):
    """fn's status with the named arguments of `good` replaced."""
    assert set(bad) <= set(good), bad
    return int(fn(*{**good, **bad}.values(), None))


def expect(fn, good, table):
    for status, bad in table:
        assert call(fn, good, **bad) == status, bad
        assert fn.__name__.encode() in B.lib().moe_last_error(), bad


SORT = [(INV, dict(T=-1)), (UNS, dict(T=1 << 31)), (UNS, dict(T=1 << 24, H=1 << 15)), (UNS, dict(H=100)), (UNS, dict(H=0)), (INV, dict(K=0)),
        (INV, dict(K=257)), (UNS, dict(E=257)), (INV, dict(plan=None)), (INV, dict(plan=plan(ptr=0))),
        (INV, dict(plan=plan(ptr=FAKE + 2))), (INV, dict(plan=plan(cap=4865))),
        (UNS, dict(plan=plan(block_m=0))), (CAP, dict(plan=plan(cap=1024)))]


def test_permute(L):
    good = dict(x=FAKE, dt=BF, T=T, H=H, E=E, K=K, plan=plan(), rows=FAKE)
    for fn in (L.moe_permute, L.moe_permute_backward):
        expect(fn, good, SORT + [(UNS, dict(dt=2)), (INV, dict(x=None)), (INV, dict(rows=None)),
                                 (INV, dict(x=FAKE + 8)), (INV, dict(rows=FAKE + 8))])
        assert call(fn, good, T=0, x=None, rows=None) == B.MOE_OK


def test_unpermute(L):
    good = dict(rows=FAKE, rdt=BF, w=FAKE, shared=FAKE, sdt=F32, T=T, H=H, E=E, K=K, plan=plan(),
                out=FAKE, odt=BF)
    expect(L.moe_unpermute, good, SORT + [
        (UNS, dict(rdt=2)), (UNS, dict(sdt=2)), (UNS, dict(odt=-1)), (INV, dict(rows=None)),
        (INV, dict(out=None)), (INV, dict(w=FAKE + 2)), (INV, dict(shared=FAKE + 4)),
        (INV, dict(out=FAKE + 8))])
    assert call(L.moe_unpermute, good, T=0, rows=None, out=None) == B.MOE_OK


def test_unpermute_backward(L):
    good = dict(dout=FAKE, rows=FAKE, dt=BF, w=FAKE, T=T, H=H, E=E, K=K, plan=plan(), drows=FAKE,
                dw=FAKE)
    expect(L.moe_unpermute_backward, good, SORT + [
        (UNS, dict(dt=2)), (INV, dict(dout=None)), (INV, dict(rows=None)), (INV, dict(w=None)),
        (INV, dict(drows=None, dw=None)), (INV, dict(drows=FAKE + 8)), (INV, dict(dw=FAKE + 2))])
    assert call(L.moe_unpermute_backward, good, T=0, dout=None, rows=None) == B.MOE_OK


def test_route_backward(L):
    good = dict(ids=FAKE, w=FAKE, dw=FAKE, T=T, E=E, K=K, dlogits=FAKE)
    expect(L.moe_route_backward, good, [
        (INV, dict(T=-1)), (INV, dict(K=0)), (INV, dict(K=257)), (UNS, dict(E=257)), (INV, dict(ids=None)),
        (INV, dict(w=None)), (INV, dict(dw=None)), (INV, dict(dlogits=None)),
        (INV, dict(dlogits=FAKE + 2)), (UNS, dict(T=1 << 28))])
    assert call(L.moe_route_backward, good, T=0, ids=None, dlogits=None) == B.MOE_OK


def norm(kind=B.NORM_RMS, eps=1e-6, w=FAKE, b=FAKE):
    return ctypes.byref(B.moe_norm_params(kind, eps, w, b))


def gate(alpha=1.0, channel=FAKE, token=FAKE):
    return ctypes.byref(B.moe_gate_params(alpha, channel, token))


ROWS = [(INV, dict(T=-1)), (UNS, dict(T=1 << 31)), (UNS, dict(H=100)), (UNS, dict(H=16392)),
        (UNS, dict(H=0)), (UNS, dict(pdt=2)), (UNS, dict(xdt=2))]


def norm_refusals(key, none_ok):
    kinds = (3, -1) if none_ok else (0, 3, -1)
    table = [(INV, {key: None})] + [(INV, {key: norm(kind=k, w=None, b=None)}) for k in kinds]
    table += [(INV, {key: norm(eps=e)}) for e in (-1e-6, float("nan"), float("inf"))]
    table += [(INV, {key: norm(w=FAKE + 8)}), (INV, {key: norm(b=FAKE + 2)})]
    if none_ok:
        table += [(INV, {key: norm(kind=0, b=None)}), (INV, {key: norm(kind=0, w=None)})]
    return table


GATES = [(INV, dict(gate=None)), (INV, dict(gate=gate(alpha=float("nan")))),
         (INV, dict(gate=gate(alpha=float("-inf")))), (INV, dict(gate=gate(channel=FAKE + 8))),
         (INV, dict(gate=gate(token=FAKE + 2)))]


def test_norm(L):
    good = dict(x=FAKE, xdt=BF, T=T, H=H, norm=norm(), pdt=BF, n=FAKE, odt=BF)
    expect(L.moe_norm, good, ROWS + norm_refusals("norm", False) + [
        (UNS, dict(odt=2)), (INV, dict(x=None)), (INV, dict(n=None)), (INV, dict(n=FAKE + 8))])
    assert call(L.moe_norm, good, T=0, x=None, n=None) == B.MOE_OK


def test_norm_backward(L):
    ws = B.moe_norm_workspace_bytes(T, H)
    good = dict(dn=FAKE, odt=BF, x=FAKE, xdt=BF, dres=FAKE, T=T, H=H, norm=norm(), pdt=BF, dx=FAKE,
                dw=FAKE, db=FAKE, ws=FAKE, n=ws)
    expect(L.moe_norm_backward, good, ROWS + norm_refusals("norm", False) + [
        (UNS, dict(odt=2)), (CAP, dict(n=ws - 1)), (INV, dict(ws=None)), (INV, dict(dn=None)),
        (INV, dict(x=None)), (INV, dict(dx=None)), (INV, dict(dres=FAKE + 8)), (INV, dict(dw=FAKE + 4)),
        (INV, dict(db=FAKE + 8))])
    # no parameter gradient, no tokens: nothing to do
    assert call(L.moe_norm_backward, good, T=0, dw=None, db=None, ws=None, n=0, dx=None) == B.MOE_OK


def test_norm_residual(L):
    good = dict(y=FAKE, ydt=BF, x=FAKE, xdt=F32, T=T, H=H, post=norm(), gate=gate(), pdt=BF, r=FAKE,
                pre=norm(B.NORM_LAYER), n=FAKE)
    both = ROWS + norm_refusals("post", True) + GATES + [
        (UNS, dict(ydt=2)), (INV, dict(x=None)), (INV, dict(r=None)), (INV, dict(n=None)),
        (INV, dict(pre=None)), (INV, dict(r=FAKE + 8)), (INV, dict(n=FAKE + 8)),
        (INV, dict(pre=norm(kind=0, w=None, b=None)))]
    expect(L.moe_norm_residual, good, both + [(INV, dict(y=None))])
    assert call(L.moe_norm_residual, good, T=0, y=None, x=None, r=None) == B.MOE_OK
    good = dict(y=FAKE, ydt=BF, w=FAKE, shared=FAKE, sdt=F32, x=FAKE, xdt=F32, T=T, K=K, H=H,
                post=norm(), gate=gate(), pdt=BF, r=FAKE, pre=norm(), n=FAKE)
    expect(L.moe_combine_norm_residual, good, both + [
        (INV, dict(y=None)), (UNS, dict(sdt=2)), (INV, dict(K=0)), (INV, dict(w=None)),
        (INV, dict(shared=FAKE + 8)), (UNS, dict(T=1 << 28))])
    assert call(L.moe_combine_norm_residual, good, T=0, y=None, r=None) == B.MOE_OK


def test_norm_residual_backward(L):
    ws = B.moe_norm_workspace_bytes(T, H)
    good = dict(dr=FAKE, xdt=BF, y=FAKE, ydt=BF, T=T, H=H, post=norm(), gate=gate(), pdt=BF, dy=FAKE,
                dw=FAKE, db=FAKE, dc=FAKE, dq=FAKE, ws=FAKE, n=ws)
    none = norm(kind=0, w=None, b=None)
    expect(L.moe_norm_residual_backward, good, ROWS + norm_refusals("post", True) + GATES + [
        (UNS, dict(ydt=2)), (CAP, dict(n=ws - 1)), (INV, dict(ws=None)), (INV, dict(dr=None)),
        (INV, dict(y=None)), (INV, dict(dy=None)), (INV, dict(dc=FAKE + 8)), (INV, dict(dq=FAKE + 2)),
        (INV, dict(post=none)), (INV, dict(post=none, dw=None)),
        (INV, dict(gate=gate(channel=None))), (INV, dict(gate=gate(token=None)))])
    assert call(L.moe_norm_residual_backward, good, T=0, dw=None, db=None, dc=None, ws=None, n=0,
                dy=None) == B.MOE_OK


def test_workspace_bytes(L):
    assert B.moe_norm_workspace_bytes(0, 64) == 0
    assert B.moe_norm_workspace_bytes(1, 64) == 2 * 64 * 4   # two fp32 sums a column
    for t, h in ((-1, 64), (1 << 31, 64), (4, 0), (4, 12), (4, 16392)):
        assert B.moe_norm_workspace_bytes(t, h) == -1
    for h in (8, 512, 7168, 16384):   # enough for more tokens is enough for fewer
        sizes = [B.moe_norm_workspace_bytes(t, h) for t in range(0, 20000, 7)]
        assert sizes == sorted(sizes)


# ------------------------------------------------------------------ the binding


def refused(status, fn, *a, **k):
    with pytest.raises(B.MoEError) as e:
        fn(*a, **k)
    assert e.value.status == status, e.value


def test_binding_refuses_rows():
    p = B.Plan(4, 2, 4, 16, "cpu")
    x, rows, w = torch.zeros(4, 64), torch.zeros(p.cap, 64), torch.zeros(4, 2)
    refused(INV, B.moe_permute, x, p, rows)                                  # not on a GPU
    refused(INV, B.moe_permute, x[:3], p, rows)                              # tokens
    refused(INV, B.moe_permute, torch.zeros(64, 4).t(), p, rows)             # layout
    refused(INV, B.moe_permute, x, p, rows[:-1])                             # too few rows
    refused(INV, B.moe_permute, x, p, torch.zeros(p.cap, 72))
    refused(UNS, B.moe_permute, x, p, rows.bfloat16())
    refused(INV, B.moe_permute_backward, rows[:-1], p, x)
    refused(UNS, B.moe_permute_backward, rows, p, x.bfloat16())
    refused(INV, B.moe_unpermute, rows, w[:, :1], p, x)
    refused(UNS, B.moe_unpermute, rows, w.double(), p, x)
    refused(INV, B.moe_unpermute, rows, w.t().contiguous().t(), p, x)
    refused(INV, B.moe_unpermute, rows, w, p, x, shared=x[:2])
    refused(INV, B.moe_unpermute, rows, w, p, x)
    refused(INV, B.moe_unpermute_backward, x, rows, w, p, rows[:-1], w)
    refused(UNS, B.moe_unpermute_backward, x, rows, w, p, rows, w.double())
    refused(UNS, B.moe_unpermute_backward, x, rows.bfloat16(), w, p, rows, w)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    refused(UNS, B.moe_route_backward, ids.long(), w, w, x)
    refused(INV, B.moe_route_backward, ids, w, w[:3], x)
    refused(INV, B.moe_route_backward, ids, w, w, x[:2])
    refused(INV, B.moe_route_backward, ids, w, w, x)


def test_binding_refuses_norms():
    x, v = torch.zeros(4, 64), torch.zeros(64)
    n, g = B.Norm(B.NORM_RMS, 1e-6, v), B.Gate(1.0, v)
    refused(INV, B.moe_norm, x, n, x)                                        # not on a GPU
    refused(INV, B.moe_norm, x, n, x[:2])
    refused(INV, B.moe_norm, x[0], n, x[0])
    refused(INV, B.moe_norm, x, B.Norm(B.NORM_RMS, 1e-6, v[:8]), x)
    refused(UNS, B.moe_norm, x, B.Norm(B.NORM_RMS, 1e-6, v, v.bfloat16()), x)
    refused(UNS, B.moe_norm, x, B.Norm(B.NORM_RMS, 1e-6, v.half()), x)
    refused(UNS, B.moe_norm_backward, x, x, n, x.bfloat16())
    refused(UNS, B.moe_norm_backward, x, x, n, x, dres=x.bfloat16())
    refused(INV, B.moe_norm_backward, x, x, n, x, dweight=v[:8])
    refused(UNS, B.moe_norm_backward, x, x, n, x, dweight=v.bfloat16())
    refused(UNS, B.moe_norm_residual, x, x, n, g, x.bfloat16())
    refused(UNS, B.moe_norm_residual, x, x, n, g, x, pre=n, n=x.bfloat16())
    refused(UNS, B.moe_norm_residual, x, x, n, B.Gate(1.0, v.bfloat16()), x)
    refused(INV, B.moe_norm_residual, x, x, n, B.Gate(1.0, None, v[:3]), x)
    refused(UNS, B.moe_norm_residual, x, x, n, B.Gate(1.0, None, v[:4].double()), x)
    refused(INV, B.moe_norm_residual, x[:3], x, n, g, x)
    refused(INV, B.moe_combine_norm_residual, x, torch.zeros(4, 2), x, n, g, x)
    refused(INV, B.moe_combine_norm_residual, torch.zeros(8, 64), torch.zeros(3, 2), x, n, g, x)
    refused(INV, B.moe_norm_residual_backward, x, x[:3], n, g, x[:3])
    refused(UNS, B.moe_norm_residual_backward, x, x, n, g, x.bfloat16())
    refused(INV, B.moe_norm_residual_backward, x, x, n, g, x, dtoken=v)
    refused(INV, B.moe_norm_residual_backward, x, x, n, g, x)
