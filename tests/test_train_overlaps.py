"""Training the experts without a GPU: buffers that overlap where a value would be lost are refused
before anything is launched, buffers side by side are not."""
import ctypes

import pytest

from mixture_experts_layer_30_amd import binding as B
from test_train_refusals import L  # noqa: F401  (the library, built where it is not there)

T, H, I, E, K, CAP = 128, 256, 192, 8, 2, 384
BF, F32 = B.MOE_BF16, B.MOE_F32


class Space:
    """Addresses of buffers side by side, never dereferenced: every call here is refused."""

    def __init__(self, **sizes):
        self.at, self.size, p = {}, sizes, 1 << 20
        for k, n in sizes.items():
            self.at[k] = p
            p += (n + 15) // 16 * 16

    def last(self, k):
        """16-byte aligned, in the buffer's last bytes"""
        return self.at[k] + (self.size[k] - 1) // 16 * 16


def sizes(rows, matrices, dwdt, fp8):
    n = B.lib().moe_ffn_backward_workspace_bytes(rows, H, I)
    e = 2 if dwdt == BF else 4
    return dict(dx=rows * H * 2, dy=rows * H * 2, x=T * H * 2, w13=matrices * 4 * I * H,
                w2=matrices * 2 * I * H, h=rows * 2 * I * (1 if fp8 else 2), scales=rows * 2 * I // 32,
                dw13=matrices * 2 * I * H * e, dw2=matrices * I * H * e, workspace=n)


def backward(grouped, s, dwdt, fp8, **other):
    a = {**s.at, **other}
    saved = ctypes.byref(B.moe_saved(int(fp8), a["h"], a["scales"] if fp8 else None))
    n = s.size["workspace"]
    if grouped:
        ptr = 1 << 16
        plan = ctypes.byref(B.moe_plan(ptr, ptr, ptr, ptr, ptr, 16, CAP))
        return B.lib().moe_grouped_ffn_backward(
            a["dy"], a["x"], T, H, I, E, K, a["w13"], a["w2"], plan, saved, a["workspace"], n,
            a["dx"], a["dw13"], a["dw2"], dwdt, None)
    return B.lib().dense_ffn_backward(a["dy"], a["x"], T, H, I, a["w13"], a["w2"], saved,
                                      a["workspace"], n, a["dx"], a["dw13"], a["dw2"], dwdt, None)


# what is written, and what it may not overlap
LOST = [(w, o) for w in ("dx", "dw13", "dw2") for o in ("dy", "x", "w13")]
LOST += [("dw13", "dw2"), ("dx", "dw13"), ("dx", "dw2")]
LOST += [("workspace", o) for o in ("dx", "dw13", "dw2", "dy", "x", "w13", "w2", "h")]


@pytest.mark.parametrize("grouped", [True, False])
@pytest.mark.parametrize("dwdt", [BF, F32])
@pytest.mark.parametrize("fp8", [True, False])
def test_backward(L, grouped, dwdt, fp8):  # noqa: F811
    s = Space(**sizes(CAP if grouped else T, E if grouped else 1, dwdt, fp8))
    for a, b in LOST + ([("workspace", "scales")] if fp8 else []):
        for w, o in ((a, b), (b, a)):
            # the same address, and the other's last bytes
            for at in (s.at[o], s.last(o)):
                # everything else out of the way
                far = Space(**{"_": 1 << 40, **s.size})
                far.at[o] = s.at[o]
                assert backward(grouped, far, dwdt, fp8, **{w: at}) == B.MOE_EINVAL, (w, o)
                err = B.lib().moe_last_error()
                assert b"over" in err, (w, o, err)


def test_what_is_not_read_may_be_overwritten(L):  # noqa: F811
    """x where dw13 is not asked for, w13 where dx is not: here the workspace
    at w2, which is looked at last, is what is refused."""
    s = Space(**sizes(T, 1, BF, False))

    def said(**other):
        assert backward(False, s, BF, False, **other) == B.MOE_EINVAL
        return B.lib().moe_last_error()

    last = dict(w2=s.at["workspace"])   # the last of the checks
    assert b"workspace overwrites w2" in said(**last)
    assert b"workspace overwrites w2" in said(dw2=s.at["x"], dw13=None, dx=None, **last)
    assert b"workspace overwrites w2" in said(dw13=s.at["w13"], dx=None, dw2=None, **last)
    assert b"workspace overwrites w2" in said(w13=None, dx=None, **last)
    # without tokens nothing is read and the workspace is not used
    plan = ctypes.byref(B.moe_plan(1 << 16, 1 << 16, 1 << 16, 1 << 16, 1 << 16, 16, CAP))
    saved = ctypes.byref(B.moe_saved(0, None, None))
    assert B.lib().moe_grouped_ffn_backward(
        s.at["dx"], s.at["dx"], 0, H, I, E, K, s.at["dx"], s.at["dx"], plan, saved, s.at["dx"],
        B.lib().moe_ffn_backward_workspace_bytes(CAP, H, I), s.at["dx"], None, None, BF, None) == B.MOE_OK
    assert B.lib().dense_ffn_backward(None, None, 0, H, I, s.at["dw13"], None,
                                      ctypes.byref(B.moe_saved(0, None, None)), None, 0, None,
                                      s.at["dw13"], s.at["dw13"], BF, None) == B.MOE_EINVAL
    assert b"dw13 and dw2 overlap" in B.lib().moe_last_error()


@pytest.mark.parametrize("grouped", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
def test_forward(L, grouped, fp8):  # noqa: F811
    rows = CAP if grouped else T
    n = B.lib().moe_ffn_train_workspace_bytes(rows, H, I)
    size = sizes(rows, E if grouped else 1, BF, fp8)
    size = {**{k: size[k] for k in ("x", "w13", "w2", "h", "scales")}, "rows": rows * H * 2,
            "workspace": n}

    def forward(a):
        saved = ctypes.byref(B.moe_saved(int(fp8), a["h"], a["scales"] if fp8 else None))
        if grouped:
            ptr = 1 << 16
            plan = ctypes.byref(B.moe_plan(ptr, ptr, ptr, ptr, ptr, 16, CAP))
            return B.lib().moe_grouped_ffn_train(a["x"], T, H, I, E, K, a["w13"], a["w2"], plan, saved,
                                                 a["workspace"], n, a["rows"], None)
        return B.lib().dense_ffn_train(a["x"], T, H, I, a["w13"], a["w2"], saved, a["workspace"], n,
                                       a["rows"], None)

    s = Space(**size)
    far = Space(**{"_": 1 << 40, **size})
    pairs = [(w, o) for w in ("h", "workspace") + (("scales",) if fp8 else ())
             for o in ("x", "w13", "w2", "rows")] + [("h", "workspace"), ("rows", "w2")]
    for a, b in pairs + ([("h", "scales"), ("scales", "workspace")] if fp8 else []):
        for w, o in ((a, b), (b, a)):
            for at in (s.at[o], s.last(o)):
                assert forward({**far.at, o: s.at[o], w: at}) == B.MOE_EINVAL, (w, o)
                assert b"over" in B.lib().moe_last_error(), (w, o)


@pytest.mark.parametrize("dt", [BF, F32])
def test_pack(L, dt):  # noqa: F811
    size = dict(x=T * H * (2 if dt == BF else 4), codes=T * H, scales=T * H // 32)
    far = Space(**{"_": 1 << 40, **size})

    def pack(a):
        return B.lib().moe_pack_fp8(a["x"], dt, T, H, a["codes"], a["scales"], None)

    def unpack(a):
        return B.lib().moe_unpack_fp8(a["codes"], a["scales"], T, H, a["x"], dt, None)

    s = Space(**size)
    for fn, pairs in ((pack, [("x", "codes"), ("x", "scales"), ("codes", "scales")]),
                      (unpack, [("x", "codes"), ("x", "scales")])):
        for a, b in pairs:
            for w, o in ((a, b), (b, a)):
                for at in (s.at[o], s.last(o)):
                    assert fn({**far.at, o: s.at[o], w: at}) == B.MOE_EINVAL, (fn, w, o)
                    assert b"over" in B.lib().moe_last_error(), (fn, w, o)
