"""Measured cases of training the experts of an MoE layer:

  forward      the experts' gated feed-forward over the rows of an alignment (or the
               dense one of the shared experts), which keeps its gate and up values
  backward     its gradients: rows, gate/up and down weights, from the kept values
  step         both, one after the other, with the kept values in bf16 or in 8 bits
  checkpoint   activations kept in 8 bits with a scale for each 32, and read back

``own = False``: plain torch operations in 32 bits.
``own = True``: the library's entry points.

Values kept in 8 bits: each 32 neighbours of a row share the least power of two s with
max |v| <= 448 s (no less than 2^-127), and v is kept as the e4m3 value nearest to v / s.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SZ = {"bf16": 2, "f32": 4, "fp8": 33 / 32}


# ------------------------------------------------------------------ the cases

def _experts(name, op, T, H, I, E, K, block, routing="uniform", pad="block", budget=False,
             save="bf16", want="all"):
    return dict(name=name, op=op, dense=False, T=T, H=H, I=I, E=E, K=K, block=block,
                routing=routing, pad=pad, budget=budget, save=save, want=want)


def _dense(name, op, T, H, I, save="bf16", want="all"):
    return dict(name=name, op=op, dense=True, T=T, H=H, I=I, E=1, K=1, block=1, routing="uniform",
                pad="block", budget=False, save=save, want=want)


def listed():
    return [
        # a step of the tiny layer, where launches are all there is
        _experts("step_tiny", "step", 64, 128, 256, 8, 2, 16),
        # one token of a Mixtral-shaped layer: its two experts' weights read once
        _experts("forward_one", "forward", 1, 4096, 14336, 8, 2, 16),
        # a Mixtral-shaped layer's forward on a training batch of 4096 tokens
        _experts("forward_batch", "forward", 4096, 4096, 14336, 8, 2, 128),
        # and its backward: the largest case
        _experts("backward_batch", "backward", 4096, 4096, 14336, 8, 2, 128),
        # a Qwen2-shaped layer with skewed routing and a budget for each token, 8-bit values kept
        _experts("step_skewed", "step", 3001, 3584, 2560, 64, 8, 128, routing="zipf", budget=True,
                 save="fp8"),
        # few tokens for many experts: the weights' gradients are mostly written, not computed
        _experts("backward_few", "backward", 128, 3584, 2560, 64, 8, 16, save="fp8"),
        # frozen experts (an adapter is trained before them): the rows' gradient alone
        _experts("backward_frozen", "backward", 1024, 3584, 2560, 64, 8, 128, want="rows"),
        # DeepSeek-V3-shaped shared expert on a training batch, 8-bit values kept
        _dense("step_shared", "step", 4096, 7168, 2048, save="fp8"),
        # a small feed-forward with odd sizes: no tile divides them
        _dense("backward_odd", "backward", 1003, 1088, 1856),
        # a decode-sized batch's tokens kept in 8 bits and read back
        dict(name="checkpoint_small", op="checkpoint", T=32, H=4096, dt="bf16"),
        # DeepSeek-V3-shaped layer inputs of a long batch
        dict(name="checkpoint_batch", op="checkpoint", T=16384, H=7168, dt="bf16"),
        # an fp32 residual stream of an odd number of tokens
        dict(name="checkpoint_f32", op="checkpoint", T=5003, H=3584, dt="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# the largest listed case: its experts' weights, and its pairs times an expert's weights
_MOST_W = 8 * 4096 * 14336
_MOST = 8192 * 4096 * 14336


def draw(rng):
    op = rng.choice(["forward", "backward", "backward", "step", "step", "checkpoint"])
    if op == "checkpoint":
        T, H = _log_int(rng, 1, 16384), 32 * _log_int(rng, 1, 256)
        return dict(op=op, T=T, H=H, dt=rng.choice(["bf16", "bf16", "f32"]))
    H = rng.choice([128, 3584, 4096, 7168]) if rng.random() < 0.3 else 64 * _log_int(rng, 1, 112)
    I = rng.choice([256, 2048, 2560, 14336]) if rng.random() < 0.3 else 64 * _log_int(rng, 1, 224)
    T = _log_int(rng, 1, 8192)
    save = rng.choice(["bf16", "fp8"]) if op != "forward" else "bf16"
    want = rng.choice(["all", "all", "rows", "weights"]) if op == "backward" else "all"
    if rng.random() < 0.3:
        while T * H * I > _MOST // 2:
            T = T * 2 // 3
        return {k: v for k, v in _dense("", op, T, H, I, save, want).items() if k != "name"}
    E = _log_int(rng, 1, 64)
    while E * H * I > _MOST_W:
        E //= 2
    K = min(E, _log_int(rng, 1, 8))
    while T * K * H * I > _MOST // 2:
        T = T * 2 // 3
    c = _experts("", op, T, H, I, E, K, rng.choice([1, 16, 64, 128]),
                 rng.choice(["uniform", "zipf"]), rng.choice(["block", "block", "max"]),
                 rng.random() < 0.3, save, want)
    del c["name"]
    return c


def _cap(T, K, E, B, pad):
    if pad == "max":
        return E * (-(-T // B) * B)
    return -(-(T * K + min(E, T * K) * (B - 1)) // B) * B


# ----------------------------------------------------------------- the inputs

class _Rand:
    """Normal and uniform values on the GPU, from one seed."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(1000003 * (seed + 1))

    def normal(self, *shape, std=1.0, dt="bf16"):
        if len(shape) == 3:   # weights: a matrix at a time, their fp32 values are large
            out = torch.empty(*shape, dtype=_DT[dt], device="cuda")
            for m in out:
                m.copy_(torch.randn(*shape[1:], generator=self.g, device="cuda") * std)
            return out
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(_DT[dt])

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")


def _routing(c, rnd):
    """The alignment of a routed batch, as the library's plan holds it."""
    T, K, E, B = c["T"], c["K"], c["E"], c["block"]
    logits = rnd.normal(T, E, dt="f32")
    if c["routing"] == "zipf":
        logits -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    ids = torch.topk(logits, K, dim=1)[1]
    if c["budget"]:   # a budget of 0..K slots for each token
        k_t = (rnd.uniform(T, 1) * (K + 1)).long().clamp(max=K)
        ids = ids.masked_fill(torch.arange(K, device="cuda")[None] >= k_t, -1)
    flat = ids.reshape(-1)
    used = flat >= 0
    counts = torch.bincount(flat[used], minlength=E)
    if c["pad"] == "max":
        size = ((counts.max() + B - 1) // B * B).expand(E)
    else:
        size = (counts + B - 1) // B * B
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.cumsum(size, 0)
    first = torch.cumsum(counts, 0) - counts
    order = torch.argsort(torch.where(used, flat, E), stable=True)[:int(used.sum())]
    e = flat[order]
    pos = off[e] + torch.arange(order.numel(), device="cuda") - first[e]
    cap = _cap(T, K, E, B, c["pad"])
    sorted_ids = torch.full((cap,), T * K, dtype=torch.int32, device="cuda")
    sorted_ids[pos] = order.int()
    inv = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    inv[order] = pos.int()
    rows = torch.arange(0, cap, B, device="cuda")
    block = torch.searchsorted(off, rows, right=True) - 1
    block = torch.where(rows < off[E], block, -1).int()
    return dict(counts=counts.int(), off=off.int(), sorted=sorted_ids, inv=inv, block=block)


def _inputs(c, seed):
    rnd = _Rand(seed)
    T, H = c["T"], c["H"]
    if c["op"] == "checkpoint":
        # a residual stream: a spread of row scales, and a few channels far above the rest
        x = rnd.normal(T, H, std=2.0, dt="f32") * (0.5 + 1.5 * rnd.uniform(T, 1))
        x[:, ::97] *= 6.0
        return dict(x=x.to(_DT[c["dt"]]))
    I, E = c["I"], c["E"]
    s = {} if c["dense"] else _routing(c, rnd)
    R = T if c["dense"] else s["sorted"].numel()
    s["x"] = rnd.normal(T, H)
    s["w13"] = rnd.normal(E, 2 * I, H, std=H ** -0.5)
    s["w2"] = rnd.normal(E, H, I, std=I ** -0.5)
    if c["op"] != "forward":
        s["dy"] = rnd.normal(R, H, std=0.1)
    if c["op"] == "backward":
        # gate and up values as a forward leaves them
        s["h"] = rnd.normal(R, 2 * I)
        if c["save"] == "fp8":
            s["codes"], s["exps"] = _kept(s.pop("h"))
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = c
    if c["op"] != "checkpoint":
        s["groups"] = _groups(c, s)
    if own:
        _handles(c, s)
    return s


def _groups(c, s):
    """[(experts, rows)]: the experts that have rows in classes of like counts, and their rows
    [experts][most], the row past the last where an expert has fewer."""
    if c["dense"]:
        one = torch.zeros(1, dtype=torch.int64, device="cuda")
        return [(one, torch.arange(c["T"], device="cuda")[None])]
    cap = s["sorted"].numel()
    left = sorted(((n, e) for e, n in enumerate(s["counts"].tolist()) if n), reverse=True)
    groups = []
    while left:
        most = left[0][0]
        e = torch.tensor([e for n, e in left if 3 * n > 2 * most], device="cuda")
        left = [(n, i) for n, i in left if 3 * n <= 2 * most]
        j = torch.arange(most, device="cuda")[None]
        rows = s["off"][e].long()[:, None] + j
        groups.append((e, torch.where(j < s["counts"][e][:, None], rows, cap)))
    return groups


def _handles(c, s):
    """The library's plan and kept values, and the buffers that a program allocates once."""
    from mixture_experts_layer_30_amd import binding as B
    T, H = c["T"], c["H"]

    def new(dt, *shape):
        return torch.empty(*shape, dtype=dt, device="cuda")

    if c["op"] == "checkpoint":
        s["o_codes"], s["o_scales"] = new(torch.uint8, T, H), new(torch.uint8, T, H // 32)
        s["o_x"] = torch.empty_like(s["x"])
        return
    I, E = c["I"], c["E"]
    R = T
    if not c["dense"]:
        p = s["plan"] = B.Plan(T, c["K"], E, c["block"], "cuda",
                               pad=B.PAD_MAX if c["pad"] == "max" else B.PAD_BLOCK)
        R = p.cap
        p.expert_counts.copy_(s["counts"])
        p.expert_offsets.copy_(s["off"])
        p.sorted_ids[:R].copy_(s["sorted"])
        p.block_expert[:s["block"].numel()].copy_(s["block"])
        p.inv_pos.copy_(s["inv"])
    s["saved"] = B.Saved(R, I, B.SAVE_FP8 if c["save"] == "fp8" else B.SAVE_BF16, "cuda")
    if c["op"] == "backward":
        if c["save"] == "fp8":
            s["saved"].h.copy_(s["codes"].view(torch.uint8))
            s["saved"].scales.copy_((s["exps"] + 127).to(torch.uint8))
        else:
            s["saved"].h.copy_(s["h"])
    else:
        s["saved"].h.zero_()
        s["fws"] = new(torch.uint8, B.moe_ffn_train_workspace_bytes(R, H, I))
        # rows that hold no pair are left as they were
        s["o_y"] = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    if c["op"] != "forward":
        s["bws"] = new(torch.uint8, B.moe_ffn_backward_workspace_bytes(R, H, I))
        s["o_dx"] = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda") \
            if c["want"] != "weights" else None
        s["o_dw13"] = new(torch.bfloat16, E, 2 * I, H) if c["want"] != "rows" else None
        s["o_dw2"] = new(torch.bfloat16, E, H, I) if c["want"] != "rows" else None


# ------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state["case"], state)
    return _run_plain(state["case"], state)


def _outs(**kw):
    return {k: v for k, v in kw.items() if v is not None}


def _run_own(c, s):
    from mixture_experts_layer_30_amd import binding as B
    op = c["op"]
    if op == "checkpoint":
        B.moe_pack_fp8(s["x"], s["o_codes"], s["o_scales"])
        B.moe_unpack_fp8(s["o_codes"], s["o_scales"], s["o_x"])
        return s["o_x"]
    out = {}
    if op in ("forward", "step"):
        if c["dense"]:
            B.dense_ffn_train(s["x"], s["w13"][0], s["w2"][0], s["saved"], s["fws"], s["o_y"])
        else:
            B.moe_grouped_ffn_train(s["x"], s["w13"], s["w2"], s["plan"], s["saved"], s["fws"],
                                    s["o_y"])
        out["y"] = s["o_y"]
        if op == "forward":
            out["h"] = s["saved"].h
    if op in ("backward", "step"):
        if c["dense"]:
            one = c["want"] != "rows"
            B.dense_ffn_backward(s["dy"], s["x"], s["w13"][0], s["w2"][0], s["saved"], s["bws"],
                                 dx=s["o_dx"], dw13=s["o_dw13"][0] if one else None,
                                 dw2=s["o_dw2"][0] if one else None)
        else:
            B.moe_grouped_ffn_backward(s["dy"], s["x"], s["w13"], s["w2"], s["plan"], s["saved"],
                                       s["bws"], dxrows=s["o_dx"], dw13=s["o_dw13"],
                                       dw2=s["o_dw2"])
        out.update(_outs(dx=s["o_dx"], dw13=s["o_dw13"], dw2=s["o_dw2"]))
    return out


def _kept(v):
    """The e4m3 codes of v's blocks of 32 in a row, and the exponents of their scales."""
    b = v.float().unflatten(-1, (-1, 32))
    m, k = torch.frexp(b.abs().amax(-1))                 # max = m 2^k, 1/2 <= m < 1
    e = (k - 9 + (m > 0.875)).clamp(min=-127)            # 448 = 0.875 2^9
    e = torch.where(m == 0, -127, e)
    codes = (b * _pow2(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.flatten(-2), e


def _pow2(e):
    """2^e in fp32, exactly, for -149 <= e <= 127"""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _read_back(codes, e):
    return (codes.float().unflatten(-1, (-1, 32)) * _pow2(e)[..., None]).flatten(-2)


def _gather(t, rows):
    """Rows of t in fp32, [experts][most]; zeros where there is none."""
    n = t.shape[0]
    return t[rows.clamp(max=n - 1)].float().masked_fill_((rows >= n)[..., None], 0.0)


def _run_plain(c, s):
    op, H = c["op"], c["H"]
    if op == "checkpoint":
        return _read_back(*_kept(s["x"])).to(s["x"].dtype)
    T, I, E = c["T"], c["I"], c["E"]
    R = T if c["dense"] else s["sorted"].numel()
    bf = torch.bfloat16

    def zeros(*shape):
        return torch.zeros(*shape, dtype=bf, device="cuda")

    forward, backward = op in ("forward", "step"), op in ("backward", "step")
    # one row more, for those that an expert of fewer rows than its class lacks
    y = zeros(R + 1, H) if forward else None
    h_all = zeros(R + 1, 2 * I) if op == "forward" else None
    dx = zeros(R + 1, H) if backward and c["want"] != "weights" else None
    dw13 = zeros(E, 2 * I, H) if backward and c["want"] != "rows" else None
    dw2 = zeros(E, H, I) if backward and c["want"] != "rows" else None
    for e, rows in s["groups"]:
        flat = rows.reshape(-1)
        w13, w2 = s["w13"][e].float(), s["w2"][e].float()
        x = None
        if forward or dw13 is not None:
            tok = rows if c["dense"] else s["sorted"][rows.clamp(max=R - 1)].long() // c["K"]
            x = _gather(s["x"], torch.where(rows < R, tok, T))
        if forward:
            h = torch.bmm(x, w13.transpose(1, 2))
            a = torch.sigmoid(h[..., :I]) * h[..., :I] * h[..., I:]
            y[flat] = torch.bmm(a, w2.transpose(1, 2)).to(bf).view(-1, H)
            if op == "forward":
                h_all[flat] = h.to(bf).view(-1, 2 * I)
                continue
            if c["save"] == "fp8":
                h = _read_back(*_kept(h))
        elif c["save"] == "fp8":
            at = rows.clamp(max=R - 1)
            h = _read_back(s["codes"].view(torch.uint8)[at].view(torch.float8_e4m3fn), s["exps"][at])
        else:
            h = _gather(s["h"], rows)
        g, u = h[..., :I], h[..., I:]
        dy = _gather(s["dy"], rows)
        da = torch.bmm(dy, w2)
        sg = torch.sigmoid(g)
        dh = torch.cat([da * u * (sg * (1.0 + g * (1.0 - sg))), da * (g * sg)], -1)
        if dx is not None:
            dx[flat] = torch.bmm(dh, w13).to(bf).view(-1, H)
        if dw13 is not None:
            dw13[e] = torch.bmm(dh.transpose(1, 2), x).to(bf)
            dw2[e] = torch.bmm(dy.transpose(1, 2), g * sg * u).to(bf)
    if op == "forward":
        return dict(y=y[:R], h=h_all[:R])
    return _outs(y=y[:R] if forward else None, dx=dx[:R] if dx is not None else None, dw13=dw13,
                 dw2=dw2)


# ----------------------------------------------------------- work and definition

def work(case):
    """Bytes and operations of one pass.  Rows are counted at the pairs alone: how many
    padding rows and unused slots there are depends on the routing; so does how many experts
    have tokens, of which no more than the pairs are counted."""
    c = case
    T, H = c["T"], c["H"]
    if c["op"] == "checkpoint":
        return dict(bytes=int(T * H * (2 * _SZ[c["dt"]] + 2 * _SZ["fp8"])), flops=4 * T * H)
    I, E = c["I"], c["E"]
    pairs = max(1, int(T * c["K"] * (0.5 if c["budget"] else 1.0)))
    weights = min(E, pairs) * 3 * H * I
    h = pairs * 2 * I * _SZ[c["save"]]
    mm = 2 * pairs * H * I   # operations of a product of [pairs][I] values with a weight
    b, f = 2 * weights, 0
    if c["op"] in ("forward", "step"):
        b += 2 * T * H + h + 2 * pairs * H
        f += 3 * mm
    if c["op"] in ("backward", "step"):
        b += h + 2 * pairs * H
        f += mm
        if c["want"] != "weights":
            b += 2 * pairs * H
            f += 2 * mm
        if c["want"] != "rows":
            b += 2 * E * 3 * H * I + (2 * T * H if c["op"] == "backward" else 0)
            f += 3 * mm
    return dict(bytes=int(b), flops=int(f))


def _nearest_e4m3(v):
    """v (64 bits, |v| <= 448) to the nearest e4m3 value, ties to the even one: steps of 2^-3
    of the value's power of two, of 2^-9 below 2^-6."""
    k = torch.frexp(v)[1] - 1
    step = _power(k.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _power(e):
    """2^e in 64 bits, -200 <= e <= 200, from a table: the GPU's pow need not be exact."""
    table = torch.tensor([2.0 ** k for k in range(-200, 201)], dtype=torch.float64, device=e.device)
    return table[e.long() + 200]


def _kept_exact(v):
    b = v.double().unflatten(-1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(most / 448.0)).clamp(-127, 127)
    e = torch.where(most == 0, torch.full_like(e, -127), e)
    # the logarithm is rounded: one step either way, by the definition itself
    e = torch.where(most > 448.0 * _power(e), e + 1, e)
    e = torch.where((e > -127) & (most <= 448.0 * _power(e - 1)), e - 1, e)
    s = _power(e)
    return (_nearest_e4m3(b / s) * s).flatten(-2)


def _kept_values(codes, e):
    return (codes.float().double().unflatten(-1, (-1, 32)) * _power(e)[..., None]).flatten(-2)


def exact(case, seed):
    """What run returns, from the definitions in 64 bits, an expert at a time."""
    c = case
    s = _inputs(c, seed)
    D = torch.float64
    if c["op"] == "checkpoint":
        return torch.cat([_kept_exact(x) for x in s["x"].split(2048)])
    op, T, H, I, E = c["op"], c["T"], c["H"], c["I"], c["E"]
    R = T if c["dense"] else s["sorted"].numel()

    def zeros(*shape):
        return torch.zeros(*shape, dtype=D, device="cuda")

    out = {}
    if op in ("forward", "step"):
        out["y"] = zeros(R, H)
    if op == "forward":
        out["h"] = zeros(R, 2 * I)
    if op != "forward":
        if c["want"] != "weights":
            out["dx"] = zeros(R, H)
        if c["want"] != "rows":
            out["dw13"], out["dw2"] = zeros(E, 2 * I, H), zeros(E, H, I)
    counts = [T] if c["dense"] else s["counts"].tolist()
    first = [0] if c["dense"] else s["off"].tolist()
    for e in range(E):
        if not counts[e]:
            continue
        at = slice(first[e], first[e] + counts[e])
        x = s["x"] if c["dense"] else s["x"][s["sorted"][at].long() // c["K"]]
        x, w13, w2 = x.double(), s["w13"][e].double(), s["w2"][e].double()
        if op == "backward":
            h = s["h"][at].double() if c["save"] == "bf16" else \
                _kept_values(s["codes"][at], s["exps"][at])
        else:
            h = x @ w13.t()
            a = h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]
            out["y"][at] = a @ w2.t()
            if op == "forward":
                out["h"][at] = h
                continue
            if c["save"] == "fp8":
                h = _kept_exact(h)
        g, u = h[:, :I], h[:, I:]
        dy = s["dy"][at].double()
        da = dy @ w2
        q = 1 / (1 + torch.exp(-g))
        dh = torch.cat([da * u * q * (1 + g - g * q), da * g * q], 1)
        if "dx" in out:
            out["dx"][at] = dh @ w13
        if "dw13" in out:
            out["dw13"][e] = dh.t() @ x
            out["dw2"][e] = dy.t() @ (g * q * u)
    return out
