"""Measured cases of three operators that stand next to the MoE layer in training and serving.

gate     routing from given logits: scores (sigmoid, softmax or sqrt-softplus), a balance bias that only the
         selection sees, group-limited top-k, renormalised weights; and the gradient with respect to the logits.
linear   the matrix product with E4M3 operands and an fp32 scale for each 128 of the contraction (activations:
         per row; weights: per 128x128 block), from bf16 activations: forward, backward, and the quantisation of
         the weights in both layouts that those two read.
clip     the global gradient norm over many tensors, and the gradients scaled down to a largest norm.

Each case runs through ``run`` in one of two ways: ``own`` false, elementary torch operations in fp32; ``own``
true, the calls of :mod:`fp4_weight_grouped_amd.v4moe`.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SCORES = ("sigmoid", "softmax", "sqrtsoftplus")
MASK = 1e30        # logits at or below -MASK, and NaN, are masked; those above MASK count as MASK
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------------------------------------
def _gate(**kw):
    return dict(dict(op="gate", way="forward", T=1, E=256, topk=8, score="sigmoid", bias=True, groups=1, kept=1,
                     renorm=True, scale=1.0, type="f32", pad=0, masked=0.0), **kw)


def _linear(**kw):
    return dict(dict(op="linear", way="forward", M=1, N=4096, K=4096, type="bf16"), **kw)


def _clip(**kw):
    return dict(dict(op="clip", count=1, total=1, bf16=0.0, odd=True, over=4.0), **kw)


def listed():
    return [
        # one token of a decode step: launch latency
        _gate(name="gate_token", T=1, groups=8, kept=4, scale=2.5),
        # a prefill batch of the repository's layer (T = 8192, E = 256, top-8), groups and balance bias
        _gate(name="gate_prefill", T=8192, groups=8, kept=4, scale=2.5),
        # an odd batch over 72 experts, bf16 logits inside wider rows, some experts and some whole rows masked
        _gate(name="gate_softmax_odd", T=3001, E=72, topk=6, score="softmax", bias=False, renorm=False, type="bf16",
              pad=9, masked=0.1),
        # the gradient for the repository's ragged batch of 19,647 tokens; softmax without renormalisation reaches
        # every logit
        _gate(name="gate_backward", way="backward", T=19647, score="softmax", bias=False, renorm=False),
        # one token through a dense projection: weight streaming and latency
        _linear(name="linear_token", M=1, N=4096, K=2048),
        # the repository's decode batch
        _linear(name="linear_decode", M=128, N=4096, K=4096),
        # the repository's prefill batch
        _linear(name="linear_prefill", M=8192, N=4096, K=4096),
        # a ragged training batch, no size a multiple of a tile or of 16
        _linear(name="linear_backward_odd", way="backward", M=1237, N=1999, K=1001),
        # a training batch's data and weight gradients
        _linear(name="linear_backward", way="backward", M=8192, N=2048, K=4096),
        # fp32 master weights to E4M3 after an optimizer step, in the layout of each direction
        _linear(name="linear_weights", way="weights", M=0, N=16384, K=4096, type="f32"),
        # a small model's gradients, both types, odd sizes, unaligned views
        _clip(name="clip_small", count=23, total=3_000_001, bf16=0.5),
        # one layer's expert gradients on one GPU: three fp32 tensors
        _clip(name="clip_experts", count=3, total=3 * 32 * 2048 * 4096, odd=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gate", "gate", "linear", "linear", "linear", "clip"))
    if op == "gate":
        groups = rng.choice((1, 1, 2, 4, 8))
        size = _log_int(rng, 2, 512 // groups)          # experts per group
        E = groups * size
        kept = rng.randint(1, groups)
        topk = rng.randint(1, min(16, kept * size))
        score = rng.choice(SCORES)
        way = rng.choice(("forward", "forward", "backward"))
        return _gate(way=way, T=_log_int(rng, 1, 20000), E=E, topk=topk, score=score, bias=rng.random() < 0.6,
                     groups=groups, kept=kept, renorm=rng.random() < 0.6 and topk > 1, scale=rng.choice((1.0, 2.5)),
                     type=rng.choice(("f32", "bf16")), pad=rng.choice((0, 0, 1, 8)), masked=rng.choice((0.0, 0.0, 0.05)))
    if op == "linear":
        way = rng.choice(("forward", "forward", "forward", "backward", "backward", "weights"))
        unit = rng.choice((1, 16, 128))
        size = lambda: max(1, _log_int(rng, 64, 3000) // unit) * unit  # noqa: E731
        M = 0 if way == "weights" else _log_int(rng, 1, 8192)
        return _linear(way=way, M=M, N=size(), K=size(), type="bf16" if way != "weights" else rng.choice(("f32", "bf16")))
    return _clip(count=_log_int(rng, 1, 60), total=_log_int(rng, 2000, 300_000_000), bf16=rng.choice((0.0, 0.5, 1.0)),
                 odd=rng.random() < 0.7, over=rng.choice((0.5, 4.0)))


# ---- inputs -----------------------------------------------------------------------------------------------
def _up(n, m):
    return (n + m - 1) // m * m


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, type=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(type)

    c = case
    if c["op"] == "gate":
        T, E, t = c["T"], c["E"], TYPES[c["type"]]
        z = normal(T, E, std=1.3)
        if c["masked"]:
            # single experts switched off by the type's lowest value or -inf, and whole rows (padding tokens)
            off = torch.rand(T, E, generator=g, device=DEV) < c["masked"]
            low = torch.where(torch.rand(T, 1, generator=g, device=DEV) < 0.5, torch.finfo(t).min, -math.inf)
            off |= torch.rand(T, 1, generator=g, device=DEV) < c["masked"]
            z = torch.where(off, low, z)
        wide = torch.zeros(T, E + c["pad"], dtype=t, device=DEV)
        wide[:, :E] = z
        s = dict(case=c, logits=wide[:, :E], bias=None)
        if c["bias"]:
            s["bias"] = normal(E, std={"sigmoid": 0.05, "softmax": 0.3 / E, "sqrtsoftplus": 0.1}[c["score"]])
        if c["way"] == "backward":
            # what the forward gave: distinct ids, and weights of the layer's size; dead slots have weight zero
            ids, w = _plain_gate(c, s["logits"], s["bias"])
            s.update(ids=ids, w=w, dw=normal(T, c["topk"]))
        return s
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        w = normal(N, K, std=0.02)
        if c["way"] == "weights":
            return dict(case=c, w=w.to(TYPES[c["type"]]))
        # a checkpoint's E4M3 weights: codes in rows padded with zeros to 16 bytes, both orders, and block scales
        q, blk = _plain_blocks(w)
        codes = torch.zeros(N, _up(K, 16), dtype=torch.uint8, device=DEV)
        codes[:, :K] = q.view(torch.uint8)
        codes_t = torch.zeros(K, _up(N, 16), dtype=torch.uint8, device=DEV)
        codes_t[:, :N] = q.view(torch.uint8).t()
        # activations: a few channels much larger than the rest, as the layer meets them
        x = normal(M, K) * (1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.01))
        s = dict(case=c, q=codes, qt=codes_t, blk=blk, x=x.to(torch.bfloat16))
        if c["way"] == "backward":
            s["dy"] = normal(M, N, std=1e-3, type=torch.bfloat16) * torch.rand(M, 1, generator=g, device=DEV).to(torch.bfloat16)
        return s
    n = c["count"]
    share = torch.rand(n, generator=torch.Generator().manual_seed(n)) + 0.05 if c["odd"] else torch.ones(n)
    sizes = [max(1, int(c["total"] * v)) for v in (share / share.sum()).tolist()]
    grads, outs = [], []
    for i, k in enumerate(sizes):
        t = torch.bfloat16 if (i * 0.618034) % 1 < c["bf16"] else torch.float32
        at = i % 4 if c["odd"] else 0          # views that begin inside a buffer
        buf = torch.empty(k + at, dtype=t, device=DEV)
        buf.normal_(generator=g).mul_(1e-3 * (1 + i % 5))
        grads.append(buf[at:])
        outs.append(torch.empty(k + at, dtype=t, device=DEV)[at:])
    # the largest norm: a fixed share of about what these gradients have
    about = math.sqrt(sum(k * (1e-3 * (1 + i % 5)) ** 2 for i, k in enumerate(sizes)))
    return dict(case=c, grads=grads, outs=outs, max_norm=about / c["over"])


# ---- the plain forms --------------------------------------------------------------------------------------
def _plain_scores(c, logits):
    z = logits.float()
    masked = torch.isnan(z) | (z <= -MASK)
    z = torch.where(masked, -math.inf, z.clamp(max=MASK))
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    elif c["score"] == "softmax":
        m = z.max(dim=-1, keepdim=True).values
        e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
        # the sum in 64 bits: its 32-bit value, and with it the selection, then does not depend on the order
        total = e.double().sum(dim=-1, keepdim=True).float()
        s = torch.where(total > 0, e / total, 0.0)
    else:
        s = torch.sqrt(z.clamp(min=0.0) + torch.log1p(torch.exp(-z.abs())))
    return z, s, masked


def _plain_gate(c, logits, bias):
    T, E, G = c["T"], c["E"], c["groups"]
    z, s, masked = _plain_scores(c, logits)
    key = s if bias is None else s + bias
    key = torch.where(masked | torch.isnan(key), -math.inf, key)
    if G > 1:
        top = torch.sort(key.view(T, G, E // G), dim=-1, descending=True).values[..., :2]
        group = top[..., 0]
        if E // G > 1:
            group = group + torch.where(top[..., 1] == -math.inf, 0.0, top[..., 1])
        kept = torch.sort(group, dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True)
    ids = order.indices[:, :c["topk"]]
    w = torch.where(order.values[:, :c["topk"]] == -math.inf, 0.0, s.gather(1, ids))
    if c["renorm"]:
        total = w.sum(dim=-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), w * c["scale"]


def _plain_gate_backward(c, logits, ids, w, dw):
    z, s, _ = _plain_scores(c, logits)
    ids = ids.long()
    alive = w != 0
    sj = torch.where(alive, s.gather(1, ids), 0.0)
    if c["renorm"]:
        # d(s_j / S): sums of differences, so equal dw give exactly zero
        total = sj.sum(dim=-1, keepdim=True)
        q = torch.where(total > 0, sj / total, 0.0)
        ds = (q.unsqueeze(1) * (dw.unsqueeze(2) - dw.unsqueeze(1))).sum(dim=-1) * c["scale"] / torch.where(total > 0, total, 1.0)
    else:
        ds = dw * c["scale"]
    ds = torch.where(alive, ds, 0.0)
    zj = z.gather(1, ids)
    if c["score"] == "softmax":
        dz = torch.zeros_like(z).scatter_(1, ids, ds * sj)
        if not c["renorm"]:
            dz = dz - s * (ds * sj).sum(dim=-1, keepdim=True)
    else:
        up = 1.0 / (1.0 + torch.exp(zj))
        d = sj * up if c["score"] == "sigmoid" else 1.0 / (1.0 + torch.exp(-zj)) / (2.0 * torch.where(alive, sj, 1.0))
        dz = torch.zeros_like(z).scatter_(1, ids, torch.where(alive, ds * d, 0.0))
    return dz.to(logits.dtype)


def _plain_scale(amax):
    # divided by a tensor: a division by a number would be a product with its rounded reciprocal
    return torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), 1.0)


def _plain_codes(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_rows(x):
    """The values that x's E4M3 codes stand for, a scale for each row and 128 columns."""
    R, C = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _up(C, 128) - C)).view(R, -1, 128)
    amax = v.abs().amax(dim=-1, keepdim=True)
    s = _plain_scale(amax)
    return (_plain_codes(v / s).float() * s).view(R, -1)[:, :C]


def _plain_blocks(w):
    """E4M3 codes [N][K] of w and the scale of each 128x128 block."""
    N, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, _up(K, 128) - K, 0, _up(N, 128) - N))
    v = v.view(_up(N, 128) // 128, 128, _up(K, 128) // 128, 128)
    amax = v.abs().amax(dim=(1, 3), keepdim=True)
    s = _plain_scale(amax)
    q = _plain_codes(v / s).view(_up(N, 128), _up(K, 128))[:N, :K].contiguous()
    return q, s[:, 0, :, 0].contiguous()


def _plain_weights(s):
    N, K = s["case"]["N"], s["case"]["K"]
    blk = s["blk"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return s["q"][:, :K].view(torch.float8_e4m3fn).float() * blk


def _plain(s):
    c = s["case"]
    if c["op"] == "gate":
        if c["way"] == "forward":
            ids, w = _plain_gate(c, s["logits"], s["bias"])
            return {"ids": ids, "w": w}
        return {"dlogits": _plain_gate_backward(c, s["logits"], s["ids"], s["w"], s["dw"])}
    if c["op"] == "linear":
        if c["way"] == "weights":
            q, blk = _plain_blocks(s["w"])
            return {"q": q, "qt": q.t().contiguous(), "blk": blk}
        if c["way"] == "forward":
            return {"y": (_plain_rows(s["x"]) @ _plain_weights(s).t()).to(torch.bfloat16)}
        dx = _plain_rows(s["dy"]) @ _plain_weights(s)
        dw = _plain_rows(s["dy"].t()) @ _plain_rows(s["x"].t()).t()
        return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}
    norm = torch.sqrt(sum(g.float().square().sum() for g in s["grads"]))
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    return {"norm": norm, "grads": [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]}


# ---- the framework's calls --------------------------------------------------------------------------------
def _own(s):
    from fp4_weight_grouped_amd import v4moe
    c = s["case"]
    if c["op"] == "gate":
        how = dict(score=SCORES.index(c["score"]), renorm=c["renorm"], scale=c["scale"])
        if c["way"] == "forward":
            ids, w = v4moe.gate(s["logits"], c["topk"], bias=s["bias"], groups=c["groups"], topk_groups=c["kept"], **how)
            return {"ids": ids, "w": w}
        return {"dlogits": v4moe.gate_backward(s["logits"], s["ids"], s["w"], s["dw"], **how)}
    if c["op"] == "linear":
        if c["way"] == "weights":
            m = v4moe.fp8_weights(s["w"])
            q, qt = m.q[:, :c["K"]], m.qt[:, :c["N"]]
            return {"q": q.view(torch.float8_e4m3fn), "qt": qt.view(torch.float8_e4m3fn), "blk": m.blk}
        m = v4moe.FP8Matrix(c["N"], c["K"], s["q"], s["qt"], s["blk"])
        if c["way"] == "forward":
            return {"y": v4moe.fp8_linear(s["x"], m)}
        dx, dw = v4moe.fp8_linear_backward(s["x"], s["dy"], m)
        return {"dx": dx, "dw": dw}
    norm = v4moe.clip_grads(s["grads"], s["max_norm"], out=s["outs"])
    return {"norm": norm, "grads": s["outs"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "gate":
        T, E, k, size = c["T"], c["E"], c["topk"], 4 if c["type"] == "f32" else 2
        if c["way"] == "forward":
            return {"bytes": T * E * size + T * k * 8 + (4 * E if c["bias"] else 0), "flops": T * E * 8}
        dense = c["score"] == "softmax" and not c["renorm"]        # otherwise only the picked logits are needed
        return {"bytes": T * E * size + T * (E if dense else k) * size + T * k * 12, "flops": T * (E if dense else k) * 8}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        blocks = _up(N, 128) // 128 * (_up(K, 128) // 128) * 4
        if c["way"] == "weights":
            return {"bytes": N * K * ((4 if c["type"] == "f32" else 2) + 2) + blocks, "flops": 3 * N * K}
        if c["way"] == "forward":
            return {"bytes": 2 * M * K + N * K + blocks + 2 * M * N, "flops": 2 * M * N * K}
        return {"bytes": 2 * M * K + 2 * M * N + N * K + blocks + 2 * M * K + 2 * N * K, "flops": 4 * M * N * K}
    n = c["total"]
    return {"bytes": 2 * n * (4 - 2 * c["bf16"]), "flops": 3 * n}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------
def _exact_scores(c, logits):
    z = torch.nan_to_num(logits.double(), nan=-math.inf, posinf=MASK, neginf=-math.inf)
    z[z <= -MASK] = -math.inf
    z[z > MASK] = MASK
    if c["score"] == "sigmoid":
        return z, torch.sigmoid(z)
    if c["score"] == "softmax":
        return z, torch.nan_to_num(torch.softmax(z, dim=-1), nan=0.0)
    return z, torch.sqrt(torch.logaddexp(z, torch.zeros_like(z)))


def _exact_gate(c, s):
    z, p = _exact_scores(c, s["logits"])
    key = p + (0.0 if s["bias"] is None else s["bias"].double())
    key[z == -math.inf] = -math.inf
    G, n = c["groups"], c["E"] // c["groups"]
    if G > 1:
        top = key.view(-1, G, n).topk(min(2, n), dim=-1).values
        second = top[..., 1:].clone()
        second[second == -math.inf] = 0.0
        group = top[..., 0] + second.sum(dim=-1)
        # a group is out if at least `kept` others are larger, or equal with a lower number
        less = torch.arange(G, device=DEV)[:, None] > torch.arange(G, device=DEV)[None, :]
        ahead = (group[:, None, :] > group[:, :, None]) | ((group[:, None, :] == group[:, :, None]) & less)
        out = ahead.sum(dim=-1) >= c["kept"]
        key.view(-1, G, n)[out] = -math.inf
    order = torch.argsort(-key, dim=-1, stable=True)[:, :c["topk"]]
    w = p.gather(1, order) * (key.gather(1, order) > -math.inf)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(dim=-1, keepdim=True), nan=0.0)
    return {"ids": None, "w": w * c["scale"]}


def _exact_gate_backward(c, s):
    z, _ = _exact_scores(c, s["logits"])
    ids, alive = s["ids"].long(), s["w"] != 0
    with torch.enable_grad():
        z = z.clamp(min=-MASK).requires_grad_(True)
        if c["score"] == "sigmoid":
            p = torch.sigmoid(z)
        elif c["score"] == "softmax":
            p = torch.softmax(z, dim=-1)
        else:
            # d sqrt(softplus) = sigmoid(z) / (2 sqrt(softplus)); zero where the score is
            p = torch.sqrt(torch.logaddexp(z, torch.zeros_like(z)).clamp(min=1e-300))
        pj = torch.where(alive, p.gather(1, ids), 0.0)
        w = pj / pj.sum(dim=-1, keepdim=True).clamp(min=1e-300) if c["renorm"] else pj
        (c["scale"] * (w * s["dw"].double()).sum()).backward()
    return {"dlogits": torch.nan_to_num(z.grad, nan=0.0)}


def _exact_codes(v):
    """The nearest E4M3 values, ties to the even code."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_scaled(x, tile):
    """(E4M3 values, scales spread over the elements) of x, a scale for each tile = (rows, columns)."""
    R, C = x.shape
    r, k = tile
    v = torch.zeros(_up(R, r), _up(C, k), dtype=torch.float64, device=DEV)
    v[:R, :C] = x.double()
    t = v.unfold(0, r, r).unfold(1, k, k)
    amax = t.abs().amax(dim=(-1, -2))
    s = torch.where(amax > 0, (amax / E4M3_MAX).float().double(), 1.0)       # scales are fp32 by definition
    wide = s.repeat_interleave(r, 0)[:R].repeat_interleave(k, 1)[:, :C]
    # the quotient is fp32 by definition too: many of them lie on a tie, which the rounding of s would undo
    return _exact_codes((v[:R, :C] / wide).float().double()), wide, s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gate":
        return _exact_gate(c, s) if c["way"] == "forward" else _exact_gate_backward(c, s)
    if c["op"] == "linear":
        if c["way"] == "weights":
            q, _, blk = _exact_scaled(s["w"], (128, 128))
            return {"q": q, "qt": q.t().contiguous(), "blk": blk}
        N, K = c["N"], c["K"]
        code = s["q"][:, :K].long()
        sign, e, m = 1.0 - 2.0 * (code >> 7), (code >> 3) & 15, (code & 7).double()
        w = sign * torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
        row, col = torch.arange(N, device=DEV) // 128, torch.arange(K, device=DEV) // 128
        w = w * s["blk"].double()[row][:, col]
        values = lambda x: (lambda q, wide, _: q * wide)(*_exact_scaled(x, (1, 128)))  # noqa: E731
        if c["way"] == "forward":
            return {"y": values(s["x"]) @ w.t()}
        return {"dx": values(s["dy"]) @ w, "dw": values(s["dy"].t()) @ values(s["x"].t()).t()}
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
    coef = min(1.0, s["max_norm"] / norm)
    return {"norm": norm, "grads": [g.double() * coef for g in s["grads"]]}
