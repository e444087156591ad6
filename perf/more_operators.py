"""Measured cases of three operators that train and serve a model around the MoE layer.

grouped  products grouped by expert with ragged sizes: rows sorted by expert (the layer's ``expert_offsets``) times each
         expert's bf16 weight; forward, data gradient and weight gradient.
xent     softmax cross entropy over a large vocabulary from the hidden states and the head's weight, in pieces of the
         vocabulary, without keeping the logits; loss and log-sum-exp, and the gradients of both operands.
lora     low-rank adapters of many requests beside a shared projection: each row names its adapter or none; added to
         the projection's result, and the gradients of the input and of every adapter.

Each case runs through ``run`` in one of two ways: ``own`` false, elementary torch operations in fp32; ``own``
true, the calls of :mod:`fp4_weight_grouped_amd.v4moe`.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ---- cases ------------------------------------------------------------------------------------------------
def _grouped(**kw):
    return dict(dict(op="grouped", way="forward", M=8, N=2048, K=4096, E=256, spread=0.3, pad=0), **kw)


def _xent(**kw):
    return dict(dict(op="xent", way="forward", T=16, H=4096, V=131072, ignored=0.0, weighted=False, pad=0), **kw)


def _lora(**kw):
    return dict(dict(op="lora", way="forward", M=64, N=4096, K=4096, r=16, L=64, none=0.1, runs=False, pad=0), **kw)


def listed():
    return [
        # one token of a decode step, top-8: one row for each of eight experts
        _grouped(name="grouped_token", M=8, spread=0.0),
        # the repository's decode batch (T = 128, top-8, E = 256): four rows an expert, the weights' bytes
        _grouped(name="grouped_decode", M=1024),
        # the repository's prefill batch (T = 8192, top-8): matrix products of some 256 rows each
        _grouped(name="grouped_prefill", M=65536),
        # a small training batch over a few experts, no size a multiple of 8, inside wider rows
        _grouped(name="grouped_backward_odd", way="backward", M=3001, N=1001, K=499, E=12, spread=0.8, pad=9),
        # a training batch's data and weight gradients
        _grouped(name="grouped_backward", way="backward", M=32768, N=4096, K=2048, E=32),
        # the log-likelihoods of a few tokens: the head's bytes
        _xent(name="xent_tokens", T=16),
        # scoring a long batch, some tokens without a target
        _xent(name="xent_forward", T=8192, ignored=0.1),
        # a batch and a vocabulary of odd sizes, most tokens without a target (prompts), a weight for each token
        _xent(name="xent_backward_odd", way="backward", T=1237, H=1001, V=50021, ignored=0.6, weighted=True, pad=3),
        # a training step's gradients
        _xent(name="xent_backward", way="backward", T=4096),
        # a decode batch: 64 requests, each with an adapter of its own
        _lora(name="lora_decode"),
        # a prefill batch of a few requests
        _lora(name="lora_prefill", M=8192, r=64, L=16, runs=True),
        # a training batch of a few adapters
        _lora(name="lora_backward", way="backward", M=8192, N=2048, r=32, L=8, runs=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped", "xent", "lora"))
    unit = rng.choice((1, 8, 64))
    size = lambda lo, hi: max(1, _log_int(rng, lo, hi) // unit) * unit  # noqa: E731
    pad = rng.choice((0, 0, 8, 3))
    if op == "grouped":
        return _grouped(way=rng.choice(("forward", "forward", "backward")), M=_log_int(rng, 1, 16384), N=size(64, 4096),
                        K=size(64, 4096), E=_log_int(rng, 1, 96), spread=rng.choice((0.0, 0.3, 0.8)), pad=pad)
    if op == "xent":
        return _xent(way=rng.choice(("forward", "backward")), T=_log_int(rng, 1, 4096), H=size(64, 3000),
                     V=size(512, 100000), ignored=rng.choice((0.0, 0.1, 0.6)), weighted=rng.random() < 0.5, pad=pad)
    return _lora(way=rng.choice(("forward", "forward", "backward")), M=_log_int(rng, 1, 8192), N=size(64, 4096),
                 K=size(64, 4096), r=rng.choice((4, 8, 16, 16, 32, 64, 24)), L=_log_int(rng, 1, 64),
                 none=rng.choice((0.0, 0.1, 0.5)), runs=rng.random() < 0.6, pad=pad)


# ---- inputs -----------------------------------------------------------------------------------------------
def _plan(group, count):
    """Where each row of a group goes in a padded batch: (rows, their group's place, their place in it, the groups that
    have rows, the largest), which a program that batches its rows has made once; rows of group < 0 are left out."""
    rows = torch.nonzero(group >= 0).flatten()
    order = torch.argsort(group[rows], stable=True)
    rows = rows[order]
    sizes = torch.bincount(group[rows], minlength=count)
    active = torch.nonzero(sizes).flatten()
    place = torch.zeros(count, dtype=torch.int64)
    place[active] = torch.arange(len(active))
    begin = torch.cumsum(sizes, 0) - sizes
    g = group[rows]
    inside = torch.arange(len(rows)) - begin[g]
    return dict(rows=rows.to(DEV), place=place[g].to(DEV), inside=inside.to(DEV), active=active.to(DEV),
                most=int(sizes.max()) if len(rows) else 0)


def _groups(c, seed):
    """A group for each row, on the host."""
    g = torch.Generator().manual_seed(seed)
    if c["op"] == "grouped":
        if c["spread"] == 0.0 and c["M"] <= c["E"]:
            return torch.randperm(c["E"], generator=g)[:c["M"]].sort().values      # a token's experts are distinct
        share = torch.exp(c["spread"] * torch.randn(c["E"], generator=g))
        return torch.multinomial(share, c["M"], replacement=True, generator=g).sort().values
    if c["runs"]:                                                                  # requests of some length, in order
        cuts = (torch.rand(c["M"], generator=g) < 2 * c["L"] / c["M"]).long()
        ids = torch.randint(0, c["L"], (c["M"] + 1,), generator=g)
        off = torch.rand(c["M"] + 1, generator=g) < c["none"]
        run = torch.cumsum(cuts, 0)
        return torch.where(off[run], -1, ids[run])
    ids = torch.randint(0, c["L"], (c["M"],), generator=g)
    return torch.where(torch.rand(c["M"], generator=g) < c["none"], -1, ids)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=BF16, device=DEV).normal_(generator=g).mul_(std)

    def wide(rows, cols, std=1.0):          # rows of a wider matrix
        return normal(rows, cols + c["pad"], std=std)[:, :cols]

    s = dict(case=c)
    if c["op"] == "grouped":
        group = _groups(c, seed)
        counts = torch.bincount(group, minlength=c["E"])
        offsets = torch.zeros(c["E"] + 1, dtype=torch.int32)
        offsets[1:] = torch.cumsum(counts, 0)
        s.update(x=wide(c["M"], c["K"]), w=normal(c["E"], c["N"], c["K"], std=c["K"] ** -0.5), offsets=offsets.to(DEV),
                 plan=_plan(group, c["E"]))
        if c["way"] == "backward":
            s["dy"] = wide(c["M"], c["N"], std=1e-3)
        return s
    if c["op"] == "xent":
        T, H, V = c["T"], c["H"], c["V"]
        s.update(x=wide(T, H), w=normal(V, H, std=1.3 * H ** -0.5))
        targets = torch.randint(0, V, (T,), generator=g, device=DEV)
        targets[torch.rand(T, generator=g, device=DEV) < c["ignored"]] = -100
        s["targets"] = targets
        if c["way"] == "backward":
            kept = (targets >= 0).sum().clamp(min=1)
            s["lse"] = _plain_xent(s["x"], s["w"], targets)["lse"]
            if c["weighted"]:
                s["dloss"] = torch.rand(T, generator=g, device=DEV) / kept
            else:
                s["dloss"] = (1.0 / kept.float()).expand(T)       # what the mean's backward gives
        return s
    M, N, K, r, L = c["M"], c["N"], c["K"], c["r"], c["L"]
    group = _groups(c, seed)
    s.update(x=wide(M, K), a=normal(L, r, K, std=K ** -0.5), b=normal(L, r, N, std=0.5 * r ** -0.5),
             ids=group.to(torch.int32).to(DEV), scale=torch.rand(L, generator=g, device=DEV) + 0.5, plan=_plan(group, L))
    if c["way"] == "backward":
        s.update(dy=wide(M, N, std=1e-3), base=normal(M, K, std=1e-3))
    else:
        s["y"] = normal(M, N)
    return s


# ---- the plain forms --------------------------------------------------------------------------------------
def _padded(plan, t):
    """Rows of t in a batch of groups: [groups with rows][the largest][columns], fp32, zeros behind a group's rows."""
    p = torch.zeros(len(plan["active"]), plan["most"], t.shape[1], device=DEV)
    p[plan["place"], plan["inside"]] = t[plan["rows"]].float()
    return p


def _unpadded(plan, p, base):
    """base (fp32) with the groups' rows added."""
    base[plan["rows"]] += p[plan["place"], plan["inside"]]
    return base


def _spread(plan, t, count):
    """[groups with rows][...] in [all groups][...], zeros for groups without."""
    full = torch.zeros(count, *t.shape[1:], device=DEV)
    full[plan["active"]] = t
    return full


def _plain_grouped(s):
    c, plan = s["case"], s["plan"]
    x, w = _padded(plan, s["x"]), s["w"][plan["active"]].float()
    if c["way"] == "forward":
        y = torch.bmm(x, w.transpose(1, 2).contiguous())
        return {"y": _unpadded(plan, y, torch.zeros(c["M"], c["N"], device=DEV)).to(BF16)}
    dy = _padded(plan, s["dy"])
    dx = _unpadded(plan, torch.bmm(dy, w), torch.zeros(c["M"], c["K"], device=DEV))
    dw = _spread(plan, torch.bmm(dy.transpose(1, 2).contiguous(), x), c["E"])
    return {"dx": dx.to(BF16), "dw": dw.to(BF16)}


def _plain_xent(x, w, targets):
    z = x.float() @ w.float().t()
    m = z.max(dim=1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))).flatten()
    kept = targets >= 0
    zy = z.gather(1, targets.clamp(min=0).unsqueeze(1)).flatten()
    return {"loss": torch.where(kept, lse - zy, 0.0), "lse": torch.where(kept, lse, 0.0)}


def _plain_xent_backward(s):
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    kept = (targets >= 0).unsqueeze(1)
    p = torch.exp(x @ w.t() - s["lse"].unsqueeze(1))
    p.scatter_add_(1, targets.clamp(min=0).unsqueeze(1), torch.full_like(p[:, :1], -1.0))
    p = torch.where(kept, p * s["dloss"].unsqueeze(1), 0.0)
    return {"dx": (p @ w).to(BF16), "dw": (p.t() @ torch.where(kept, x, 0.0)).to(BF16)}


def _plain_lora(s):
    c, plan = s["case"], s["plan"]
    a, b = s["a"][plan["active"]].float(), s["b"][plan["active"]].float()
    scale = s["scale"][plan["active"]].view(-1, 1, 1)
    x = _padded(plan, s["x"])
    u = torch.bmm(x, a.transpose(1, 2).contiguous()) * scale
    if c["way"] == "forward":
        return {"out": _unpadded(plan, torch.bmm(u, b), s["y"].float()).to(BF16)}
    dy = _padded(plan, s["dy"])
    du = torch.bmm(dy, b.transpose(1, 2).contiguous()) * scale
    dx = _unpadded(plan, torch.bmm(du, a), s["base"].float())
    da = torch.bmm(du.transpose(1, 2).contiguous(), x)
    db = torch.bmm(u.transpose(1, 2).contiguous(), dy)
    return {"dx": dx.to(BF16), "da": _spread(plan, da, c["L"]).to(BF16), "db": _spread(plan, db, c["L"]).to(BF16)}


def _plain(s):
    c = s["case"]
    if c["op"] == "grouped":
        return _plain_grouped(s)
    if c["op"] == "xent":
        return _plain_xent(s["x"], s["w"], s["targets"]) if c["way"] == "forward" else _plain_xent_backward(s)
    return _plain_lora(s)


# ---- the framework's calls --------------------------------------------------------------------------------
def _own(s):
    from fp4_weight_grouped_amd import v4moe
    c = s["case"]
    if c["op"] == "grouped":
        if c["way"] == "forward":
            return {"y": v4moe.grouped_linear(s["x"], s["w"], s["offsets"])}
        dx, dw = v4moe.grouped_linear_backward(s["x"], s["dy"], s["w"], s["offsets"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "xent":
        if c["way"] == "forward":
            loss, lse = v4moe.linear_xent(s["x"], s["w"], s["targets"])
            return {"loss": loss, "lse": lse}
        dx, dw = v4moe.linear_xent_backward(s["x"], s["w"], s["targets"], s["lse"], s["dloss"])
        return {"dx": dx, "dw": dw}
    if c["way"] == "forward":
        return {"out": v4moe.lora_add(s["y"], s["x"], s["a"], s["b"], s["ids"], s["scale"])}
    dx, da, db = v4moe.lora_backward(s["x"], s["dy"], s["a"], s["b"], s["ids"], s["scale"], base=s["base"])
    return {"dx": dx, "da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "grouped":
        M, N, K = c["M"], c["N"], c["K"]
        E = min(c["E"], M)                                   # experts with rows, at most
        if c["way"] == "forward":
            return {"bytes": 2 * (M * K + E * N * K + M * N), "flops": 2 * M * N * K}
        return {"bytes": 2 * (2 * M * K + M * N + E * N * K + c["E"] * N * K), "flops": 4 * M * N * K}
    if c["op"] == "xent":
        T, H, V = c["T"] * (1 - c["ignored"]), c["H"], c["V"]
        if c["way"] == "forward":
            return {"bytes": int(2 * (T * H + V * H)) + 16 * c["T"], "flops": int(2 * T * H * V)}
        # the logits again, then both gradients
        return {"bytes": int(2 * (T * H + c["T"] * H + 2 * V * H)) + 16 * c["T"], "flops": int(6 * T * H * V)}
    M, N, K, r = c["M"], c["N"], c["K"], c["r"]
    R = int(M * (1 - c["none"]))                             # rows with an adapter
    L = min(c["L"], R)                                       # adapters with rows, at most
    if c["way"] == "forward":
        return {"bytes": 2 * (R * K + 2 * M * N + L * r * (K + N)) + 4 * M, "flops": 2 * R * r * (K + N)}
    return {"bytes": 2 * (R * K + R * N + 2 * M * K + (L + c["L"]) * r * (K + N)) + 4 * M, "flops": 6 * R * r * (K + N)}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------
def _exact_grouped(s):
    c = s["case"]
    x, at = s["x"].double(), s["offsets"].tolist()
    back = c["way"] == "backward"
    y = torch.zeros(c["M"], c["K"] if back else c["N"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device=DEV) if back else None
    for e in range(c["E"]):
        i, j = at[e], at[e + 1]
        if i == j:
            continue
        w = s["w"][e].double()
        if not back:
            y[i:j] = x[i:j] @ w.t()
            continue
        dy = s["dy"][i:j].double()
        y[i:j] = dy @ w
        dw[e] = dy.t() @ x[i:j]
    return {"dx": y, "dw": dw} if back else {"y": y}


def _exact_xent(s):
    c = s["case"]
    targets = s["targets"]
    rows = torch.nonzero(targets >= 0).flatten()
    x, w, y = s["x"].double()[rows], s["w"].double(), targets[rows]
    z = x @ w.t()
    T, H, V = c["T"], c["H"], c["V"]
    if c["way"] == "forward":
        lse = torch.logsumexp(z, dim=1)
        loss = lse - z[torch.arange(len(rows), device=DEV), y]
        full = torch.zeros(2, T, dtype=torch.float64, device=DEV)
        full[0, rows], full[1, rows] = loss, lse
        return {"loss": full[0], "lse": full[1]}
    # d loss_t = dloss_t (softmax(z_t) - e_y)
    d = torch.softmax(z, dim=1)
    d[torch.arange(len(rows), device=DEV), y] -= 1.0
    d *= s["dloss"].double()[rows].unsqueeze(1)
    dx = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    dx[rows] = d @ w
    return {"dx": dx, "dw": d.t() @ x}


def _exact_lora(s):
    c = s["case"]
    x, ids = s["x"].double(), s["ids"]
    back = c["way"] == "backward"
    out = (s["base"] if back else s["y"]).double()
    da = torch.zeros(c["L"], c["r"], c["K"], dtype=torch.float64, device=DEV) if back else None
    db = torch.zeros(c["L"], c["r"], c["N"], dtype=torch.float64, device=DEV) if back else None
    for i in range(c["L"]):
        rows = torch.nonzero(ids == i).flatten()
        if len(rows) == 0:
            continue
        a, b, k = s["a"][i].double(), s["b"][i].double(), float(s["scale"][i])
        if not back:
            out[rows] += k * (x[rows] @ a.t()) @ b
            continue
        dy = s["dy"][rows].double()
        out[rows] += k * (dy @ b.t()) @ a
        da[i] = k * (dy @ b.t()).t() @ x[rows]
        db[i] = k * (x[rows] @ a.t()).t() @ dy
    return {"dx": out, "da": da, "db": db} if back else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"grouped": _exact_grouped, "xent": _exact_xent, "lora": _exact_lora}[case["op"]](s)
