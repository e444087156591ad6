"""The grouped products, the cross entropy and the adapters together, as a model uses them: in one step with the
projection, the gate, the permutation, the combination and the clipping; captured; by several threads; and their
refusals of other devices."""
import threading

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _float32():
    old = torch.get_default_dtype()
    torch.set_default_dtype(F32)
    yield
    torch.set_default_dtype(old)


class Model:
    """a -> projection + adapters -> gate -> experts (squared ReLU, bf16 weights) -> head -> loss, and back."""

    def __init__(self, T, H, I, E, k, V, r, L, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=DEV).mul_(shape[-1] ** -0.5).to(BF16)

        self.T, self.H, self.E, self.k, self.L = T, H, E, k, L
        self.dims = v4moe.dims(T, H, 256, E, k, v4moe.ACT_RELU2)     # (the permutation and the combination read no I)
        self.projection = v4moe.fp8_weights(weight(H, H).float())
        self.a, self.b = weight(L, r, H), torch.randn(L, r, H, generator=g, device=DEV).mul_(r ** -0.5).to(BF16)
        self.scale = torch.rand(L, generator=g, device=DEV) + 0.5
        self.router, self.up, self.down, self.head = weight(1, E, H), weight(E, I, H), weight(E, H, I), weight(V, H)
        self.whole = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        self.dloss = torch.full((1,), 1.0 / T, device=DEV).expand(T)
        self.ws = torch.empty(v4moe.moe_workspace_bytes(self.dims), dtype=torch.uint8, device=DEV)

    def step(self, x, ids, targets):
        """Every tensor that the operators read and write, by name."""
        T, H, k, d = self.T, self.H, self.k, self.dims
        new = lambda *shape, t=F32: torch.empty(*shape, dtype=t, device=DEV)  # noqa: E731
        y0 = v4moe.fp8_linear(x, self.projection)
        h = v4moe.lora_add(y0, x, self.a, self.b, ids, self.scale)
        logits = v4moe.grouped_linear(h, self.router, self.whole, out=new(T, self.E))
        topk, w = v4moe.gate(logits, k)
        off, sp, pp = new(self.E + 1, t=torch.int32), new(T * k, t=torch.int32), new(T * k, t=torch.int32)
        v4moe.moe_permute(d, h, topk, off, sp, pp, new(T, H, t=torch.uint8), new(T, H // 128), self.ws)
        rows = h[sp.long() // k]
        u = v4moe.grouped_linear(rows, self.up, off)
        v = u.relu().square()
        yd = v4moe.grouped_linear(v, self.down, off)
        y, out = torch.empty_like(yd), new(T, H, t=BF16)
        y[sp.long()] = yd
        v4moe.moe_combine(d, y, w, out)
        loss, lse = v4moe.linear_xent(out, self.head, targets)

        dout, dhead = v4moe.linear_xent_backward(out, self.head, targets, lse, self.dloss, dw=new(*self.head.shape))
        per_pair = dout.float()[:, None].expand(T, k, H)
        dw = (per_pair * y.view(T, k, H).float()).sum(2)
        dyd = (per_pair * w[:, :, None]).to(BF16).view(T * k, H)[sp.long()]
        dv, ddown = v4moe.grouped_linear_backward(v, dyd, self.down, off, dw=new(*self.down.shape))
        du = (2.0 * u.float().relu() * dv.float()).to(BF16)
        drows, dup = v4moe.grouped_linear_backward(rows, du, self.up, off, dx=new(T * k, H), dw=new(*self.up.shape))
        dlogits = v4moe.gate_backward(logits, topk, w, dw).to(BF16)
        droute, drouter = v4moe.grouped_linear_backward(h, dlogits, self.router, self.whole, dx=new(T, H), dw=new(*self.router.shape))
        back = drows[pp.long()].view(T, k, H)
        dh = droute
        for i in range(k):
            dh = dh + back[:, i]
        dh = dh.to(BF16)
        dx, _ = v4moe.fp8_linear_backward(x, dh, self.projection, dx=new(T, H), dw=new(H, H))
        base = dx.clone()
        dx, da, db = v4moe.lora_backward(x, dh, self.a, self.b, ids, self.scale, base=dx, dx=dx, da=new(*self.a.shape),
                                         db=new(*self.b.shape))
        grads = [dhead, ddown, dup, drouter, da, db]
        norm = v4moe.clip_grads(grads, 0.1, out=[torch.empty_like(t) for t in grads])
        return dict(y0=y0, h=h, logits=logits, off=off, rows=rows, u=u, v=v, yd=yd, out=out, loss=loss, lse=lse, dout=dout,
                    dhead=dhead, dyd=dyd, dv=dv, ddown=ddown, du=du, drows=drows, dup=dup, dlogits=dlogits, droute=droute,
                    drouter=drouter, dh=dh, base=base, dx=dx, da=da, db=db, norm=norm)

    def inputs(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T = self.T
        targets = torch.randint(0, self.head.shape[0], (T,), generator=g, device=DEV)
        targets[torch.rand(T, generator=g, device=DEV) < 0.3] = -100
        return (torch.randn(T, self.H, generator=g, device=DEV).to(BF16),
                torch.randint(-1, self.L, (T,), generator=g, device=DEV).to(torch.int32), targets)


STEP32 = 2.0 ** -23            # an addition's rounding, twice, as the instructions may cut


def near(got, want, bound):
    """Within the bound and the rounding to got's type; the smallest normal number's steps are below."""
    eps = torch.finfo(got.dtype).eps / 2
    slack = bound + want.abs() * eps * (1 + eps) + 2.0 ** -126
    assert bool(((got.double() - want).abs() <= slack).all()), float(((got.double() - want).abs() / slack).max())


def product(p, q):
    """p q^T in 64 bits and the bound of its sum in fp32."""
    p, q = p.double(), q.double()
    return p @ q.t(), (p.shape[1] + 64) * STEP32 * (p.abs() @ q.abs().t())


@pytest.mark.parametrize("T,H,I,E,k,V,r,L", [(1, 256, 72, 8, 2, 500, 4, 3), (70, 256, 200, 16, 4, 1003, 16, 5),
                                             (600, 512, 264, 32, 4, 4096, 20, 8)])
def test_a_step(T, H, I, E, k, V, r, L):
    """Each operator's result from what it was given there, against its formula in 64 bits."""
    m = Model(T, H, I, E, k, V, r, L)
    x, ids, targets = m.inputs(1)
    s = m.step(x, ids, targets)
    off = s["off"].tolist()
    assert off[0] == 0 and off[-1] == T * k

    near(s["logits"], *product(s["h"], m.router[0]))
    near(s["droute"], *product(s["dlogits"], m.router[0].t()))
    near(s["drouter"][0], *product(s["dlogits"].t(), s["h"].t()))
    for e in range(E):
        i = slice(off[e], off[e + 1])
        near(s["u"][i], *product(s["rows"][i], m.up[e]))
        near(s["yd"][i], *product(s["v"][i], m.down[e]))
        near(s["dv"][i], *product(s["dyd"][i], m.down[e].t()))
        near(s["drows"][i], *product(s["du"][i], m.up[e].t()))
        near(s["ddown"][e], *product(s["dyd"][i].t(), s["v"][i].t()))
        near(s["dup"][e], *product(s["du"][i].t(), s["rows"][i].t()))

    # the loss: a log of a sum of V exponentials, each off by its logit's error (and a few steps of its own)
    z, zb = product(s["out"], m.head)
    has = targets >= 0
    lse = torch.logsumexp(z, 1) * has
    each = zb.amax(1, keepdim=True) + (V + 64) * STEP32 + lse.abs()[:, None] * 4 * STEP32 + 8 * STEP32
    near(s["lse"], lse, each[:, 0])
    near(s["loss"], (lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0]) * has, 3 * each[:, 0])
    p = (z - lse[:, None]).exp()
    hot = torch.zeros_like(p).scatter_(1, targets.clamp(min=0)[:, None], 1.0)
    d = (p - hot) * has[:, None] / T
    # d: p's relative error is that of its exponent's (twice, lse's and z's), then bf16's rounding
    db = (p * 3 * each / T + d.abs() * (2.0 ** -8 + 8 * STEP32)) * has[:, None]
    head = m.head.double()
    near(s["dout"], d @ head, db @ head.abs() + (V + 64) * STEP32 * ((d.abs() + db) @ head.abs()))
    o = s["out"].double().abs()
    near(s["dhead"], d.t() @ s["out"].double(), db.t() @ o + (T + 64) * STEP32 * ((d.abs() + db).t() @ o))

    # the adapters
    def shrink(v, f):
        u, ub = torch.zeros(T, r, dtype=torch.float64, device=DEV), torch.zeros(T, r, dtype=torch.float64, device=DEV)
        for i in range(L):
            at = ids == i
            w, wb = product(v[at], f[i])
            u[at], ub[at] = w * m.scale[i].double(), wb * m.scale[i].double()
        return u, ub + u.abs() * (2.0 ** -16 + 2.0 ** -22)

    def expand(u, ub, f, base):
        w, wb = base.double().clone(), torch.zeros_like(base, dtype=torch.float64)
        for i in range(L):
            at, q = ids == i, f[i].double()
            w[at] += u[at] @ q
            wb[at] = ub[at] @ q.abs() + (2 * r + 64) * STEP32 * ((u[at].abs() + ub[at]) @ q.abs()) + STEP32 * w[at].abs()
        return w, wb

    u, ub = shrink(x, m.a)
    near(s["h"], *expand(u, ub, m.b, s["y0"]))
    du, dub = shrink(s["dh"], m.b)
    near(s["dx"], *expand(du, dub, m.a, s["base"]))
    for got, (w, wb), v in ((s["da"], (du, dub), x), (s["db"], (u, ub), s["dh"])):
        for i in range(L):
            at = ids == i
            q = v[at].double()
            near(got[i], w[at].t() @ q, wb[at].t() @ q.abs() + (2 * int(at.sum()) + 64) * STEP32 * ((w[at].abs() + wb[at]).t() @ q.abs()))

    squares = sum(s[n].double().square().sum() for n in ("dhead", "ddown", "dup", "drouter", "da", "db"))
    assert abs(float(s["norm"]) - float(squares.sqrt())) <= 1e-5 * float(squares.sqrt())


def test_two_captured_steps():
    """Two captured steps of different models, replayed in turn with other inputs and eager work between: the eager
    steps' results, bit for bit."""
    models = [Model(300, 256, 136, 16, 4, 1001, 12, 5), Model(40, 256, 72, 8, 2, 777, 8, 300, seed=3)]
    held, graphs, results = [m.inputs(0) for m in models], [], []
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for m, h in zip(models, held):
            m.step(*h)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    for m, h in zip(models, held):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            results.append(m.step(*h))
        graphs.append(graph)
    for seed in range(4):
        want = []
        for m, h, graph in zip(models, held, graphs):
            new = m.inputs(10 + seed)
            for t, n in zip(h, new):
                t.copy_(n)
            graph.replay()
            want.append(m.step(*new))
        torch.cuda.synchronize()
        for w, got in zip(want, results):
            bad = [n for n in w if not torch.equal(w[n], got[n])]
            assert not bad, (seed, bad)


def test_threads():
    """Products of each tile (whose kernels are set up on first use) by four threads, each on its own stream."""
    g = torch.Generator(device=DEV).manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(BF16)

    E, w, head = 4, randn(4, 264, 328), randn(3001, 328)
    xs = [randn(m, 328) for m in (5, 70, 300, 900, 9000)]
    offs = [torch.tensor([0, m // 5, m // 2, m // 2, m], dtype=torch.int32, device=DEV) for m in (5, 70, 300, 900, 9000)]
    a, b, scale = randn(E, 24, 328), randn(E, 24, 264), torch.rand(E, generator=g, device=DEV)

    def work():
        out = []
        for x, off in zip(xs, offs):
            y = v4moe.grouped_linear(x, w, off)
            out += [y, *v4moe.grouped_linear_backward(x, y, w, off)]
            ids = (torch.arange(len(x), device=DEV) % (E + 1)).to(torch.int32)
            out += [v4moe.lora_add(y, x, a, b, ids, scale), *v4moe.lora_backward(x, y, a, b, ids, scale)]
            if len(x) < 1000:
                t = torch.arange(len(x), device=DEV) * 3
                loss, lse = v4moe.linear_xent(x, head, t)
                out += [loss, lse, *v4moe.linear_xent_backward(x, head, t, lse, torch.ones_like(loss))]
        return out

    results, errors = [None] * 4, []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    results[i] = work()
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # reported by the test itself
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(results))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    want = work()
    for r in results:
        assert all(torch.equal(p.nan_to_num(), q.nan_to_num()) for p, q in zip(r, want))


class Elsewhere(torch.Tensor):
    """A tensor that says it is on GPU 1 (its memory is on GPU 0: what is not refused still runs)."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


def refused(call, args):
    """call(**args) runs; with any one of the arguments elsewhere it does not."""
    call(**args)
    for name in args:
        with pytest.raises(ValueError, match="GPU 1"):
            call(**dict(args, **{name: args[name].as_subclass(Elsewhere)}))


def ones(*shape, t=BF16):
    return torch.ones(*shape, dtype=t, device=DEV)


def test_other_devices():
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    w = ones(2, 8, 16)
    refused(v4moe.grouped_linear, dict(x=ones(4, 16), w=w, offsets=off, out=ones(4, 8)))
    refused(v4moe.grouped_linear_backward, dict(x=ones(4, 16), dy=ones(4, 8), w=w, offsets=off, dx=ones(4, 16), dw=ones(2, 8, 16)))
    head, t, f = ones(9, 16), torch.zeros(4, dtype=torch.int64, device=DEV), ones(4, t=F32)
    refused(v4moe.linear_xent, dict(x=ones(4, 16), w=head, targets=t))
    refused(v4moe.linear_xent_backward, dict(x=ones(4, 16), w=head, targets=t, lse=f, dloss=f, dx=ones(4, 16), dw=ones(9, 16)))
    ids, scale = torch.zeros(4, dtype=torch.int32, device=DEV), ones(2, t=F32)
    ab = dict(a=ones(2, 3, 16), b=ones(2, 3, 8), ids=ids, scale=scale)
    refused(v4moe.lora_add, dict(y=ones(4, 8), x=ones(4, 16), out=ones(4, 8), **ab))
    refused(v4moe.lora_backward, dict(x=ones(4, 16), dy=ones(4, 8), base=ones(4, 16), dx=ones(4, 16), da=ones(2, 3, 16), db=ones(2, 3, 8), **ab))


@pytest.mark.parametrize("M,L", [(300, 1025), (300, 3000), (20000, 7), (9001, 1024)])
def test_adapters_by_the_thousand_and_rows_beyond(M, L):
    """Batches on each side of the rule that lists rows by adapter: a batch's rows equal those of a batch of its own."""
    g = torch.Generator(device=DEV).manual_seed(M + L)
    a, b = (torch.randn(L, 3, n, generator=g, device=DEV).to(BF16) for n in (72, 40))
    x, y = (torch.randn(M, n, generator=g, device=DEV).to(BF16) for n in (72, 40))
    ids = torch.randint(-2, L + 2, (M,), generator=g, device=DEV).to(torch.int32)
    scale = torch.rand(L, generator=g, device=DEV)
    whole = v4moe.lora_add(y, x, a, b, ids, scale)
    dx, da, db = v4moe.lora_backward(x, y, a, b, ids, scale, da=ones(L, 3, 72, t=F32), db=ones(L, 3, 40, t=F32))
    for i in range(0, M, max(M // 7, 1)):
        part = slice(i, i + 5)
        assert torch.equal(whole[part], v4moe.lora_add(y[part], x[part], a, b, ids[part], scale))
        assert torch.equal(dx[part], v4moe.lora_backward(x[part], y[part], a, b, ids[part], scale)[0])
    # the gradients' totals over the adapters: of sums of the rows' products
    at = (ids >= 0) & (ids < L)
    i = ids.long()[at]
    xd, yd, s = x.double()[at], y.double()[at], scale.double()[i]
    du = torch.empty(len(i), 3, dtype=torch.float64, device=DEV)
    u = torch.empty_like(du)
    for c in range(0, len(i), 4096):
        k = slice(c, c + 4096)
        du[k] = (b.double()[i[k]] * yd[k, None]).sum(2) * s[k, None]
        u[k] = (a.double()[i[k]] * xd[k, None]).sum(2) * s[k, None]
    for got, v, w in ((da, du, xd), (db, u, yd)):
        want, mag = (torch.zeros(L, 3, w.shape[1], dtype=torch.float64, device=DEV) for _ in range(2))
        p = v[:, :, None] * w[:, None]
        want.index_add_(0, i, p)
        # u's products: at most 72 of them, of magnitudes whose sum is below |factor| |row|
        n = torch.bincount(i, minlength=L)[:, None, None]
        f, q = (b, yd) if w is xd else (a, xd)
        most = torch.empty(len(i), 3, dtype=torch.float64, device=DEV)
        for c in range(0, len(i), 4096):
            k = slice(c, c + 4096)
            most[k] = (f.double()[i[k]].abs() * q[k, None].abs()).sum(2) * s[k, None]
        mag.index_add_(0, i, most[:, :, None] * w.abs()[:, None])
        near(got, want, mag * ((72 + 64) * STEP32 + 2.0 ** -16 + (2 * n + 64) * STEP32))


def test_nothing_to_do():
    """Empty batches: empty results, gradients of weights of zeros, or left alone where added to."""
    x, w, off = ones(0, 16), ones(3, 8, 16), torch.zeros(4, dtype=torch.int32, device=DEV)
    assert v4moe.grouped_linear(x, w, off).shape == (0, 8)
    dx, dw = v4moe.grouped_linear_backward(x, ones(0, 8), w, off)
    assert dx.shape == (0, 16) and not dw.any()
    held = ones(3, 8, 16)
    v4moe.grouped_linear_backward(x, ones(0, 8), w, off, dw=held, accumulate=True)
    head, t, f = ones(9, 16), torch.zeros(0, dtype=torch.int64, device=DEV), ones(0, t=F32)
    loss, lse = v4moe.linear_xent(x, head, t)
    assert loss.shape == lse.shape == (0,)
    dx, dhead = v4moe.linear_xent_backward(x, head, t, lse, f)
    assert dx.shape == (0, 16) and not dhead.any()
    kept = ones(9, 16)
    v4moe.linear_xent_backward(x, head, t, lse, f, dw=kept, accumulate=True)
    a, b, ids, scale = ones(2, 3, 16), ones(2, 3, 8), torch.zeros(0, dtype=torch.int32, device=DEV), ones(2, t=F32)
    assert v4moe.lora_add(ones(0, 8), x, a, b, ids, scale).shape == (0, 8)
    dx, da, db = v4moe.lora_backward(x, ones(0, 8), a, b, ids, scale)
    assert dx.shape == (0, 16) and not da.any() and not db.any()
    da, db = ones(2, 3, 16), ones(2, 3, 8)
    v4moe.lora_backward(x, ones(0, 8), a, b, ids, scale, da=da, db=db, accumulate=True)
    torch.cuda.synchronize()
    assert all(bool((t == 1).all()) for t in (held, kept, da, db))


def test_beyond_32_bits():
    """Operands of more than 2^32 bytes: the last rows equal those of a small call (a row does not depend on others)."""
    M, K, N = 300007, 8192, 48
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(M, K, dtype=BF16, device=DEV).normal_(generator=g)
    w = torch.randn(2, N, K, generator=g, device=DEV).to(BF16)
    off = torch.tensor([0, M - 100, M], dtype=torch.int32, device=DEV)
    last = slice(M - 100, M)
    y = v4moe.grouped_linear(x, w, off)
    few = torch.tensor([0, 0, 100], dtype=torch.int32, device=DEV)
    assert torch.equal(y[last], v4moe.grouped_linear(x[last].clone(), w, few))
    dx, dw = v4moe.grouped_linear_backward(x, y, w, off)
    small = v4moe.grouped_linear_backward(x[last].clone(), y[last].clone(), w, few)
    assert torch.equal(dx[last], small[0]) and torch.equal(dw[1], small[1][1])
    a, b, scale = w[:, :8].contiguous(), torch.randn(2, 8, N, generator=g, device=DEV).to(BF16), torch.ones(2, device=DEV)
    ids = (torch.arange(M, device=DEV) >= M - 100).to(torch.int32)
    out = v4moe.lora_add(y, x, a, b, ids, scale)
    assert torch.equal(out[last], v4moe.lora_add(y[last], x[last].clone(), a, b, ids[last], scale))
    dx2, da, _ = v4moe.lora_backward(x, y, a, b, ids, scale, dx=dx)
    small = v4moe.lora_backward(x[last].clone(), y[last].clone(), a, b, ids[last], scale)
    assert torch.equal(dx2[last], small[0])
    near(da[1].float(), small[1][1].double(), 2.0 ** -7 * small[1][1].double().abs())        # (the rows' order of waves may differ)
    # the head's rows are the long operand
    t = torch.tensor([0, M - 1, 77, M - 50], device=DEV)
    few = torch.randn(4, K, generator=g, device=DEV).mul_(K ** -0.5).to(BF16)
    loss, lse = v4moe.linear_xent(few, x, t)
    z = few.float() @ x[t].float().t()
    assert bool(((lse - z.diagonal()) - loss).abs().max() <= 2.0 ** -23 * ((K + 64) * (few.float().abs() @ x[t].float().abs().t()).max() + 64 * lse.abs().max()))
    dhead = v4moe.linear_xent_backward(few, x, t, lse, torch.ones(4, device=DEV), dw=dx)[1]
    alone = v4moe.linear_xent_backward(few, x[t].clone(), torch.arange(4, device=DEV), lse, torch.ones(4, device=DEV))[1]
    assert torch.equal(dhead[t], alone)


@pytest.mark.parametrize("T", [1, 3, 4095, 4096, 4097, 8193])
def test_tokens_on_each_side_of_the_ways_to_number_them(T):
    """Losses of a batch equal those of its halves, bit for bit; all against 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x, w = torch.randn(T, 96, generator=g, device=DEV).to(BF16), torch.randn(200, 96, generator=g, device=DEV).mul_(0.1).to(BF16)
    t = torch.randint(-60, 260, (T,), generator=g, device=DEV)
    has = (t >= 0) & (t < 200)
    loss, lse = v4moe.linear_xent(x, w, t)
    assert not loss[~has].any() and not lse[~has].any()
    half = (T + 1) // 2
    for part in (slice(0, half), slice(half, T)):
        a, b = v4moe.linear_xent(x[part], w, t[part].contiguous())
        assert torch.equal(a, loss[part]) and torch.equal(b, lse[part])
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1) * has
    near(lse, want, ((96 + 64) * STEP32 * (x.double().abs() @ w.double().abs().t()).amax(1) + (200 + 64) * STEP32 + want.abs() * 4 * STEP32 + 8 * STEP32))
    dloss = torch.rand(T, generator=g, device=DEV)
    dx, dw = v4moe.linear_xent_backward(x, w, t, lse, dloss, dx=torch.empty(T, 96, device=DEV), dw=torch.empty(200, 96, device=DEV))
    p = (z - want[:, None]).exp()
    hot = torch.zeros_like(p).scatter_(1, t.clamp(0, 199)[:, None], 1.0)
    d = (p - hot) * (has * dloss.double())[:, None]
    each = (96 + 64) * STEP32 * (x.double().abs() @ w.double().abs().t()).amax(1, keepdim=True) + (200 + 64) * STEP32 + 16 * STEP32
    db = (p * 3 * each * dloss.double()[:, None] + d.abs() * (2.0 ** -8 + 8 * STEP32)) * has[:, None]
    wa, xa = w.double().abs(), x.double().abs()
    near(dx, d @ w.double(), db @ wa + (200 + 64) * STEP32 * ((d.abs() + db) @ wa))
    near(dw, d.t() @ x.double(), db.t() @ xa + (T + 64) * STEP32 * ((d.abs() + db).t() @ xa))
