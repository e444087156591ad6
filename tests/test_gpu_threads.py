"""The operators next to the layer called by several host threads at once, each on its own stream."""
import threading

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_threads():
    """Products of each tile (whose kernels are set up on first use), a routing and a clipping: the results of one thread."""
    g = torch.Generator(device=DEV).manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    w = v4moe.fp8_weights(randn(512, 384))
    xs = [randn(m, 384).to(torch.bfloat16) for m in (1, 20, 100, 600, 3000, 20000)]
    z, grads = randn(5000, 64), [randn(10000), randn(77)]

    def work():
        return [v4moe.fp8_linear(x, w) for x in xs] + list(v4moe.gate(z, 6)) + \
            list(v4moe.fp8_linear_backward(xs[4], xs[4][:, :256].repeat(1, 2), w)) + \
            [v4moe.clip_grads(grads, 0.5, out=[torch.empty_like(t) for t in grads])]

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
        assert all(torch.equal(a, b) for a, b in zip(r, want))
