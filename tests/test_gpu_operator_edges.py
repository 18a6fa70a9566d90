"""Edges of the 16-bit operators on the GPU that their main suites do not reach:
what a kernel leaves under way when it ends, flags of rows that do not exist,
far tails of the activations, calls beside the library's other kernels."""
import numpy as np
import pytest

import operator_ref as R
from test_gpu_dense import check, milo, n64, rand      # noqa: F401 (milo is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_pairs_of_ctas_end_with_nothing_under_way(milo):
    """Pairs of CTAs (both products of a gradient, a product alone; fewer slices
    than stages, and more) whose SMs go at once to other kernels with barriers
    in the same places: every commit's arrival has landed before its CTA left,
    so no later kernel's barrier gets one too many."""
    rng = np.random.default_rng(21)
    pairs = []
    for M, N, K in ((2600, 2312, 72), (2600, 2312, 648), (4100, 1032, 136)):
        x, W, dy = rand(rng, (M, K), "bf16"), rand(rng, (N, K), "bf16", K ** -0.5), rand(rng, (M, N), "bf16")
        pairs.append((x, W, dy, milo.milo_dense_linear(x, W), milo.milo_dense_linear_backward(dy, x, W)))
    x, W = rand(rng, (300, 2048), "bf16"), rand(rng, (64, 2048), "bf16")          # a split sum
    x1, W1 = rand(rng, (40, 512), "bf16"), rand(rng, (2048, 512), "bf16")         # tokens as columns
    y, y1 = milo.milo_dense_linear(x, W), milo.milo_dense_linear(x1, W1)
    st = milo.new_status()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            a, b, dy, want, g = pairs[i % 3]
            got.append((milo.milo_dense_linear(a, b, dev_status=st), want))
            got.append((milo.milo_dense_linear(x, W, dev_status=st), y))
            g2 = milo.milo_dense_linear_backward(dy, a, b, dev_status=st)
            got += [(g2[n], g[n]) for n in g]
            got.append((milo.milo_dense_linear(x1, W1, dev_status=st), y1))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(a, b) for a, b in got)
