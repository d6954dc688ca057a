"""FP8Weights: quantised and updated in place, on the stream that is given.  Products are bitwise
reproducible, so those on a side stream are compared exactly with those of fresh objects."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def weights(N, K, seed):
    return torch.randn(1, N, K, generator=ref.gen(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("as_handle", [False, True])
def test_update_on_a_side_stream(moe, as_handle):
    M, N, K = 300, 512, 1024
    W1, W2 = weights(N, K, 1), weights(N, K, 2)
    a, d = (torch.randn(M, c, generator=ref.gen(c)).to(torch.bfloat16).cuda() for c in (K, N))
    qa, sa = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(M, K // 128, device="cuda")
    qd, sd = torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.empty(M, N // 128, device="cuda")
    moe.moe_quantize_fp8_act(a, M, K, qa, sa)
    moe.moe_quantize_fp8_act(d, M, N, qd, sd)
    want = []
    for W in (W1, W2):
        w = moe.FP8Weights(W, training=True)
        want += [w.product(qa, sa), w.input_gradient(qd, sd)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = side.cuda_stream if as_handle else side
    w = moe.FP8Weights(W1, training=True, stream=stream)
    at = [t.data_ptr() for t in (w.q, w.s, w.qt, w.st)]
    got = [w.product(qa, sa, stream=stream), w.input_gradient(qd, sd, stream=stream)]
    w.update(W2, stream=stream)
    got += [w.product(qa, sa, stream=stream), w.input_gradient(qd, sd, stream=stream)]
    assert at == [t.data_ptr() for t in (w.q, w.s, w.qt, w.st)]
    assert w.status(stream) == moe.MOE_OK
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert torch.equal(g, v)


def test_graph_sees_updated_weights(moe):
    """A captured product reads the weights that were updated after its capture."""
    M, N, K = 16, 256, 256
    W1, W2 = weights(N, K, 3), weights(N, K, 4)
    q, s = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(M, K // 128, device="cuda")
    w = moe.FP8Weights(W1)
    out = w.product(q, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.product(q, s, out=out)
    w.update(W2)
    graph.replay()
    assert torch.equal(out, moe.FP8Weights(W2).product(q, s))


def test_update_refuses_other_weights(moe):
    w = moe.FP8Weights(weights(256, 128, 5))
    with pytest.raises(ValueError):
        w.update(weights(128, 128, 5))
    with pytest.raises(ValueError):
        w.update(weights(128, 256, 5).transpose(1, 2))
    with pytest.raises(TypeError):
        w.update(weights(256, 128, 5).float())
