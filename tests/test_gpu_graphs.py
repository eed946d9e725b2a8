"""Captured graphs of calls that take a workspace: what runs after the capture neither disturbs a replay nor is
disturbed by it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from dora_adapter_linear_gb300.build import build
    build()
    from dora_adapter_linear_gb300 import ops as _ops
    return _ops


def backward(ops, M, D, seed):
    """A call of block_norm_bwd whose row sums go through partials in the workspace."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)  # noqa: E731
    X, Y, dH, dX, w, u, g = n(M, D), n(M, D), n(M, D), n(M, D), n(D), n(D), n(2, D)
    how = dict(w_pre=w, w_post=u, gate=g, rows_per_gate=-(-M // 2), post_norm=True)
    z, _, r_pre, r_post = ops.block_norm_fwd(X, Y, **how)
    return lambda: ops.block_norm_bwd(z, Y, r_pre, r_post, dH, dX, **how)


def captured(call, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = call()
    return graph, out


@pytest.mark.parametrize("M,D", [(601, 512), (600, 1032), (40, 20488)])     # the three backwards
@pytest.mark.parametrize("warm", [True, False])
def test_a_replay_keeps_to_its_own_memory(ops, M, D, warm):
    side = torch.cuda.Stream()
    call, larger = backward(ops, M, D, 1), backward(ops, 5000, 4096, 2)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(side):
            call()
        side.synchronize()
    graph, got = captured(call, side)
    with torch.cuda.stream(side):
        larger()                            # asks for more than the workspace of the capture
        side.synchronize()
        others = [torch.full((1 << n,), 7.0, device=DEV) for n in range(8, 23) for _ in range(3)]
        ref = [t.clone() for t in larger()]
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
        again = larger()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(again, ref))
    assert all(bool((t == 7.0).all()) for t in others)


def test_graphs_captured_on_one_stream_replay_on_two(ops):
    side, streams = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    calls = [backward(ops, 3000, 4096, seed) for seed in (3, 4)]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    graphs = [captured(call, side) for call in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, got), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_several_calls_of_one_graph(ops):
    """Calls that follow one another in a graph share its workspace, which grows within the capture."""
    side = torch.cuda.Stream()
    calls = [backward(ops, M, D, M) for M, D in ((100, 1024), (700, 4096), (300, 2048))]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    graph, got = captured(lambda: [call() for call in calls], side)
    with torch.cuda.stream(side):
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_capture_numbers(ops):
    L = ops.L
    side = torch.cuda.Stream()
    numbers = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        x = torch.zeros(8, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            numbers.append(L.capture_id(side.cuda_stream))
            x.add_(1)
            numbers.append(L.capture_id(side.cuda_stream))
    assert numbers[0] == numbers[1] != numbers[2] == numbers[3] and 0 not in numbers
    assert L.capture_id(0) == 0 and L.capture_id(L.current_stream()) == 0
    with torch.cuda.stream(side):
        assert L.capture_id(side.cuda_stream) == 0
