"""Clipping by groups against its fp64 reference, element by element."""
import numpy as np
import pytest
import torch

from dora_adapter_linear_gb300 import optim
from multi_cases import f64
from oracle import multi_oracle as O

pytestmark = pytest.mark.gpu


def check(grads, max_norm, groups=None):
    """A call on clones of `grads` against the reference.  A unit's squares are summed over threads of at most 72
    elements, 32 lanes and 8 warps: 72 + 5 + 5 roundings of 2^-24 at most (half as much in the root), and a few
    for the root, the factor and the product."""
    grads = [None if g is None else g.cuda() for g in grads]
    keep = [None if g is None else g.clone() for g in grads]
    norms = optim.clip_grads(grads, max_norm, groups)
    if isinstance(groups, int):
        count, entries = groups, [(f64(k[j]), j, f64(g[j]), g.dtype) for k, g in zip(keep, grads) if g is not None
                                  for j in range(groups)]
    else:
        each = [0] * len(grads) if groups is None else groups
        count, entries = max(each) + 1, [(f64(k), j, f64(g), g.dtype) for k, g, j in zip(keep, grads, each) if g is not None]
    with np.errstate(all="ignore"):
        want, clipped = O.clip([e[0] for e in entries], max_norm, [e[1] for e in entries], count)
    norms = f64(norms)
    assert norms.shape == (count,)
    off = 48 * 2.0 ** -24
    fine = np.isfinite(want)
    assert (np.isfinite(norms) == fine).all()
    assert (abs(norms - want)[fine] <= off * want[fine]).all()
    for (before, j, got, dtype), ref in zip(entries, clipped):
        h = torch.finfo(dtype).eps / 2 + off + 8 * 2.0 ** -24
        tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps        # below the normal numbers: one step
        assert (abs(got - ref) <= abs(ref) * h + (0 if max_norm is None else tiny)).all()
        if max_norm is None or (fine[j] and want[j] * (1 + off) + 1e-6 < max_norm):
            assert (got == before).all() or not np.isfinite(before).all()
    return norms


def normal(*shape, dtype=torch.float32, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape))) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 255, 2048, 2049, 16383, 16384, 16385, 40000, 3 * 16384])
def test_one_group(n, dtype):
    for scale in (1e-3, 3.0):
        check([normal(n, dtype=dtype, scale=scale), normal(5, 3, dtype=torch.float32, scale=scale)], 0.5)


@pytest.mark.parametrize("shape", [(8, 512), (3, 7), (129, 127), (1,), (0, 4), (5,)])
@pytest.mark.parametrize("G", [1, 2, 5, 70])
def test_stacks(G, shape):
    """Groups of odd sizes begin anywhere, also where wide accesses cannot."""
    scale = torch.logspace(-4, 2, G).view(-1, *[1] * len(shape))
    stacks = [normal(G, *shape, dtype=dt, seed=k) * scale.to(dt) for k, dt in enumerate((torch.float32, torch.bfloat16))]
    check(stacks + [normal(G, 33)], 1.0, G)


@pytest.mark.parametrize("tensors", [3, 64, 65, 700, 1400])
def test_lists_of_any_length(tensors):
    rng = np.random.default_rng(tensors)
    groups = rng.integers(0, 9, tensors).tolist()
    groups[0] = 11                                       # some groups have no tensor
    grads = [normal(int(rng.integers(0, 3000)), dtype=(torch.float32, torch.bfloat16)[k % 2], seed=k, scale=0.01 * 4.0 ** groups[k])
             for k in range(tensors)]
    norms = check(grads, 2.0, groups)
    assert norms[10] == 0
    check([None if k % 3 == 1 else g for k, g in enumerate(grads)], 2.0, groups)


def test_large_stacks():
    check([normal(3, 700, 1024, dtype=torch.bfloat16), normal(3, 1024, 96, dtype=torch.bfloat16, scale=1e-3)] * 1, 1.0, 3)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 2.0 ** 80])
def test_a_group_that_is_not_finite_becomes_zeros(bad):
    for max_norm in (1.0, float("inf")):
        g = [normal(4, 8, 600).cuda(), normal(4, 50, 8, dtype=torch.bfloat16).cuda()]
        g[0][2, 3, 599] = bad
        keep = [t.clone() for t in g]
        norms = optim.clip_grads(g, max_norm, 4)
        assert norms.isfinite().tolist() == [True, True, False, True]
        for t, k in zip(g, keep):
            assert not t[2].any()
            if max_norm == 1.0:
                assert (t[[0, 1, 3]].abs() < k[[0, 1, 3]].abs()).float().mean() > 0.99
            else:
                assert torch.equal(t[[0, 1, 3]], k[[0, 1, 3]])


def test_norms_alone_and_zeros():
    g = [normal(2, 300).cuda()]
    keep, version = g[0].clone(), g[0]._version
    norms = optim.clip_grads(g, None, 2)
    assert torch.equal(g[0], keep) and g[0]._version == version
    assert torch.allclose(norms, keep.norm(dim=1), rtol=1e-6)
    optim.clip_grads(g, 1.0, 2)
    assert g[0]._version > version
    z = [torch.zeros(40, device="cuda")]
    assert float(optim.clip_grads(z, 1.0)) == 0 and not z[0].any()
    assert float(optim.clip_grads([torch.zeros(0, device="cuda")], 1.0)) == 0
    check([torch.full((64,), 2.0 ** -70)], 1.0)          # far below one
    check([torch.full((64,), 2.0 ** 55)], 1.0)


def test_same_bits_again():
    g = [normal(6, 333, 70).cuda() for _ in range(3)]
    first = optim.clip_grads(g, None, 6)
    for _ in range(3):
        assert torch.equal(first, optim.clip_grads(g, None, 6))


def test_captured():
    g = [normal(3, 500, seed=k).cuda() for k in range(2)]
    new = [[normal(3, 500, seed=10 * k + j, scale=10.0 ** k).cuda() for j in range(2)] for k in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norms = optim.clip_grads(g, 1.0, [0, 1])
        norms2 = optim.clip_grads(g, 0.5, 3)
    for step in new:
        for t, v in zip(g, step):
            t.copy_(v)
        h = [v.clone() for v in step]
        a, b = optim.clip_grads(h, 1.0, [0, 1]), optim.clip_grads(h, 0.5, 3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norms, a) and torch.equal(norms2, b)
        assert all(torch.equal(t, v) for t, v in zip(g, h))


def test_another_stream():
    side = torch.cuda.Stream()
    g, h = [normal(3, 5000).cuda()], [normal(3, 5000).cuda()]
    a = optim.clip_grads(h, 1.0, 3)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = optim.clip_grads(g, 1.0, 3)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(g[0], h[0])


def test_a_tensor_past_32_bits():
    """2^31 + 11 elements: the last ones count and are scaled."""
    n = 2 ** 31 + 11
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:], g[0] = 3.0, 4.0
    norm = optim.clip_grads([g], 1.0)
    assert abs(float(norm) - 43 ** 0.5) < 1e-5
    want = (torch.tensor([3.0, 4.0]) / (43 ** 0.5 + 1e-6)).bfloat16().tolist()
    assert g[-3:].tolist() == want[:1] * 3 and float(g[0]) == want[1] and not g[1:-3].any()


def test_shared_memory_is_refused():
    buf = torch.ones(100, device="cuda")
    for grads in ([buf, buf], [buf[:60], buf[50:]], [buf[60:], buf[:61]], [buf[90:], buf[:10], buf[5:20]]):
        with pytest.raises(ValueError, match="share memory"):
            optim.clip_grads(grads, 1.0)
    assert (buf == 1).all()
    optim.clip_grads([buf[50:], buf[:50]], 1.0)


def test_what_it_does_not_take_is_named():
    g = torch.ones(4, 6, device="cuda")
    for grads, groups, what in (([g.t()], None, "contiguous"), ([g.double()], None, "fp32 or bf16"), ([g], 3, "stack of 3"),
                                ([g, 1.0], None, "tensor or None"), ([g], [-1], "1 to 65535"), ([g, g[0]], [1, -1], "not in 0 to 1"),
                                ([g, torch.ones(3)], None, "CUDA")):
        with pytest.raises(ValueError, match=what):
            optim.clip_grads(grads, 1.0, groups)
    assert (g == 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_ends_of_a_norms_range(dtype):
    """A norm below 2^64 counts as finite.  Values whose mean square is at least 2^-126 give a norm as exact as any:
    a square below 2^-126 is off by half of 2^-149, which is 2^-24 of that mean.  A factor below 2^-126 is off by half
    of 2^-149 itself, and so an element by its own size times 2^-150."""
    off = 48 * 2.0 ** -24
    for g in ([torch.full((16,), 1.3 * 2.0 ** 61).to(dtype)],                    # 1.3 * 2^63
              [torch.full((3 * 16384,), 1.01 * 2.0 ** 56).to(dtype)],            # sums of several units: 1.75 * 2^63
              [torch.full((64,), 1.3 * 2.0 ** -63).to(dtype)],
              [normal(5000, dtype=dtype, scale=1.5 * 2.0 ** -63)],
              [torch.cat((torch.full((999,), 1.7 * 2.0 ** -72), torch.full((1,), 1.9 * 2.0 ** -58))).to(dtype)]):
        for max_norm in (None, 2.0 ** -70, 1.0):
            x = [t.cuda() for t in g]
            norms = f64(optim.clip_grads(x, max_norm))
            want, clipped = O.clip([f64(t) for t in g], max_norm, [0], 1)
            assert abs(norms[0] - want[0]) <= off * want[0]
            h = torch.finfo(dtype).eps / 2 + off + 8 * 2.0 ** -24
            most = abs(clipped[0]) * h + abs(f64(g[0])) * 2.0 ** -150 * (1 + h) + 2.0 ** (-150 if dtype == torch.float32 else -134)
            assert (abs(f64(x[0]) - clipped[0]) <= (0 if max_norm is None else most)).all()
    g = [torch.full((16,), 1.01 * 2.0 ** 62, device="cuda").to(dtype)]           # 1.01 * 2^64
    assert optim.clip_grads(g, 1.0).isinf().all() and not g[0].any()
