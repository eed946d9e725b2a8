"""The host side of the short calls: it takes every well-formed call, agrees with the Python wrappers bit
for bit, and leaves malformed operands to them, which name the fault."""
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


class NoHost:
    """Stands in for the host module: no call is for it."""

    def __getattr__(self, name):
        return lambda *a: None


def both(ops, monkeypatch, call):
    fast = call()
    with monkeypatch.context() as m:
        m.setattr(ops.L, "host", NoHost)
        slow = call()
    for a, b in zip(fast, slow):
        assert (a is None and b is None) or (torch.equal(a, b) and a.stride() == b.stride() and a.dtype == b.dtype)


def rows(*shape, pad=0):
    t = torch.randn(shape[0], shape[1] + pad, device=DEV).to(BF16)
    return t[:, :shape[1]]


@pytest.mark.parametrize("pad", [0, 16])
@pytest.mark.parametrize("gate,per", [(None, None), (1, None), (6, None), (4, 7), (24, 1)])
@pytest.mark.parametrize("post", [False, True])
def test_norm(ops, monkeypatch, pad, gate, per, post):
    M, D = 24, 264
    X, Y, dH, dZ = (rows(M, D, pad=pad) for _ in range(4))
    how = dict(w_pre=rows(1, D)[0], w_post=rows(1, D)[0] if post else None, gate=rows(gate, D) if gate else None,
               rows_per_gate=per, post_norm=post, alpha=0.5, w_offset=1.0)
    assert ops.L.host().block_norm_fwd(X, Y, how["w_pre"], how["w_post"], how["gate"], per, 0.5, 1e-6, 1.0, True, post)
    both(ops, monkeypatch, lambda: ops.block_norm_fwd(X, Y, **how))
    z, _, r_pre, r_post = ops.block_norm_fwd(X, Y, **how)
    both(ops, monkeypatch, lambda: ops.block_norm_bwd(z, Y, r_pre, r_post, dH, dZ, **how))
    both(ops, monkeypatch, lambda: ops.block_norm_bwd(z, Y, r_pre, r_post, dH, None, need_dx=False, need_dw=False, **how))
    both(ops, monkeypatch, lambda: ops.block_norm_fwd(X, w_pre=how["w_pre"]))


def z(*shape, dtype=BF16, device=DEV):
    return torch.zeros(*shape, dtype=dtype, device=device)


@pytest.mark.parametrize("bad", [
    lambda: dict(Y=z(8, 24)), lambda: dict(Y=z(8, 32, dtype=torch.float32)), lambda: dict(Y=z(32, 8).t()),
    lambda: dict(Y=z(1, 32).expand(8, 32)), lambda: dict(Y=z(8, 32, device="cpu")), lambda: dict(w_pre=z(24)),
    lambda: dict(w_pre=z(64)[::2]), lambda: dict(w_pre=z(32, device="cpu")), lambda: dict(w_post=z(32)),
    lambda: dict(Y=None, post_norm=True), lambda: dict(gate=z(3, 32)), lambda: dict(gate=z(4, 32), rows_per_gate=3),
    lambda: dict(gate=z(4, 32), rows_per_gate=0), lambda: dict(gate=z(8, 64)[:, :32]),
    lambda: dict(X=z(8, 32, dtype=torch.half)), lambda: dict(X=z(8, 2, 16)), lambda: dict(w_pre=z(32), pre_norm=False),
    lambda: dict(X=z(8, 64)[:, ::2]), lambda: dict(eps="a"),
])
def test_norm_refusals_on_the_gpu(ops, bad):
    with pytest.raises((ValueError, TypeError)):
        ops.block_norm_fwd(**{"X": z(8, 32), "Y": z(8, 32), **bad()})


@pytest.mark.parametrize("bad", [
    lambda: dict(dH=None, dXout=None), lambda: dict(dH=z(8, 24)), lambda: dict(dXout=z(8, 32, device="cpu")),
    lambda: dict(r_pre=None), lambda: dict(r_post=None), lambda: dict(r_pre=z(7, dtype=torch.float32)),
    lambda: dict(r_pre=z(8)), lambda: dict(r_post=z(16, dtype=torch.float32)[::2]), lambda: dict(Y=None),
    lambda: dict(w_post=z(24)), lambda: dict(gate=z(3, 32)), lambda: dict(Xout=z(8, 32, dtype=torch.half)),
])
def test_norm_backward_refusals_on_the_gpu(ops, bad):
    f = torch.float32
    a = dict(Xout=z(8, 32), Y=z(8, 32), r_pre=z(8, dtype=f), r_post=z(8, dtype=f), dH=z(8, 32), dXout=z(8, 32),
             post_norm=True)
    with pytest.raises((ValueError, TypeError)):
        ops.block_norm_bwd(**{**a, **bad()})


def test_errors_of_the_library_are_raised(ops):
    with pytest.raises(ops.L.LoraError) as e:
        ops.block_norm_fwd(torch.zeros(4, 12, device=DEV), torch.zeros(4, 12, device=DEV))
    assert e.value.status == 2          # D a multiple of 8
    with pytest.raises(ops.L.LoraError) as e:
        ops.block_norm_fwd(torch.zeros(4, 16, device=DEV), torch.zeros(4, 16, device=DEV), eps=0.0)
    assert e.value.status == 1
    flat = torch.zeros(8 * 16 + 4, device=DEV, dtype=BF16)
    with pytest.raises(ops.L.LoraError) as e:
        ops.block_norm_fwd(flat[4:].view(8, 16), flat[:128].view(8, 16))
    assert e.value.status == 3          # not at 16 bytes


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary(ops, monkeypatch, layout):
    plan = ops.rotary_plan(32, layout=layout, scaling="linear", factor=2.0, device=DEV)
    X = torch.randn(9, 6 * 48, device=DEV).to(BF16)[:, :4 * 48].view(9, 4, 48)
    for pos in (torch.arange(9, device=DEV), torch.arange(9, device=DEV, dtype=torch.int32)):
        assert ops.L.host().rotary(False, X, pos, plan.freq, 32, 1.0, plan.layout, None) is not None
        both(ops, monkeypatch, lambda: [ops.rotary_fwd(X, pos, plan), ops.rotary_bwd(X, pos, plan)])
        both(ops, monkeypatch, lambda: [ops.rotary_fwd(X, pos, plan, out=torch.zeros(4, 9, 48, device=DEV, dtype=BF16)
                                                       .transpose(0, 1))])
    X2 = X.clone()
    assert ops.rotary_fwd(X2, pos, plan, out=X2) is X2
    for bad in (dict(X=X.float().half()), dict(pos=pos.float()), dict(pos=pos[:4]), dict(pos=pos.cpu()), dict(X=X[..., :16]),
                dict(out=torch.zeros(9, 4, 48, device=DEV)), dict(out=torch.zeros(9, 4, 40, device=DEV, dtype=BF16)),
                dict(X=X.transpose(1, 2)), dict(X=X[0])):
        a = {"X": X, "pos": pos, "out": None, **bad}
        with pytest.raises((ValueError, TypeError)):
            ops.rotary_fwd(a["X"], a["pos"], plan, out=a["out"])


def test_gradient_addresses(ops):
    import struct
    p = [torch.zeros(3, 5, device=DEV), torch.zeros(8, device=DEV, dtype=BF16)]
    g = [torch.zeros(3, 5, device=DEV), torch.zeros(8, device=DEV, dtype=BF16)]
    at = ops.L.host().pointers
    assert struct.unpack("2Q", at(g, p)) == (g[0].data_ptr(), g[1].data_ptr())
    assert struct.unpack("2Q", at((None, g[1]), p)) == (0, g[1].data_ptr())
    for bad in (g[:1], [g[0].t(), g[1]], [g[0].double(), g[1]], [g[0].cpu(), g[1]], [1, g[1]],
                [torch.zeros(5, 3, device=DEV).t(), g[1]]):
        assert at(bad, p) is None


def test_norms_of_consecutive_steps_are_their_own(ops):
    from dora_adapter_linear_gb300 import optim
    p = [torch.zeros(40, 8, device="cuda")]
    opt = optim.AdamW(p)
    norms = [opt.step([torch.full_like(p[0], float(i))], max_norm=1.0) for i in range(1, 6)]
    assert all(n.shape == () and n.dtype is torch.float32 and n.is_cuda for n in norms)
    want = torch.arange(1, 6) * 320 ** 0.5
    assert torch.allclose(torch.stack(norms).cpu(), want, rtol=1e-6)
    copy = norms[2].clone()
    assert copy.item() == norms[2].item() and norms[2].view(1).sum().item() == copy.item()
