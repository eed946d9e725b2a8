"""The native calls beside other Python threads."""
import ctypes
import threading

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


def norm_case(M, D, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)  # noqa: E731
    return dict(X=n(M, D), Y=n(M, D), dH=n(M, D), dX=n(M, D), w=n(D), g=n(2, D))


def backward(ops, c):
    how = dict(w_pre=c["w"], w_post=c["w"], gate=c["g"], rows_per_gate=-(-c["X"].shape[0] // 2), post_norm=True)
    z, h, r_pre, r_post = ops.block_norm_fwd(c["X"], c["Y"], **how)
    return (z, h) + ops.block_norm_bwd(z, c["Y"], r_pre, r_post, c["dH"], c["dX"], **how)


def test_the_interpreter_is_free_during_the_c_call(ops):
    """The entry points are replaced by PyGILState_Check: it answers 1, an error status, if this thread
    holds the interpreter's lock."""
    host, lib = ops.L.host(), ops.L._lib()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    c = norm_case(6, 64, 1)
    r = torch.ones(6, device=DEV)
    plan, pos = ops.rotary_plan(32, device=DEV), torch.arange(6, device=DEV)
    heads = torch.zeros(6, 2, 32, device=DEV)
    try:
        host.bind(*[address(ctypes.pythonapi.PyGILState_Check)] * 4)
        ops.block_norm_fwd(c["X"], c["Y"])
        ops.block_norm_bwd(c["X"], c["Y"], r, None, c["dH"], c["dX"])
        ops.rotary_fwd(heads, pos, plan)
        ops.rotary_bwd(heads, pos, plan, out=heads)
    finally:
        host.bind(*[address(getattr(lib, n)) for n in ("block_norm_fwd", "block_norm_bwd", "rotary_fwd", "rotary_bwd")])


def test_threads_on_one_stream(ops):
    """The calls' launches come in any order; each call has to find its own partial sums."""
    cases = [norm_case(M, D, D) for M, D in ((900, 512), (900, 4096), (901, 1536), (64, 20488))]
    want = [backward(ops, c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        for _ in range(50):
            got = backward(ops, cases[i])
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
