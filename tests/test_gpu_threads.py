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


def first_call(f, threads=2):
    """What f raises as the first call of a new thread, in several threads one after another: later ones get an
    earlier one's number and find its workspace, so that nothing but f comes before f."""
    said = []

    def run():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            said.append(e)

    for _ in range(threads):
        t = threading.Thread(target=run)
        t.start()
        t.join()
    torch.cuda.synchronize()
    return said


@pytest.mark.parametrize("M", [3, 40, 300])
def test_many_adapters_as_a_threads_first_call(ops, M):
    """A new thread has no CUDA context until a call makes one current."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)  # noqa: E731
    X, W0, A, B, dY = n(M, 136), n(264, 136), n(3, 16, 136), n(3, 264, 16), n(M, 264)
    plan = ops.adapter_plan(torch.arange(M, device=DEV) % 3, 3)
    Y, Z = ops.lora_multi_fwd(X, W0, A, B, 0.5, plan)
    grads = ops.lora_multi_bwd(X, W0, A, B, Z, dY, 0.5, plan)
    got = {}
    assert first_call(lambda: got.update(f=ops.lora_multi_fwd(X, W0, A, B, 0.5, plan)), 4) == []
    assert torch.equal(got["f"][0], Y) and torch.equal(got["f"][1], Z)
    assert first_call(lambda: got.update(b=ops.lora_multi_bwd(X, W0, A, B, Z, dY, 0.5, plan)), 4) == []
    assert all(torch.equal(a, b) for a, b in zip(got["b"][:3], grads[:3]))


def test_entry_points_as_a_threads_first_call(ops):
    """With everything in hand before, workspaces too: nothing but the entry point runs in the thread."""
    L = ops.L
    M, d, o, r = 1024, 512, 384, 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(BF16)  # noqa: E731
    X, W0, A, B, dY = n(M, d), n(o, d), n(r, d), n(o, r), n(M, o)
    ws, stream = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV), int(torch.cuda.current_stream().cuda_stream)
    Y, Z, dX, dA, dB = (torch.empty_like(t) for t in (dY, n(M, r), X, A, B))
    sh = L.shape(M, d, o, r, L.dtype_code(X))
    A3, B3, plan = torch.stack((A, A, A)), torch.stack((B, B, B)), ops.adapter_plan(torch.zeros(M, dtype=torch.int64, device=DEV), 3)
    ms, few = L.LoraMultiShape(M, d, o, r, 3, L.LORA_BF16), L.LoraMultiShape(20, d, o, r, 3, L.LORA_BF16)
    plan20 = ops.adapter_plan(torch.zeros(20, dtype=torch.int64, device=DEV), 3)
    dA3, dB3 = torch.empty_like(A3), torch.empty_like(B3)
    Xq, Wq = (torch.randint(-127, 128, t.shape, generator=gen, device=DEV, dtype=torch.int8) for t in (X, W0))
    sx, sw = torch.rand(M, device=DEV), torch.rand(o, device=DEV)
    calls = {
        "lora_linear_fwd": lambda: L.lora_linear_fwd(sh, X, W0, A, B, None, 0.5, Y, Z, ws, stream),
        "lora_linear_bwd": lambda: L.lora_linear_bwd(sh, X, W0, A, B, Z, dY, 0.5, dX, dA, dB, None, ws, stream),
        "w8a8_lora_fwd": lambda: L.w8a8_lora_fwd(M, d, o, r, Xq, sx, Wq, sw, Z, B, 0.5, None, Y, None, ws, stream),
        "lora_multi_fwd": lambda: L.lora_multi_fwd(ms, X, W0, A3, B3, None, 0.5, plan.buffer, Y, Z, ws, stream),
        "few rows": lambda: L.lora_multi_fwd(few, X, W0, A3, B3, None, 0.5, plan20.buffer, Y, Z, ws, stream),
        "lora_multi_bwd": lambda: L.lora_multi_bwd(ms, X, W0, A3, B3, Z, dY, 0.5, plan.buffer, dX, dA3, dB3, None, ws, stream),
    }
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    assert {k: first_call(f, 1) for k, f in calls.items()} == {k: [] for k in calls}
