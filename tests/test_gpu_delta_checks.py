"""The bounds-checked debug build on the edge shapes of the delta-rule and state-pool kernels, and
the failure path of the chunked ones.

In the debug build a failed index check skips the access and records RWKV_ERR_BOUNDS in the
device status word; these calls have to leave it at 0 and give the values of the 64-bit
reference (tolerances: those of test_gpu_delta.py, derived there).
"""
import os
import threading

import pytest
import torch

import delta_ref as ref
from test_gpu_delta import BF16, F32, SCALE, _args, _check_backward, _check_forward, _cu
from wkv_recurrence_02_b200 import build, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_lib():
    if not os.path.exists(build.LIB_DEBUG):
        build.build(debug_bounds=True)
    with ops.using_library(build.LIB_DEBUG) as lib:
        assert lib.rwkv_debug_bounds() == 1
        assert ops.device_status() == 0
        yield lib


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hk,H", [(2, 1, 1, 2), (3, 7, 2, 2), (1, 27, 1, 3), (2, 28, 2, 2), (2, 65, 1, 2), (1, 300, 2, 2)])
def test_debug_forward(debug_lib, dtype, B, T, Hk, H):
    _check_forward(ref.inputs(B, T, Hk, H, dtype, seed=T), dtype=dtype)


PACKED = [([5, 0, 1, 64, 3], 0, 0), ([65, 130, 0], 2, 3), ([1, 1, 1, 1], 0, 4), ([0, 63, 129, 0, 1], 1, 70)]


def _packed(lens, lead, tail, dtype):
    x = ref.inputs(1, lead + sum(lens) + tail, 1, 2, dtype, seed=len(lens), nseq=len(lens))
    spans = ref.spans_of(lens, lead)
    return x, spans, [a for a, _ in spans] + [lead + sum(lens)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,lead,tail", PACKED)
def test_debug_forward_packed(debug_lib, dtype, lens, lead, tail):
    x, spans, offsets = _packed(lens, lead, tail, dtype)
    _check_forward(x, spans, offsets, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hk,H", [(2, 1, 1, 2), (1, 9, 2, 2), (2, 10, 1, 2), (1, 65, 2, 2), (2, 200, 1, 3)])
def test_debug_backward(debug_lib, dtype, B, T, Hk, H):
    _check_backward(ref.inputs(B, T, Hk, H, dtype, seed=T), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,lead,tail", PACKED[:2] + PACKED[3:])
def test_debug_backward_packed(debug_lib, dtype, lens, lead, tail):
    x, spans, offsets = _packed(lens, lead, tail, dtype)
    _check_backward(x, dtype, spans, offsets)


@pytest.mark.parametrize("shape,dim", [((6, 4), 0), ((3, 33, 5, 64), 1), ((40, 12004), 0)])
def test_debug_pool(debug_lib, shape, dim):
    gen = torch.Generator().manual_seed(sum(shape))
    pool, P = torch.randn(*shape, generator=gen), shape[dim]
    src = torch.randint(-1, P, (P,), generator=gen).tolist()
    dst = torch.randint(-1, P, (P,), generator=gen).tolist()
    got = pool.cuda()
    ops.state_copy(got, *(torch.tensor(i, dtype=torch.int32, device="cuda") for i in (src, dst)), slot_dim=dim)
    assert torch.equal(got.cpu(), ref.copied(pool, src, dst, dim))
    live = torch.rand(P, generator=gen) < 0.6
    got = pool.cuda()
    new, count = ops.state_compact(got, live.cuda(), slot_dim=dim)
    n = int(live.sum())
    assert ops.device_status() == 0 and int(count) == n
    assert torch.equal(got.cpu().narrow(dim, 0, n), pool.index_select(dim, live.nonzero()[:, 0]))


def test_a_wait_that_runs_out_is_reported_and_the_context_survives():
    """The wait is made to run out on the host's word: a barrier that nothing signals."""
    lib = ops.load()
    x = ref.inputs(1, 200, 2, 2, BF16, seed=3)
    d = _cu(x)
    for call in (lambda: ops.delta_forward(*_args(d), s0=d["s0"]), lambda: ops.delta_backward(*_args(d), d["do"])):
        assert ops.device_status() == 0
        prev = lib.rwkv_debug_inject_timeout(1)
        try:
            call()
            status = ops.device_status()
        finally:
            lib.rwkv_debug_inject_timeout(prev)
        assert status == -6
        _check_forward(x)
        _check_backward(x, BF16)


@pytest.mark.parametrize("Hk,H,lens", [(2, 2, None), (1, 3, None), (2, 2, [70, 0, 1, 129])])
def test_every_kernel_whose_wait_runs_out_writes_nothing(Hk, H, lens):
    """T's kernel, both walks and the gradient kernel each: no output, nothing in the workspace but the
    sums of the value heads' shares; the next call is as if nothing had been."""
    lib, p = ops.load(), ops._ptr
    T, n = (200, 1) if lens is None else (sum(lens), len(lens))
    x = _cu(ref.inputs(1, T, Hk, H, BF16, seed=4, nseq=n))
    off = None if lens is None else torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    bytes_f = ops.delta_forward_workspace_bytes(1, T, Hk, H, nseq=n, packed=lens is not None)
    bytes_b = ops.delta_backward_workspace_bytes(1, T, Hk, H, nseq=n, packed=lens is not None)
    shares = 0 if H == Hk else 2 * T * H * 64 * 4

    def run():
        ops._use_current_stream(lib, x["q"].device)
        ws = [torch.full((b,), 171, dtype=torch.uint8, device="cuda") for b in (bytes_f, bytes_b)]
        out = {m: torch.full_like(x[i], 5.0) for m, i in
               (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta"), ("sT", "s0"), ("ds0", "s0"))}
        a = [1, T, Hk, H, 64, *[p(t) for t in _args(x)], SCALE, n, p(off)]
        ops._check(lib.rwkv_delta_forward_bf16(*a, 0, None, p(x["s0"]), p(out["o"]), p(out["sT"]), p(ws[0]), bytes_f))
        ops._check(lib.rwkv_delta_backward_bf16(*a, p(x["s0"]), p(x["do"]), p(x["dsT"]),
                                                *[p(out[m]) for m in ("dq", "dk", "dv", "dg", "dbeta", "ds0")], p(ws[1]),
                                                bytes_b))
        return out, ws

    want, _ = run()
    assert ops.device_status() == 0
    prev = lib.rwkv_debug_inject_timeout(1)
    try:
        out, ws = run()
        status = ops.device_status()
    finally:
        lib.rwkv_debug_inject_timeout(prev)
    assert status == -6
    assert (ws[0] == 171).all() and (ws[1][:bytes_b - shares] == 171).all()
    for m, t in out.items():
        if H == Hk or m not in ("dq", "dk"):  # those are sums of shares, which nothing wrote
            assert (t == 5.0).all(), m
    again, _ = run()
    assert ops.device_status() == 0
    for m in want:
        assert torch.equal(want[m], again[m]), m


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 130, 37, 74), (1, 130, 25, 75), (3, 65, 32, 32), (5, 29, 20, 40), (2, 12, 75, 75)])
def test_many_heads(dtype, B, T, Hk, H):
    """Both sides of the choices by the number of (sequence, head) pairs."""
    x = ref.inputs(B, T, Hk, H, dtype, seed=B + H)
    _check_forward(x, dtype=dtype)
    _check_backward(x, dtype)


UNEVEN = [40, 0, 1, 129, 64, 63, 65, 28, 200, 2]


@pytest.mark.parametrize("lens,H", [(UNEVEN, 2), (UNEVEN, 16), ([66, 64, 65, 1, 66], 20)])
def test_many_packed_sequences(lens, H):
    """Few and many pairs, of even and of uneven lengths."""
    lead = 3
    x = ref.inputs(1, lead + sum(lens) + 5, 2, H, BF16, seed=H, nseq=len(lens))
    spans = ref.spans_of(lens, lead)
    offsets = [a for a, _ in spans] + [lead + sum(lens)]
    _check_forward(x, spans, offsets)
    _check_backward(x, BF16, spans, offsets)


def test_most_packed_pairs():
    """More pairs than the blocks look over for their lengths."""
    lens = [24] * 519 + [25]
    x = ref.inputs(1, sum(lens), 1, 2, BF16, seed=5, nseq=len(lens))
    spans = ref.spans_of(lens)
    _check_forward(x, spans, [a for a, _ in spans] + [sum(lens)])


def test_two_threads_on_their_own_streams():
    """Calls that overlap, each with its own workspace: the values of calls made alone."""
    cases = [(1, 700, 2, 4, BF16), (2, 300, 1, 2, F32)]
    xs = [_cu(ref.inputs(*c, seed=i)) for i, c in enumerate(cases)]

    def run(x):
        o, sT = ops.delta_forward(*_args(x), s0=x["s0"])
        return [o, sT, *ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"]).values()]

    alone = [run(x) for x in xs]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = run(xs[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(alone, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [1, 70])
def test_decode_and_prefill_captured_after_an_eager_call(T):
    """A captured call of packed sequences whose offsets and slots change between replays."""
    x = _cu(ref.inputs(1, 3 * T, 1, 2, BF16, seed=T, nseq=3))
    offsets = torch.tensor([0, T, 2 * T, 3 * T], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    pool, o = x["s0"].clone(), torch.empty_like(x["v"])
    ops.delta_forward(*_args(x), s0=pool, offsets=offsets, slots=slots, o=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.delta_forward(*_args(x), s0=pool, offsets=offsets, slots=slots, o=o)
    for lens, order in (([T, T, T], [2, 0, 1]), ([2 * T, 0, T], [1, -1, 0]), ([1, 3 * T - 2, 1], [0, 1, 2])):
        offsets.copy_(torch.tensor([sum(lens[:i]) for i in range(4)], dtype=torch.int32))
        slots.copy_(torch.tensor(order, dtype=torch.int32))
        pool.copy_(x["s0"])
        graph.replay()
        want_pool = x["s0"].clone()
        want, _ = ops.delta_forward(*_args(x), s0=want_pool, offsets=offsets, slots=slots)
        assert torch.equal(o, want) and torch.equal(pool, want_pool)
    assert ops.device_status() == 0


def test_offsets_beyond_32_bits():
    """2^31 elements of v and more: the last tokens as in a call of their own, which starts from the state
    that the tokens before leave (chunks then start at the same tokens)."""
    T, H, n = (1 << 20) + 64, 32, 192
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(BF16)  # noqa: E731
    x = [unit(rn(1, T, 1, 64)), unit(rn(1, T, 1, 64)), rn(1, T, H, 64), -rn(1, T, H).abs(), torch.sigmoid(rn(1, T, H))]
    assert x[2].numel() > 1 << 31
    head, tail = [t[:, :T - n] for t in x], [t[:, T - n:] for t in x]
    o, sT = ops.delta_forward(*x)
    o_tail = o[:, T - n:].clone()
    _, mid = ops.delta_forward(*head, o=o[:, :T - n])
    o2, sT2 = ops.delta_forward(*tail, s0=mid)
    assert torch.equal(o_tail, o2) and torch.equal(sT, sT2)
    del o, o2, head
    do, dsT = rn(1, T, H, 64), 0.1 * torch.randn(1, H, 64, 64, generator=gen, device="cuda")
    got = {m: t[:, T - n:].clone() for m, t in ops.delta_backward(*x, do, dsT=dsT, want_ds0=False).items()}
    want = ops.delta_backward(*tail, do[:, T - n:].contiguous(), s0=mid, dsT=dsT, want_ds0=False)
    for m in want:  # bf16 roundings of two forms of the same sums: 2^-8 each
        assert ref.rel(got[m], want[m].cpu()) <= 2 * 2.0 ** -8, m
    assert ops.device_status() == 0


def test_pools_beyond_32_bits():
    P, H = 140000, 4
    pool = torch.empty(P, H, 64, 64, device="cuda")
    assert pool.numel() > 1 << 31
    x = _cu(ref.inputs(2, 1, 2, H, BF16, seed=9))
    pool[P - 1], pool[7] = x["s0"][0], x["s0"][1]
    ops.state_copy(pool, *(torch.tensor(i, dtype=torch.int32, device="cuda") for i in ([P - 1], [P - 2])))
    o, _ = ops.delta_forward(*_args(x), s0=pool, slots=torch.tensor([P - 2, 7], dtype=torch.int32, device="cuda"))
    want, sT = ops.delta_forward(*_args(x), s0=x["s0"])
    assert torch.equal(o, want) and torch.equal(pool[P - 2], sT[0]) and torch.equal(pool[7], sT[1])
    assert torch.equal(pool[P - 1], x["s0"][0]) and ops.device_status() == 0
