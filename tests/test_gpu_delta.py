"""GPU parity of the gated delta rule (forward, decode, backward) with the 64-bit reference.

Tolerances, as 2-norm of the difference over the 2-norm of the reference, unit keys:
  fp32 calls     2e-5: a sum of 64 products in fp32 is off by at most 64 * 2^-24 = 3.8e-6 of its
                 terms' size; a token takes three such sums (k S, the update, q S), and unit
                 keys with gates in (0, 1) contract what earlier tokens left
  bf16 outputs   2^-6: the output's own rounding and those of the operands it is formed from
                 (scores, updates, state: three more), each at most 2^-8 of the value
  fp32 states    4e-5: a state is formed from operands kept as two bf16 terms, off by at most
  of bf16 calls  2^-16 = 1.5e-5 of the value each, and two such operands meet in a product
"""
import pytest
import torch

import delta_ref as ref
from wkv_recurrence_02_b200 import ops

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2e-5, BF16: 2.0 ** -6}
TOL_STATE = {F32: 2e-5, BF16: 4e-5}
SCALE = 0.125


def _cu(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def _args(x):
    return [x[n] for n in ("q", "k", "v", "g", "beta")]


def _check_forward(x, spans=None, offsets=None, dtype=BF16, scale=SCALE):
    d = _cu(x)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ro, rs = ref.forward(*_args(x), scale, x["s0"], spans)
    o = torch.full(x["v"].shape, 7.0, dtype=dtype, device="cuda")
    o, sT = ops.delta_forward(*_args(d), scale=scale, s0=d["s0"], offsets=off, o=o)
    assert ops.device_status() == 0
    if spans is not None:  # tokens outside every sequence are left as they were
        held = torch.zeros(x["v"].shape[1], dtype=torch.bool)
        for a, n in spans:
            held[a:a + n] = True
        assert (o.cpu()[:, ~held] == 7.0).all()
        ro = ro[:, held]
        o = o.cpu()[:, held]
    assert ref.rel(o, ro) <= TOL[dtype]
    assert ref.rel(sT, rs) <= TOL_STATE[dtype]
    return o, sT


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (3, 1, 2, 4), (2, 2, 1, 3), (2, 5, 3, 3), (1, 15, 2, 2), (2, 31, 1, 2),
                                      (1, 63, 2, 2), (2, 64, 1, 1), (1, 65, 2, 4), (2, 127, 1, 1), (1, 129, 3, 3),
                                      (1, 200, 2, 6), (1, 640, 1, 2)])
@pytest.mark.parametrize("state", [True, False])
def test_forward(dtype, B, T, Hk, H, state):
    _check_forward(ref.inputs(B, T, Hk, H, dtype, seed=T + H, state=state), dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,lead,tail", [([5, 0, 1, 64, 3], 0, 0), ([65, 130, 0], 2, 3), ([1, 1, 1, 1], 0, 4),
                                            ([63, 64, 65, 2], 1, 70), ([0, 0], 5, 5), ([200], 0, 100),
                                            ([17, 33, 100, 9, 81], 3, 1)])
def test_forward_packed(dtype, lens, lead, tail):
    T = lead + sum(lens) + tail
    x = ref.inputs(1, T, 2, 4, dtype, seed=T, nseq=len(lens))
    spans = ref.spans_of(lens, lead)
    for n in ("q", "k", "v", "g", "beta"):  # what lies outside every sequence must not matter
        x[n][:, :lead] = float("nan")
        x[n][:, lead + sum(lens):] = float("inf")
    clean = {n: t if t is None else torch.nan_to_num(t, 0.0, 0.0, 0.0) for n, t in x.items()}
    d = _cu(x)
    off = torch.tensor([a for a, _ in spans] + [lead + sum(lens)], dtype=torch.int32, device="cuda")
    ro, rs = ref.forward(*_args(clean), SCALE, x["s0"], spans)
    o = torch.full(x["v"].shape, 7.0, dtype=dtype, device="cuda")
    o, sT = ops.delta_forward(*_args(d), scale=SCALE, s0=d["s0"], offsets=off, o=o)
    assert ops.device_status() == 0
    held = slice(lead, lead + sum(lens))
    o = o.cpu()
    assert (o[:, :lead] == 7.0).all() and (o[:, lead + sum(lens):] == 7.0).all()
    assert ref.rel(o[:, held], ro[:, held]) <= TOL[dtype]
    assert ref.rel(sT, rs) <= TOL_STATE[dtype]


def test_forward_offsets_outside_the_tokens_are_clamped():
    x = ref.inputs(1, 40, 1, 2, BF16, seed=8, nseq=3)
    d = _cu(x)
    off = torch.tensor([-7, 10, 25, 1000], dtype=torch.int32, device="cuda")
    ro, rs = ref.forward(*_args(x), SCALE, x["s0"], [(0, 10), (10, 15), (25, 15)])
    o, sT = ops.delta_forward(*_args(d), scale=SCALE, s0=d["s0"], offsets=off)
    assert ref.rel(o, ro) <= TOL[BF16] and ref.rel(sT, rs) <= TOL_STATE[BF16]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 3, 100])
@pytest.mark.parametrize("inplace", [True, False])
def test_forward_slots(dtype, T, inplace):
    """A pool of 7 states, 4 rows: two with slots, one padding row, one past the pool."""
    x = ref.inputs(4, T, 1, 2, dtype, seed=T)
    pool = 0.1 * torch.randn(7, 2, 64, 64, generator=torch.Generator().manual_seed(1))
    slots = [5, -1, 0, 7]
    s0 = torch.stack([pool[s] if 0 <= s < 7 else torch.zeros(2, 64, 64) for s in slots])
    ro, rs = ref.forward(*_args(x), SCALE, s0)
    d, dpool = _cu(x), pool.cuda()
    other = None if inplace else torch.full_like(dpool, 3.0)
    assert ops.device_status() == 0
    o, sT = ops.delta_forward(*_args(d), scale=SCALE, s0=dpool, sT=other,
                              slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert ops.device_status() == -8  # the slot past the pool
    assert sT.data_ptr() == (dpool if inplace else other).data_ptr()
    assert ref.rel(o, ro) <= TOL[dtype]
    assert ref.rel(sT[[5, 0]], rs[[0, 2]]) <= TOL_STATE[dtype]
    rest = [1, 2, 3, 4, 6]
    assert torch.equal(sT.cpu()[rest], (pool if inplace else torch.full_like(pool, 3.0))[rest])
    if not inplace:
        assert torch.equal(dpool.cpu(), pool)


@pytest.mark.parametrize("T", [1, 7, 40])
def test_forward_slots_without_a_pool(T):
    """No state is read or kept, so no slot is past a pool either."""
    x = _cu(ref.inputs(2, T, 1, 2, BF16, seed=T))
    slots = torch.tensor([100, 1], dtype=torch.int32, device="cuda")
    assert ops.device_status() == 0
    o = ops.delta_forward(*_args(x), slots=slots, want_state=False)
    assert ops.device_status() == 0
    assert torch.equal(o, ops.delta_forward(*_args(x), want_state=False))


HARD = ["no_decay", "reset", "fast", "far", "gate0", "gate1_same_key", "gate2", "zero_keys", "correlated", "growth"]


def _hard(kind, B, T, H, dtype, seed=11):
    x = ref.inputs(B, T, H, H, dtype, seed=seed)
    if kind == "no_decay":
        x["g"].zero_()
    elif kind == "reset":  # forgets everything at some tokens
        x["g"][:, ::7] = -float("inf")
    elif kind == "fast":
        x["g"].fill_(-30.0)
    elif kind == "far":  # very large drops, slow decay between them
        x["g"][:, ::9] = -2000.0
    elif kind == "gate0":
        x["beta"].zero_()
    elif kind == "gate1_same_key":  # every token overwrites the same direction
        x["k"][:] = x["k"][:, :1]
        x["beta"].fill_(1.0)
    elif kind == "gate2":  # a reflection
        x["beta"].fill_(2.0)
        x["g"] -= 0.05
    elif kind == "zero_keys":
        x["k"].zero_()
    elif kind == "correlated":  # keys near one another
        x["k"] = torch.nn.functional.normalize(x["k"].float() + 2 * x["k"][:, :1].float(), dim=-1).to(dtype)
    elif kind == "growth":
        x["g"].fill_(0.02)
    return x


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", HARD)
@pytest.mark.parametrize("T", [4, 150])
def test_forward_hard(dtype, kind, T):
    x = _hard(kind, 1, T, 2, dtype)
    ro, rs = ref.forward(*_args(x), SCALE, x["s0"])
    d = _cu(x)
    o, sT = ops.delta_forward(*_args(d), scale=SCALE, s0=d["s0"])
    assert ops.device_status() == 0
    assert ref.rel(o, ro) <= TOL[dtype]
    assert ref.rel(sT, rs) <= TOL_STATE[dtype]


def test_forward_no_tokens_copies_the_state():
    x = _cu(ref.inputs(3, 0, 1, 2, BF16, seed=1))
    o, sT = ops.delta_forward(*_args(x), s0=x["s0"])
    assert o.shape == (3, 0, 2, 64) and torch.equal(sT, x["s0"])
    _, sT = ops.delta_forward(*_args(x))
    assert not sT.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_in_place_and_without_state(dtype):
    x = ref.inputs(2, 90, 1, 2, dtype, seed=5)
    d = _cu(x)
    o, sT = ops.delta_forward(*_args(d), s0=d["s0"])
    alone = ops.delta_forward(*_args(d), s0=d["s0"], want_state=False)
    s = d["s0"].clone()
    o2, _ = ops.delta_forward(*_args(d), s0=s, sT=s)
    assert torch.equal(o, alone) and torch.equal(o, o2) and torch.equal(sT, s)


def test_forward_is_deterministic_on_other_streams():
    x = _cu(ref.inputs(2, 300, 2, 4, BF16, seed=6))
    o, sT = ops.delta_forward(*_args(x), s0=x["s0"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # two calls that may run at once
        with torch.cuda.stream(s):
            got.append(ops.delta_forward(*_args(x), s0=x["s0"]))
    torch.cuda.synchronize()
    for o2, s2 in got:
        assert torch.equal(o, o2) and torch.equal(sT, s2)


@pytest.mark.parametrize("T", [1, 130])
def test_forward_replayed_in_a_graph(T):
    x = _cu(ref.inputs(2, T, 1, 2, BF16, seed=7))
    state = x["s0"].clone()
    ops.delta_forward(*_args(x), s0=state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = ops.delta_forward(*_args(x), s0=state, sT=state)
    state.copy_(x["s0"])
    graph.replay()
    graph.replay()
    o1, s1 = ops.delta_forward(*_args(x), s0=x["s0"])
    o2, s2 = ops.delta_forward(*_args(x), s0=s1)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(state, s2)


# ------------------------------------------------------------------------------- backward

GRADS = ("dq", "dk", "dv", "dg", "dbeta")


def _check_backward(x, dtype, spans=None, offsets=None, state=True, tol=None):
    d = _cu(x)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    want = ref.backward(*_args(x), x["do"], SCALE, x["s0"], x["dsT"], spans)
    got = ops.delta_backward(*_args(d), d["do"], scale=SCALE, s0=d["s0"], dsT=d["dsT"], offsets=off)
    assert ops.device_status() == 0
    for n in GRADS:
        assert got[n].dtype == dtype
        e = ref.rel(got[n], want[n])
        assert e <= (tol or TOL[dtype]), (n, e)
    e = ref.rel(got["ds0"], want["ds0"])
    assert e <= TOL_STATE[dtype], ("ds0", e)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (3, 2, 1, 2), (2, 8, 2, 2), (1, 9, 1, 3), (1, 63, 2, 2), (2, 64, 1, 1),
                                      (1, 65, 2, 4), (1, 130, 1, 3), (2, 200, 2, 2)])
@pytest.mark.parametrize("state", [True, False])
def test_backward(dtype, B, T, Hk, H, state):
    _check_backward(ref.inputs(B, T, Hk, H, dtype, seed=T + H, state=state), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,lead,tail", [([5, 0, 1, 64, 3], 0, 0), ([65, 130, 0], 2, 3), ([63, 64, 65, 2], 1, 70)])
@pytest.mark.parametrize("Hk,H", [(2, 2), (1, 3)])
def test_backward_packed(dtype, lens, lead, tail, Hk, H):
    T = lead + sum(lens) + tail
    x = ref.inputs(1, T, Hk, H, dtype, seed=T, nseq=len(lens))
    spans = ref.spans_of(lens, lead)
    got = _check_backward(x, dtype, spans, [a for a, _ in spans] + [lead + sum(lens)])
    for n in GRADS:  # tokens outside every sequence: the zeros the binding put there
        assert not got[n][:, :lead].any() and not got[n][:, lead + sum(lens):].any()


def test_backward_leaves_tokens_outside_the_sequences_as_they_were():
    """Through the C entry point, with outputs that hold something."""
    for dtype in (F32, BF16):
        x = _cu(ref.inputs(1, 90, 1, 2, dtype, seed=3, nseq=1))
        for n in ("q", "k", "v", "g", "beta", "do"):
            x[n][:, :4] = float("nan")
            x[n][:, 80:] = float("nan")
        off = torch.tensor([4, 80], dtype=torch.int32, device="cuda")
        lib = ops.load()
        out = {n: torch.full_like(x[m], 5.0) for n, m in zip(GRADS, ("q", "k", "v", "g", "beta"))}
        ds0 = torch.empty_like(x["s0"])
        ws = torch.empty(ops.delta_backward_workspace_bytes(1, 90, 1, 2, 64, 1, True, dtype == BF16), dtype=torch.uint8,
                         device="cuda")
        ops._use_current_stream(lib, x["q"].device)
        fn = lib.rwkv_delta_backward_bf16 if dtype == BF16 else lib.rwkv_delta_backward
        p = ops._ptr
        ops._check(fn(1, 90, 1, 2, 64, *[p(t) for t in _args(x)], SCALE, 1, p(off), p(x["s0"]), p(x["do"]), p(x["dsT"]),
                      *[p(out[n]) for n in GRADS], p(ds0), p(ws), ws.numel()))
        torch.cuda.synchronize()
        for n in GRADS:
            assert (out[n][:, :4] == 5.0).all() and (out[n][:, 80:] == 5.0).all()
            assert torch.isfinite(out[n]).all()
        assert torch.isfinite(ds0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [k for k in HARD if k not in ("zero_keys",)])
def test_backward_hard(dtype, kind):
    x = _hard(kind, 1, 150, 2, dtype)
    _check_backward(x, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_in_place_and_given_workspace(dtype):
    x = _cu(ref.inputs(2, 70, 1, 2, dtype, seed=9))
    a = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    need = ops.delta_backward_workspace_bytes(2, 70, 1, 2, bf16=dtype == BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    b = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"], workspace=ws)
    c = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"], want_ds0=False)
    for n in GRADS:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])
    assert torch.equal(a["ds0"], b["ds0"]) and "ds0" not in c
    with pytest.raises(ops.WkvError):
        ops.delta_backward(*_args(x), x["do"], workspace=ws[: need - 16])


def test_backward_replayed_in_a_graph_beside_an_eager_call():
    x = _cu(ref.inputs(1, 130, 1, 2, BF16, seed=12))
    want = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    graph.replay()
    eager = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n]) and torch.equal(want[n], eager[n])


# ------------------------------------------------------------------------------- together

def test_serving_run():
    """Prefill packed prompts into pool slots, fork one, decode, drop a sequence, compact, decode:
    every state and output as if each sequence had run alone."""
    H, Hk, lens = 4, 2, [70, 1, 200]
    x = ref.inputs(1, sum(lens), Hk, H, BF16, seed=21, nseq=3, state=False)
    spans = ref.spans_of(lens)
    pool = torch.full((8, H, 64, 64), float("nan"), device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ops.state_copy(pool, i32([-1, -1, -1]), i32([6, 2, 4]))  # fresh slots
    d = _cu(x)
    o, _ = ops.delta_forward(*_args(d), scale=SCALE, s0=pool, offsets=i32([0, 70, 71, 271]), slots=i32([6, 2, 4]))
    ro, rs = ref.forward(*_args(x), SCALE, None, spans)
    assert ref.rel(o, ro) <= TOL[BF16]
    ops.state_copy(pool, i32([4, 4]), i32([0, 7]))  # two more samples of the last prompt
    state = {6: rs[0], 2: rs[1], 4: rs[2], 0: rs[2], 7: rs[2]}
    rows = [6, 2, 4, 0, 7]
    for step in range(2):
        y = ref.inputs(6, 1, Hk, H, BF16, seed=30 + step, state=False)
        o, _ = ops.delta_forward(*_args(_cu(y)), scale=SCALE, s0=pool, slots=i32(rows + [-1]))
        s0 = torch.stack([state[r] for r in rows] + [torch.zeros(H, 64, 64, dtype=torch.float64)])
        ro, rs = ref.forward(*_args(y), SCALE, s0)
        assert ref.rel(o, ro) <= TOL[BF16]
        state = {r: rs[i] for i, r in enumerate(rows)}
    live = torch.zeros(8, dtype=torch.bool)
    live[[6, 4, 0, 7]] = True  # slot 2's sequence has finished
    index, count = ops.state_compact(pool, live.cuda())
    assert count.item() == 4 and index.tolist() == [0, -1, -1, -1, 1, -1, 2, 3]
    y = ref.inputs(4, 1, Hk, H, BF16, seed=40, state=False)
    o, _ = ops.delta_forward(*_args(_cu(y)), scale=SCALE, s0=pool, slots=i32([0, 1, 2, 3]))
    ro, rs = ref.forward(*_args(y), SCALE, torch.stack([state[r] for r in (0, 4, 6, 7)]))
    assert ref.rel(o, ro) <= TOL[BF16] and ref.rel(pool[:4], rs) <= TOL_STATE[BF16]
    assert ops.device_status() == 0


def test_training_run_matches_the_forward():
    """A descent step along the gradients lowers <o, do> + <sT, dsT> by what they say."""
    x = ref.inputs(2, 100, 1, 2, F32, seed=31)
    d = _cu(x)
    got = ops.delta_backward(*_args(d), d["do"], scale=SCALE, s0=d["s0"], dsT=d["dsT"])
    loss = lambda y: sum((a.double() * b.double()).sum() for a, b in zip(  # noqa: E731
        ops.delta_forward(*_args(y), scale=SCALE, s0=y["s0"]), (d["do"], d["dsT"])))
    h = 1e-2
    along = {n: got["d" + n] / got["d" + n].norm() for n in ("q", "k", "v", "g", "beta", "s0")}
    for n, a in along.items():
        up, down = dict(d), dict(d)
        up[n], down[n] = d[n] + h * a, d[n] - h * a
        num = float(loss(up) - loss(down)) / (2 * h)
        ana = float((got["d" + n].double() * a.double()).sum())
        # second differences of this smooth function are of order h^2; fp32 rounding of the loss / h
        assert abs(num - ana) <= 2e-3 * abs(ana), n


def test_binding_refusals():
    x = _cu(ref.inputs(2, 5, 2, 4, BF16, seed=1))
    a = _args(x)
    with pytest.raises(ops.WkvError):  # 3 heads do not share 2
        ops.delta_forward(a[0], a[1], a[2][:, :, :3].contiguous(), a[3][..., :3].contiguous(), a[4][..., :3].contiguous())
    with pytest.raises(ValueError):
        ops.delta_forward(a[0].transpose(1, 2), *a[1:])
    with pytest.raises(TypeError):
        ops.delta_forward(a[0], a[1], a[2], a[3].float(), a[4])
    with pytest.raises(TypeError):
        ops.delta_forward(*a, offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ops.WkvError):  # packed sequences need B = 1
        ops.delta_forward(*a, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ops.delta_forward(*a, slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ops.delta_forward(*a, s0=x["s0"][:1].contiguous())
    with pytest.raises(ValueError):
        ops.delta_backward(*a, x["do"][:, :4].contiguous())
