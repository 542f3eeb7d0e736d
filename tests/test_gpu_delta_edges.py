"""Gated delta rule: calls at the edges of what the header allows.  Where two calls do the same
arithmetic the results have to be equal bit for bit; tolerances are those of test_gpu_delta.py."""
import pytest
import torch

import delta_ref as ref
from test_gpu_delta import BF16, F32, GRADS, SCALE, TOL, TOL_STATE, _args, _check_backward, _check_forward, _cu
from wkv_recurrence_02_b200 import ops

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [[0], [63, 64], [15, 16, 17, 127, 128], list(range(140))])
def test_tokens_that_forget_everything(dtype, at):
    """g of -inf at the borders of blocks and chunks, and everywhere."""
    x = ref.inputs(1, 140, 2, 2, dtype, seed=len(at))
    x["g"][:, at] = -float("inf")
    _check_forward(x, dtype=dtype)
    got = _check_backward(x, dtype)
    if at[0] == 0:
        assert not got["ds0"].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [4, 100])
@pytest.mark.parametrize("scale", [0.0, -1.5])
def test_other_scales(dtype, T, scale):
    x = ref.inputs(1, T, 1, 2, dtype, seed=T)
    d = _cu(x)
    ro, rs = ref.forward(*_args(x), scale, x["s0"])
    o, sT = ops.delta_forward(*_args(d), scale=scale, s0=d["s0"])
    assert ref.rel(o, ro) <= TOL[dtype] and ref.rel(sT, rs) <= TOL_STATE[dtype]
    got = ops.delta_backward(*_args(d), d["do"], scale=scale, s0=d["s0"], dsT=d["dsT"])
    want = ref.backward(*_args(x), x["do"], scale, x["s0"], x["dsT"])
    for n in GRADS:
        assert ref.rel(got[n], want[n]) <= TOL[dtype], n
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[70, 61, 128, 3], [5, 4, 7, 6]])
@pytest.mark.parametrize("bad", [0, 1, 3])
def test_a_sequence_that_is_not_finite_stays_alone(dtype, lens, bad):
    """Every other sequence of the packed call is what it is beside finite ones, bit for bit."""
    n = len(lens)
    spans = ref.spans_of(lens)
    off = _i32([a for a, _ in spans] + [sum(lens)])
    x = _cu(ref.inputs(1, sum(lens), 1, 2, dtype, seed=sum(lens), nseq=n))

    def run(y):
        o, sT = ops.delta_forward(*_args(y), s0=y["s0"], offsets=off)
        return o, sT, ops.delta_backward(*_args(y), y["do"], s0=y["s0"], dsT=y["dsT"], offsets=off)

    o, sT, grads = run(x)
    y = {m: t.clone() for m, t in x.items()}
    a, k = spans[bad]
    for m in ("q", "k", "v", "g", "beta", "do"):
        y[m][:, a:a + k] = float("nan")
    y["s0"][bad] = float("inf")
    o2, sT2, grads2 = run(y)
    held = [i for i in range(n) if i != bad]
    for i in held:
        s = slice(spans[i][0], spans[i][0] + spans[i][1])
        assert torch.equal(o[:, s], o2[:, s]) and torch.equal(sT[i], sT2[i]), i
        assert torch.equal(grads["ds0"][i], grads2["ds0"][i]), i
        for m in GRADS:
            assert torch.equal(grads[m][:, s], grads2[m][:, s]), (m, i)
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 6, 90])
def test_fresh_sequences_into_slots(dtype, T):
    """No s0, a pool for the last states: the sequences start from zero whatever the slots hold."""
    x = _cu(ref.inputs(3, T, 1, 2, dtype, seed=T))
    pool = torch.full((5, 2, 64, 64), float("nan"), device="cuda")
    o, sT = ops.delta_forward(*_args(x), sT=pool, slots=_i32([4, -1, 1]))
    want, states = ops.delta_forward(*_args(x))
    assert sT is pool and torch.equal(o, want)
    assert torch.equal(pool[4], states[0]) and torch.equal(pool[1], states[2])
    assert torch.isnan(pool[[0, 2, 3]]).all() and ops.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed_calls_without_tokens_or_sequences(dtype):
    x = _cu(ref.inputs(1, 0, 1, 2, dtype, seed=1, nseq=3))
    off = _i32([0, 0, 0, 0])
    o, sT = ops.delta_forward(*_args(x), s0=x["s0"], offsets=off)
    assert o.shape == (1, 0, 2, 64) and torch.equal(sT, x["s0"])
    got = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"], offsets=off)
    assert torch.equal(got["ds0"], x["dsT"])
    y = _cu(ref.inputs(1, 30, 1, 2, dtype, seed=2, nseq=1, state=False))
    o = torch.full_like(y["v"], 7.0)
    _, sT = ops.delta_forward(*_args(y), offsets=_i32([0]), o=o)
    assert sT.shape == (0, 2, 64, 64) and (o == 7.0).all()
    got = ops.delta_backward(*_args(y), y["do"], offsets=_i32([0]))
    assert got["ds0"].shape == (0, 2, 64, 64) and not any(got[n].any() for n in GRADS)
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype,T", [(BF16, 40), (BF16, 3), (F32, 12)])
def test_backward_replayed_over_new_offsets(dtype, T):
    """A captured packed backward: the offsets are read on the device, the rest of the gradients zeroed."""
    x = _cu(ref.inputs(1, 3 * T, 1, 2, dtype, seed=T, nseq=3))
    off = _i32([0, T, 2 * T, 3 * T])
    run = lambda: ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"], offsets=off)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for new in ([0, T, 2 * T, 3 * T], [1, 1, 3 * T - 1, 3 * T - 1], [0, 0, 0, 3 * T], [2, 3, 4, 5]):
        off.copy_(_i32(new))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (n, new)
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype,n,T", [(BF16, 2000, 30), (BF16, 3000, 2), (F32, 2000, 9)])
def test_thousands_of_sequences(dtype, n, T):
    """Packed sequences of one length are the rows of a batch."""
    x = _cu(ref.inputs(n, T, 1, 1, dtype, seed=T))
    y = {m: (t if m in ("s0", "dsT") else t.view(1, n * T, *t.shape[2:])) for m, t in x.items()}
    off = torch.arange(n + 1, dtype=torch.int32, device="cuda") * T
    o, sT = ops.delta_forward(*_args(x), s0=x["s0"])
    o2, sT2 = ops.delta_forward(*_args(y), s0=y["s0"], offsets=off)
    assert torch.equal(o.view_as(o2), o2) and torch.equal(sT, sT2)
    a = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    b = ops.delta_backward(*_args(y), y["do"], s0=y["s0"], dsT=y["dsT"], offsets=off)
    for m in a:
        # a lone segment takes dsT where others take what the walk left of it, the same values
        assert torch.equal(a[m].view_as(b[m]), b[m]), m
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [70, 1000])
def test_long_keys(T):
    """Keys of norm 3 with gates that keep each update a contraction (beta |k|^2 below one)."""
    x = ref.inputs(1, T, 2, 2, BF16, seed=T)
    x["k"] = (3 * x["k"].float()).to(BF16)
    x["beta"] = (x["beta"].float() / 10).to(BF16)
    _check_forward(x)
    _check_backward(x, BF16)
    _check_forward({m: t.float() for m, t in x.items()}, dtype=F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_one_long_sequence(dtype):
    """Chained halves: the first half's gradients from the state gradient that the second half's call
    returns.  The halves meet at a chunk's border, so that both ways form the same chunks."""
    T = 4096
    x = _cu(ref.inputs(1, T, 1, 1, dtype, seed=6))
    whole = ops.delta_backward(*_args(x), x["do"], s0=x["s0"], dsT=x["dsT"])
    half = [{m: (t[:, s].contiguous() if t.dim() > 2 and t.shape[1] == T else t) for m, t in x.items()}
            for s in (slice(0, T // 2), slice(T // 2, T))]
    _, mid = ops.delta_forward(*_args(half[0]), s0=x["s0"], scale=SCALE)
    late = ops.delta_backward(*_args(half[1]), half[1]["do"], s0=mid, dsT=x["dsT"])
    early = ops.delta_backward(*_args(half[0]), half[0]["do"], s0=x["s0"], dsT=late["ds0"])
    assert ref.rel(early["ds0"], whole["ds0"].cpu()) <= 2 * TOL_STATE[dtype]
    for m in GRADS:
        assert ref.rel(torch.cat([early[m], late[m]], 1), whole[m].cpu()) <= 2 * TOL_STATE[dtype] + (
            2.0 ** -8 if dtype == BF16 else 0), m
