"""Gated delta rule: errors of every (sequence, head) by itself, so that a head whose decays make its
gradients small counts as much as the largest.

Tolerances of the chunked bf16 calls, as 2-norm of the difference over the 2-norm of the reference.  A
rounding to bf16 is off by at most half a step, 2^-8 of the value, and evenly spread over that range: at
most 2^-8 / sqrt(3) of a tensor's norm.  Roundings of their own add in squares: n of them 2^-8 sqrt(n / 3).
The terms they enter (what the state before the chunk gives, what the chunk's tokens give) may cancel
in part, since an update takes back what its key already recalls: half of the squares allowed for.
  o       its own rounding; P, U; S in Q S (its norm counts once with P U's):  3, cancelling
  dq      its own; diag(gamma) dO and S; the scores and the U in them:         3, cancelling
  dk      its own; U and dS; dW and S; scores, dW and U:                       4, cancelling
  dv      its own and dW's:                                                    2
  dbeta   its own; dW; S or U:                                                 3, cancelling
  dg      its own; three in every pair's term:                                 4, cancelling
dbeta and dg have one value a token, and those of dg in a chunk are sums of the same terms, so that few
of them are independent: twice the figure, and where a sequence has fewer than 64 of them, one norm for
all sequences and heads.  Token walks round their bf16 results only (one rounding), and
fp32 results and states are held to the tolerances derived in test_gpu_delta.py.
"""
import pytest
import torch

import delta_ref as ref
from test_gpu_delta import BF16, F32, SCALE, TOL, TOL_STATE, _args, _check_backward, _cu, _hard
from wkv_recurrence_02_b200 import ops

pytestmark = pytest.mark.gpu

CHUNKED = {n: 2.0 ** -8 * (k / 3) ** 0.5 * 2 ** 0.5 for n, k in (("o", 3), ("dq", 3), ("dk", 4), ("dbeta", 3), ("dg", 4))}
CHUNKED["dv"] = 2.0 ** -8 * (2 / 3) ** 0.5
CHUNKED["dbeta"] *= 2
CHUNKED["dg"] *= 2


def _tol(name, dtype, chunked):
    if name in ("sT", "ds0"):
        return TOL_STATE[dtype] if chunked or dtype == F32 else TOL_STATE[F32]
    if dtype == F32:
        return TOL[F32]
    return CHUNKED[name] if chunked else 2.0 ** -8 + TOL[F32]


def _each(name, got, want, spans, dtype, chunked):
    """Every (sequence, head) against its own norm; a norm below 2^-20 of the largest counts as that."""
    got, want = got.cpu().double(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    if name in ("sT", "ds0"):
        parts = [(got[i, h], want[i, h]) for i in range(want.shape[0]) for h in range(want.shape[1])]
    else:
        if spans is None:
            rows = [(got[b], want[b]) for b in range(want.shape[0])]
        else:
            rows = [(got[0, a:a + n], want[0, a:a + n]) for a, n in spans if n]
        parts = [(g[:, h], w[:, h]) for g, w in rows for h in range(w.shape[1])]
        if name in ("dg", "dbeta") and min(w.numel() for _, w in parts) < 64:
            parts = [tuple(torch.cat([p[i] for p in parts]) for i in range(2))]
    floor = 2.0 ** -20 * max(float(w.norm()) for _, w in parts)
    worst = max(float((g - w).norm()) / max(float(w.norm()), floor, 1e-30) for g, w in parts)
    assert worst <= _tol(name, dtype, chunked), (name, worst)


def _check(x, dtype, chunked, bwd_chunked, spans=None, offsets=None):
    d = _cu(x)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o = torch.zeros_like(d["v"])  # tokens outside every sequence keep it
    o, sT = ops.delta_forward(*_args(d), scale=SCALE, s0=d["s0"], offsets=off, o=o)
    ro, rs = ref.forward(*_args(x), SCALE, x["s0"], spans)
    got = ops.delta_backward(*_args(d), d["do"], scale=SCALE, s0=d["s0"], dsT=d["dsT"], offsets=off)
    want = ref.backward(*_args(x), x["do"], SCALE, x["s0"], x["dsT"], spans)
    assert ops.device_status() == 0
    _each("o", o, ro, spans, dtype, chunked)
    _each("sT", sT, rs, spans, dtype, chunked)
    for n in want:
        _each(n, got[n], want[n], spans, dtype, bwd_chunked)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H", [(2, 300, 6), (1, 700, 4), (3, 130, 26)])
def test_heads(dtype, B, T, H):
    _check(ref.inputs(B, T, H, H, dtype, seed=B + T), dtype, dtype == BF16, dtype == BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [2, 16])
def test_heads_packed(dtype, H):
    lens = [70, 300, 0, 129, 64, 190]
    spans = ref.spans_of(lens, 3)
    x = ref.inputs(1, 3 + sum(lens) + 2, H, H, dtype, seed=H, nseq=len(lens))
    _check(x, dtype, dtype == BF16, dtype == BF16, spans, [a for a, _ in spans] + [3 + sum(lens)])


@pytest.mark.parametrize("B,T,H,chunked,bwd", [(3, 8, 4, False, False), (3, 9, 4, False, True), (2, 23, 8, False, True),
                                               (2, 24, 8, True, True)])
def test_lengths_beside_the_choice_of_path(B, T, H, chunked, bwd):
    """Both sides of the shortest lengths that take the tensor cores."""
    need = ops.delta_forward_workspace_bytes(B, T, H, H)
    assert (need > 0) == chunked
    _check(ref.inputs(B, T, H, H, BF16, seed=T), BF16, chunked, bwd)


@pytest.mark.parametrize("lens,chunked,bwd", [([23, 23, 24, 23], False, True), ([24, 24, 24, 24], True, True),
                                              ([100, 1, 1, 1], True, True), ([100, 1, 1, 1, 1], False, True),
                                              ([80, 1, 1, 0, 1, 1, 1, 1, 1, 1], False, False)])
def test_packed_lengths_beside_the_choice_of_path(lens, chunked, bwd):
    spans = ref.spans_of(lens)
    x = ref.inputs(1, sum(lens), 2, 2, BF16, seed=len(lens), nseq=len(lens))
    need = ops.delta_forward_workspace_bytes(1, sum(lens), 2, 2, nseq=len(lens), packed=True)
    assert (need > 0) == chunked
    _check(x, BF16, chunked, bwd, spans, [a for a, _ in spans] + [sum(lens)])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [5, 150])
def test_backward_zero_keys(dtype, T):
    """Nothing is recalled: dv and dbeta are zero, the other gradients are those of a decaying sum."""
    got = _check_backward(_hard("zero_keys", 1, T, 2, dtype), dtype)
    assert not got["dv"].any() and not got["dbeta"].any()
