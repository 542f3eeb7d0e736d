"""Refusals of the delta-rule and state-pool entry points, without a GPU: every call either
fails validation on the host or has nothing to compute (the pointers are never followed)."""
import ctypes

import pytest
import torch

from wkv_recurrence_02_b200 import build, ops

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
STEP = 1 << 28


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def _p(i, off=0):
    return ctypes.c_void_p(FAKE + i * STEP + off)


FWD = ["q", "k", "v", "g", "beta", "offsets", "slots", "s0", "o", "sT", "ws"]


def _forward(lib, bf16=True, B=1, T=8, Hk=2, H=4, N=64, scale=0.125, nseq=2, nslots=4, wbytes=STEP, **kw):
    a = {n: _p(i) for i, n in enumerate(FWD)}
    a["offsets"] = a["slots"] = None
    a.update(kw)
    fn = lib.rwkv_delta_forward_bf16 if bf16 else lib.rwkv_delta_forward
    return fn(B, T, Hk, H, N, a["q"], a["k"], a["v"], a["g"], a["beta"], scale, nseq, a["offsets"], nslots,
              a["slots"], a["s0"], a["o"], a["sT"], a["ws"], ctypes.c_size_t(wbytes))


@pytest.mark.parametrize("bf16", [True, False])
def test_forward_refusals(lib, bf16):
    f = lambda **kw: _forward(lib, bf16, **kw)  # noqa: E731
    assert f(N=128) == -3
    assert f(B=-1) == -2 and f(T=-1) == -2 and f(H=-4) == -2 and f(N=-64) == -2
    assert f(Hk=3) == -2 and f(Hk=0) == -2                      # Hk does not divide H
    assert f(B=2, offsets=_p(5)) == -2                          # packed needs B = 1
    assert f(offsets=_p(5), nseq=-1) == -2
    assert f(slots=_p(6), nslots=-1) == -2
    assert f(T=1 << 40, B=1 << 40) == -2                        # overflow
    assert f(T=1 << 31) == -2                                   # more tokens than an index holds
    assert f(B=1 << 30) == -2                                   # (sequence, head) pairs
    assert f(scale=float("nan")) == -8 and f(scale=float("inf")) == -8
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert f(**{n: None}) == -1, n
        assert f(**{n: _p(FWD.index(n), 8)}) == -7, n
    assert f(offsets=_p(5, 2)) == -7 and f(slots=_p(6, 1)) == -7
    for n in ("q", "k", "v", "g", "beta"):
        assert f(o=_p(FWD.index(n))) == -4, n
        assert f(sT=_p(FWD.index(n))) == -4, n
    assert f(offsets=_p(5), o=_p(5)) == -4 and f(slots=_p(6), sT=_p(6)) == -4
    assert f(o=_p(7)) == -4 and f(o=_p(9)) == -4                # o over a state
    assert f(sT=_p(7, 64)) == -4                                # sT partly over s0
    assert f(ws=_p(10, 8)) == -7


def test_forward_workspace(lib):
    need = ctypes.c_size_t(7)
    size = lambda T, bf16, packed=0, nseq=1, B=1: (lib.rwkv_delta_forward_workspace_bytes(  # noqa: E731
        B, T, 2, 4, 64, nseq, packed, bf16, ctypes.byref(need)), need.value)
    assert size(1, 1) == (0, 0) and size(15, 1) == (0, 0) and size(4096, 0) == (0, 0) and size(0, 1) == (0, 0)
    rc, n = size(200, 1)
    assert rc == 0 and n > 0
    assert size(200, 1, 1, 200)[1] == 0                         # packed: one token each on average
    assert size(8, 1, B=-1)[0] == -2
    f = lambda **kw: _forward(lib, True, T=200, **kw)  # noqa: E731
    assert f(wbytes=n - 1) == -8 and f(ws=None) == -1
    for i in FWD[:5] + ["s0", "o", "sT"]:
        assert f(ws=_p(FWD.index(i))) == -4, i


def test_forward_nothing_to_do(lib):
    none = {n: None for n in FWD}
    assert _forward(lib, B=0, **none) == 0
    assert _forward(lib, H=0, Hk=0, **none) == 0
    assert _forward(lib, T=0, **none) == 0                      # no token, no state asked for
    assert _forward(lib, **{**none, "offsets": _p(5)}, nseq=0) == 0


BWD = ["q", "k", "v", "g", "beta", "offsets", "s0", "dout", "dsT", "dq", "dk", "dv", "dg", "dbeta", "ds0", "ws"]


def _backward(lib, bf16=True, B=1, T=8, Hk=2, H=4, N=64, scale=0.125, nseq=2, wbytes=STEP, **kw):
    a = {n: _p(i) for i, n in enumerate(BWD)}
    a["offsets"] = None
    a.update(kw)
    fn = lib.rwkv_delta_backward_bf16 if bf16 else lib.rwkv_delta_backward
    return fn(B, T, Hk, H, N, a["q"], a["k"], a["v"], a["g"], a["beta"], scale, nseq, a["offsets"], a["s0"],
              a["dout"], a["dsT"], a["dq"], a["dk"], a["dv"], a["dg"], a["dbeta"], a["ds0"], a["ws"],
              ctypes.c_size_t(wbytes))


@pytest.mark.parametrize("bf16", [True, False])
def test_backward_refusals(lib, bf16):
    f = lambda **kw: _backward(lib, bf16, **kw)  # noqa: E731
    assert f(N=32) == -3 and f(B=-1) == -2 and f(Hk=3) == -2 and f(B=2, offsets=_p(5)) == -2
    assert f(scale=float("nan")) == -8
    for n in BWD:
        if n not in ("offsets", "s0", "dsT", "ds0"):
            assert f(**{n: None}) == -1, n
        if n != "offsets":
            assert f(**{n: _p(BWD.index(n), 4)}) == -7, n
    assert f(offsets=_p(5, 1)) == -7
    need = ctypes.c_size_t(0)
    assert lib.rwkv_delta_backward_workspace_bytes(1, 8, 2, 4, 64, 1, 0, int(bf16), ctypes.byref(need)) == 0
    assert need.value > 0 and f(wbytes=need.value - 1) == -8
    outs = BWD[9:]
    for n in outs:
        for m in ("q", "s0", "dout"):
            assert f(**{n: _p(BWD.index(m))}) == -4, (n, m)
    assert f(dq=_p(10)) == -4 and f(ds0=_p(8, 64)) == -4 and f(ws=_p(13)) == -4


def test_backward_nothing_to_do(lib):
    none = {n: None for n in BWD}
    assert _backward(lib, B=0, wbytes=0, **none) == 0
    assert _backward(lib, T=0, wbytes=0, **none) == 0
    b = ctypes.c_size_t(7)
    assert lib.rwkv_delta_backward_workspace_bytes(0, 8, 2, 4, 64, 0, 0, 1, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.rwkv_delta_backward_workspace_bytes(1, 8, 2, 4, 64, 1, 0, 1, None) == -1
    assert lib.rwkv_delta_backward_workspace_bytes(1, 8, 3, 4, 64, 1, 0, 1, ctypes.byref(b)) == -2


@pytest.mark.parametrize("B,T,H,packed,nseq", [(1 << 21, 1, 64, 0, 0), (1 << 20, 8, 64, 0, 0), (1, 1 << 21, 64, 1, 1 << 21),
                                               (1 << 17, 9, 64, 0, 0), (1 << 24, 1, 1, 0, 0), (1, 1 << 30, 32, 0, 0)])
@pytest.mark.parametrize("shared", [1, 2])
def test_backward_workspace_of_many_sequences(lib, B, T, H, packed, nseq, shared):
    """Sizes within the limits are not refused, however many sequences they are of."""
    Hk, n = max(H // shared, 1), nseq if packed else B
    b = ctypes.c_size_t(1)
    shares = 0 if Hk == H else 2 * B * T * H * 64 * 4
    for bf16 in (0, 1):
        assert lib.rwkv_delta_backward_workspace_bytes(B, T, Hk, H, 64, nseq, packed, bf16, ctypes.byref(b)) == 0
        if not bf16 or (T // n if packed else T) < 9:  # token walks: a state and a gradient for every segment of 8 tokens
            segments = T // 8 + n if packed else B * -(-T // 8)
            states = 0 if T <= 8 and not packed else 2 * segments * H * 64 * 64 * 4
            assert b.value == states + shares
        else:  # chunks: T in two tiles of 8 KB, four more tiles
            assert b.value == B * -(-T // 64) * H * 6 * 8192 + shares


def test_state_copy_refusals(lib):
    f = lambda layers=1, nslots=8, sb=64, pool=_p(0), n=2, src=_p(1), dst=_p(2): lib.rwkv_state_copy(  # noqa: E731
        layers, nslots, sb, pool, n, src, dst)
    assert f(layers=-1) == -2 and f(nslots=-1) == -2 and f(sb=-16) == -2 and f(n=-1) == -2 and f(n=4097) == -2
    assert f(nslots=1 << 31) == -2 and f(layers=1 << 40, nslots=1 << 30, sb=1 << 20) == -2
    assert f(sb=24) == -7 and f(pool=_p(0, 8)) == -7 and f(src=_p(1, 2)) == -7 and f(dst=_p(2, 1)) == -7
    assert f(pool=None) == -1 and f(src=None) == -1 and f(dst=None) == -1
    assert f(src=_p(0, 64)) == -4 and f(dst=_p(0)) == -4
    assert f(n=0, src=None, dst=None) == 0 and f(layers=0, pool=None) == 0


def test_state_compact_refusals(lib):
    f = lambda layers=1, nslots=8, sb=64, pool=_p(0), live=_p(1), new=_p(2), count=_p(3): lib.rwkv_state_compact(  # noqa: E731
        layers, nslots, sb, pool, live, new, count)
    assert f(nslots=-1) == -2 and f(nslots=16385) == -2 and f(sb=8) == -7 and f(pool=_p(0, 4)) == -7
    assert f(pool=None) == -1 and f(live=None) == -1 and f(new=None) == -1 and f(count=None) == -1
    assert f(new=_p(2, 2)) == -7 and f(count=_p(3, 1)) == -7
    assert f(live=_p(0, 16)) == -4 and f(new=_p(0)) == -4 and f(count=_p(2, 4)) == -4 and f(live=_p(3)) == -4


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 2, 64)
    s = torch.zeros(1, 4, 2)
    with pytest.raises(TypeError, match="CUDA"):
        ops.delta_forward(x, x, x, s, s)
    with pytest.raises(TypeError, match="CUDA"):
        ops.delta_backward(x, x, x, s, s, x)
    with pytest.raises(TypeError, match="CUDA"):
        ops.state_copy(torch.zeros(4, 4), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        ops.state_compact(torch.zeros(4, 4), torch.zeros(4, dtype=torch.bool))
