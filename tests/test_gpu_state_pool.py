"""GPU: copying, forking, freeing and compacting slots of a state pool.  Results are copies, so
they have to be equal bit for bit."""
import pytest
import torch

import delta_ref as ref
from wkv_recurrence_02_b200 import ops

pytestmark = pytest.mark.gpu


def _pool(shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _copy(pool, src, dst, slot_dim=0):
    got = pool.cuda()
    ops.state_copy(got, _i32(src), _i32(dst), slot_dim=slot_dim)
    assert torch.equal(got.cpu(), ref.copied(pool, src, dst, slot_dim))


@pytest.mark.parametrize("src,dst", [
    ([0], [1]), ([], []), ([3], [3]),                       # one, none, a slot onto itself
    ([0, 1], [1, 0]), ([0, 1, 2, 3], [1, 2, 3, 0]),         # swap, cycle
    ([0, 1, 2], [1, 2, 3]), ([1, 2, 3], [0, 1, 2]),         # shifts
    ([2, 2, 2, 5], [0, 1, 3, 4]),                           # forks
    ([-1, -1], [4, 2]), ([1, -1], [3, 1]),                  # frees; free a source
    ([1, 2, 4], [0, 0, 0]), ([1, -1], [0, 0]), ([2, 0], [0, 0]),  # one destination: the last counts
    ([0, 1, -5], [-1, 2, -1]),                              # pairs left out
])
@pytest.mark.parametrize("shape,dim", [((6, 4), 0), ((6, 1000), 0), ((3, 6, 2, 64, 64), 1), ((6, 12004), 0)])
def test_copy_pairs(src, dst, shape, dim):
    _copy(_pool(shape), src, dst, dim)


@pytest.mark.parametrize("n,P,e", [(300, 700, 100), (4096, 5000, 4), (1000, 1200, 2052), (33, 40, 70000)])
def test_copy_many(n, P, e):
    gen = torch.Generator().manual_seed(n)
    src = torch.randint(-1, P, (n,), generator=gen).tolist()
    dst = torch.randint(-1, P, (n,), generator=gen).tolist()
    _copy(_pool((P, e)), src, dst)


def test_copy_bf16_and_wkv4_states():
    _copy(_pool((5, 3, 64)), [0, 4], [2, 0])
    _copy(_pool((2, 9, 8)).to(torch.bfloat16), [0, 8], [2, 0], 1)


def test_copy_outside_the_pool_is_left_out_and_recorded():
    pool = _pool((4, 8))
    got = pool.cuda()
    assert ops.device_status() == 0
    ops.state_copy(got, _i32([4, 1, 2]), _i32([0, 4, 3]))
    assert ops.device_status() == -8
    assert torch.equal(got.cpu(), ref.copied(pool, [4, 1, 2], [0, 4, 3]))
    assert ops.device_status() == 0


@pytest.mark.parametrize("shape,dim", [((1, 4), 0), ((7, 260), 0), ((3, 33, 5, 64, 64), 1), ((256, 2, 64, 64), 0),
                                       ((300, 8), 0), ((5000, 4), 0)])
@pytest.mark.parametrize("p", [0.0, 0.3, 0.9, 1.0])
def test_compact(shape, dim, p):
    pool = _pool(shape)
    gen = torch.Generator().manual_seed(int(100 * p) + shape[0])
    live = torch.rand(shape[dim], generator=gen) < p
    got = pool.cuda()
    index, count = ops.state_compact(got, live.cuda(), slot_dim=dim)
    new, ri, rn = ref.compacted(pool, live.tolist(), dim)
    assert torch.equal(got.cpu(), new) and index.tolist() == ri and count.tolist() == [rn]


@pytest.mark.parametrize("live", [[0, 0, 1], [1, 0, 0], [0, 1, 0], [255, 0, 2]])
def test_compact_uint8(live):
    pool = _pool((3, 16))
    got = pool.cuda()
    index, count = ops.state_compact(got, torch.tensor(live, dtype=torch.uint8, device="cuda"))
    new, ri, rn = ref.compacted(pool, live)
    assert torch.equal(got.cpu(), new) and index.tolist() == ri and count.item() == rn


def test_compact_largest_pool():
    pool = _pool((16384, 4))
    live = torch.rand(16384, generator=torch.Generator().manual_seed(1)) < 0.5
    got = pool.cuda()
    index, count = ops.state_compact(got, live.cuda())
    new, ri, rn = ref.compacted(pool, live.tolist())
    assert torch.equal(got.cpu(), new) and index.tolist() == ri and count.item() == rn


@pytest.mark.parametrize("shape,dim", [((0, 7, 4), 1), ((7, 0), 0), ((2, 7, 0, 64), 1), ((0, 4), 0), ((0, 0, 4), 1)])
def test_compact_pools_without_bytes(shape, dim):
    """No layers, empty slots or no slots: nothing moves, and the places are still told."""
    P = shape[dim]
    live = [i % 3 != 1 for i in range(P)]
    pool = torch.empty(shape, device="cuda")
    index, count = ops.state_compact(pool, torch.tensor(live, dtype=torch.bool, device="cuda"), slot_dim=dim)
    assert index.tolist() == [sum(live[:i]) if x else -1 for i, x in enumerate(live)]
    assert count.tolist() == [sum(live)] and ops.device_status() == 0
    one = _i32([0])
    ops.state_copy(pool, one, one, slot_dim=dim)
    assert ops.device_status() == 0


def test_copy_and_compact_replayed_in_a_graph():
    """Captured once, replayed over new indices: the calls read them from the device."""
    pool = _pool((2, 12, 512))
    got, src, dst = pool.cuda(), _i32([0, 0]), _i32([1, 2])
    live = torch.ones(12, dtype=torch.bool, device="cuda")
    ops.state_copy(got, src, dst, slot_dim=1)
    ops.state_compact(got, live, slot_dim=1)
    got.copy_(pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.state_copy(got, src, dst, slot_dim=1)
        index, count = ops.state_compact(got, live, slot_dim=1)
    want = pool
    for s, d, out in (([3, 4], [4, 3], [0, 5]), ([-1, 7], [0, 9], [2])):
        mask = torch.ones(12, dtype=torch.bool)
        mask[out] = False
        src.copy_(_i32(s)), dst.copy_(_i32(d)), live.copy_(mask)
        graph.replay()
        want, ri, rn = ref.compacted(ref.copied(want, s, d, 1), mask.tolist(), 1)
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want) and index.tolist() == ri and count.item() == rn


@pytest.mark.parametrize("shape,dim", [((3, 40, 5, 64), 1), ((6, 12004), 0), ((200, 2, 64, 64), 0)])
def test_a_wait_that_runs_out_moves_nothing(shape, dim):
    lib = ops.load()
    pool, P = _pool(shape), shape[dim]
    got = pool.cuda()
    src, dst = list(range(P)), [(i + 1) % P for i in range(P)]
    live = torch.arange(P) % 3 != 0
    assert ops.device_status() == 0
    prev = lib.rwkv_debug_inject_timeout(1)
    try:
        for call in (lambda: ops.state_copy(got, _i32(src), _i32(dst), slot_dim=dim),
                     lambda: ops.state_compact(got, live.cuda(), slot_dim=dim)):
            call()
            assert ops.device_status() == -6
            assert torch.equal(got.cpu(), pool)
    finally:
        lib.rwkv_debug_inject_timeout(prev)
    _copy(pool, src, dst, dim)
    index, count = ops.state_compact(got, live.cuda(), slot_dim=dim)
    new, ri, rn = ref.compacted(pool, live.tolist(), dim)
    assert torch.equal(got.cpu(), new) and index.tolist() == ri and count.tolist() == [rn]
    assert ops.device_status() == 0


def test_binding_refusals():
    pool = _pool((4, 8)).cuda()
    with pytest.raises(TypeError):
        ops.state_copy(pool, torch.zeros(1, dtype=torch.int64, device="cuda"), _i32([0]))
    with pytest.raises(ValueError):
        ops.state_copy(pool, _i32([0, 1]), _i32([0]))
    with pytest.raises(ValueError):
        ops.state_copy(pool.t(), _i32([0]), _i32([1]))
    with pytest.raises(ValueError):
        ops.state_copy(pool, _i32([0]), _i32([1]), slot_dim=2)
    with pytest.raises(ops.WkvError):
        ops.state_copy(pool[:, :3].contiguous(), _i32([0]), _i32([1]))  # 12-byte slots
    with pytest.raises(ValueError):
        ops.state_compact(pool, torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError):
        ops.state_compact(pool, torch.ones(4, device="cuda"))
