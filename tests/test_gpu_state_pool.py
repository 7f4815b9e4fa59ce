"""Copies, forks, freeing and compaction of the states of a pool. States move and are not computed
with, so every comparison is for equality (a change of type rounds as torch does)."""
import pytest
import torch

from oracle import speculative as sp

pytestmark = pytest.mark.gpu
BAD_INDEX = 8


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_linear_attention_gb300 import build, sala_gla
    build.build()
    return sala_gla


def _pool(L, P, H, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(L, P, H, 128, 128, generator=gen).to(dtype)


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("src_type,dst_type", [(F, F), (F, B), (B, F), (B, B)])
@pytest.mark.parametrize("L,H,n", [(1, 1, 1), (3, 5, 4), (2, 32, 7)])
def test_copy_between_pools(sg, L, H, n, src_type, dst_type):
    a, b = _pool(L, 9, H, src_type, 1), _pool(L, 12, H, dst_type, 2)
    a[0, 0, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), -0.0])
    src = torch.arange(n) % 9
    src[-1] = 0                                     # a source may serve several pairs
    dst = torch.randperm(12, generator=torch.Generator().manual_seed(3))[:n]
    d = b.cuda()
    sg.state_pool_copy(d, a.cuda(), dst.to(torch.int32).cuda(), src.to(torch.int32).cuda())
    assert sg.get_device_status() == 0
    want = b.clone()
    want[:, dst] = a[:, src].to(dst_type)
    got = d.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("dtype", [F, B])
def test_copy_within_a_pool_clears_and_skips(sg, dtype):
    a = _pool(2, 8, 3, dtype, 4)
    d = a.cuda()
    sg.state_pool_copy(d, d, _i32(1, 6, -1, 4, 3), _i32(0, 0, 2, -1, 3))   # 3 onto itself: nothing to do
    assert sg.get_device_status() == 0
    want = a.clone()
    want[:, 1] = want[:, 6] = a[:, 0]
    want[:, 4] = 0
    assert torch.equal(d.cpu(), want)
    one = a[0].cuda()                                # one layer: [P, H, 128, 128]
    sg.state_pool_copy(one, one, _i32(5), _i32(2))
    assert torch.equal(one.cpu()[5], a[0, 2])


def test_copy_reports_pairs_that_clash(sg):
    a = _pool(1, 6, 2, F, 5)
    for dst, src, kept in (((1, 6), (0, 2), [(1, 0)]), ((1, 3), (0, 6), [(1, 0)]),
                           ((1, 1), (0, 2), [(1, 0)]),            # the first pair of a destination counts
                           ((1, 2), (0, 1), [(2, 1)])):           # a slot that is read is not written
        d = a.cuda()
        sg.state_pool_copy(d, d, _i32(*dst), _i32(*src))
        assert sg.get_device_status() == BAD_INDEX
        want = a.clone()
        for t, f in kept:
            want[:, t] = a[:, f]
        assert torch.equal(d.cpu(), want), (dst, src)
    d = a.cuda()
    other = a.cuda() + 1
    sg.state_pool_copy(d, other, _i32(1, 2), _i32(0, 1))          # two pools: no clash
    assert sg.get_device_status() == 0
    assert torch.equal(d.cpu()[:, 1:3], (a + 1)[:, :2])


@pytest.mark.parametrize("n", [300, 1500])
def test_copy_of_many_slots(sg, n):
    a = _pool(1, 2 * n, 1, B, 6)
    order = torch.randperm(2 * n, generator=torch.Generator().manual_seed(7))
    d = a.cuda()
    sg.state_pool_copy(d, d, order[:n].to(torch.int32).cuda(), order[n:].to(torch.int32).cuda())
    assert sg.get_device_status() == 0
    want = a.clone()
    want[:, order[:n]] = a[:, order[n:]]
    assert torch.equal(d.cpu(), want)


def test_copy_of_more_states_than_a_grid_has_rows(sg):
    d = torch.zeros(2, 65540, 128, 128, dtype=B, device="cuda")     # two slots of 65540 heads
    d[0] = torch.arange(65540, device="cuda", dtype=torch.int32).remainder(251).to(B)[:, None, None]
    sg.state_pool_copy(d, d, _i32(1), _i32(0))
    assert torch.equal(d[0], d[1]) and sg.get_device_status() == 0


def _fork(sg, a, used, parents, status=0):
    d, u = a.cuda(), used.cuda()
    kids = sg.state_pool_fork(d, u, parents.cuda()).tolist()
    assert sg.get_device_status() == status
    want_kids, want_used = sp.fork(used.tolist(), parents.tolist())
    assert kids == want_kids
    assert [int(x != 0) for x in u.tolist()] == want_used
    want = a.clone()
    for p, k in zip(parents.tolist(), kids):
        if k >= 0:
            want[:, k] = a[:, p] if p >= 0 else 0
    assert torch.equal(d.cpu(), want)
    return kids


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("L,P,H,n", [(1, 1, 1, 1), (2, 7, 3, 3), (3, 33, 2, 20), (1, 64, 4, 64)])
def test_fork(sg, L, P, H, n, dtype):
    gen = torch.Generator().manual_seed(P + n)
    used = (torch.rand(P, generator=gen) < 0.4).to(torch.int32) * 3    # any nonzero value is "in use"
    used[0] = P > 1
    live = used.nonzero()[:, 0]
    parents = torch.full((n,), -1, dtype=torch.int32)
    if live.numel():
        pick = live[torch.randint(0, live.numel(), (n,), generator=gen)].to(torch.int32)
        parents = torch.where(torch.rand(n, generator=gen) < 0.6, pick, parents)
    parents[n // 2] = -2                                                # padding
    _fork(sg, _pool(L, P, H, dtype, 8), used, parents)


def test_fork_of_a_full_pool_and_of_bad_parents(sg):
    a = _pool(1, 5, 1, F, 9)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    assert _fork(sg, a, i(1, 1, 1, 1, 1), i(0, -1, 2)) == [-1, -1, -1]
    assert _fork(sg, a, i(1, 0, 1, 1, 1), i(0, -1, 2)) == [1, -1, -1]
    # a parent that is free (it would be handed out itself) or past the pool
    assert _fork(sg, a, i(1, 0, 1, 0, 0), i(1, 0, 5, -1), status=BAD_INDEX) == [-1, 1, -1, 3]


def test_plans_over_many_slots(sg):
    # more slots and requests than the plan's CTA has threads
    gen = torch.Generator().manual_seed(11)
    P = 5000
    used = (torch.rand(P, generator=gen) < 0.5).to(torch.int32)
    a = torch.randn(1, P, 1, 1, 1, generator=gen).to(B).expand(1, P, 1, 128, 128).contiguous()
    live = used.nonzero()[:, 0]
    parents = live[torch.randint(0, live.numel(), (2300,), generator=gen)].to(torch.int32)
    parents[::7] = -1
    parents[5::11] = -3
    _fork(sg, a, used, parents)
    _compact(sg, a, used)


def test_free(sg):
    used = _i32(1, 1, 0, 5, 1)
    sg.state_pool_free(used, _i32(3, -1, 0))
    assert sg.get_device_status() == 0 and used.tolist() == [0, 1, 0, 0, 1]
    for bad in ((2,), (5,), (1, 1), (4, 0)):
        u = _i32(0, 1, 0, 0, 1)
        sg.state_pool_free(u, _i32(*bad))
        assert sg.get_device_status() == BAD_INDEX
        assert u.tolist() == [0 if s in bad else x for s, x in enumerate([0, 1, 0, 0, 1])]


def _compact(sg, a, used):
    d, u = a.cuda(), used.cuda()
    mapping, live = sg.state_pool_compact(d, u)
    assert sg.get_device_status() == 0
    moves, want_map, m = sp.compact(used.tolist())
    assert live.tolist() == [m] and mapping.tolist() == want_map
    assert u.tolist() == [1] * m + [0] * (len(want_map) - m)
    want = a.clone()
    for f, t in moves:
        want[:, t] = a[:, f]
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("L,P,H,share", [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (2, 9, 3, 0.5), (1, 53, 5, 0.65),
                                         (3, 16, 2, 0.0), (3, 16, 2, 1.0), (1, 2, 1, 0.5)])
def test_compact(sg, L, P, H, share, dtype):
    used = (torch.rand(P, generator=torch.Generator().manual_seed(P)) < share).to(torch.int32) * 2
    if share == 0.5:
        used[0], used[-1] = 0, 2
    _compact(sg, _pool(L, P, H, dtype, 12), used)


def test_far_slots_of_a_large_pool(sg):
    # a layer stride past 2^31 elements: two layers of 4100 slots of 32 heads in bf16 (8.6 GB)
    P = 2 ** 31 // (32 * 128 * 128) + 4
    pool = torch.zeros(2, P, 32, 128, 128, dtype=B, device="cuda")
    pool[:, P - 1] = torch.randn(2, 32, 128, 128, device="cuda").to(B)
    used = torch.zeros(P, dtype=torch.int32, device="cuda")
    used[P - 1] = 1
    kids = sg.state_pool_fork(pool, used, _i32(P - 1))
    assert kids.tolist() == [0] and torch.equal(pool[:, 0], pool[:, P - 1])
    sg.state_pool_copy(pool, pool, _i32(P - 3), _i32(P - 1))
    assert torch.equal(pool[:, P - 3], pool[:, P - 1])
    assert sg.get_device_status() == 0 and int((pool[:, 1:P - 3] != 0).sum()) == 0


def test_graph_and_side_stream(sg):
    a = _pool(2, 12, 2, F, 13)
    d, used, parents = a.cuda(), _i32(*([1] * 4 + [0] * 8)), _i32(3, -1, 1)
    kids, done = torch.empty(3, dtype=torch.int32, device="cuda"), _i32(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m, live = sg.state_pool_compact(d, used, stream=side)
    side.synchronize()
    assert live.tolist() == [4] and m.tolist() == [0, 1, 2, 3] + [-1] * 8 and torch.equal(d.cpu(), a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.state_pool_free(used, done)
        sg.state_pool_fork(d, used, parents, children=kids)
    graph.replay()
    assert kids.tolist() == [0, 4, 5]
    done.copy_(kids[1:2])                              # the same graph on another occupancy
    graph.replay()
    assert kids.tolist() == [4, 6, 7] and torch.equal(d.cpu()[:, 4], a[:, 3])
    assert sg.get_device_status() == 0
