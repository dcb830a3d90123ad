"""Forking, trimming and compacting the pages of a paged cache against plain
list implementations (needs a B200). Everything is exact."""

import random

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    import kv_cache_vector_turboquant_b200 as K

    return K


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pools(nb, layers, hkv, pk, pv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        out += [torch.randint(0, 256, (nb, 16, hkv, pk), generator=g, device="cuda", dtype=torch.uint8),
                torch.randn(nb, 16, hkv, generator=g, device="cuda"),
                torch.randint(0, 256, (nb, 16, hkv, pv), generator=g, device="cuda", dtype=torch.uint8),
                torch.randn(nb, 16, hkv, generator=g, device="cuda")]
    return out


def _moved(pools, moves):
    out = [t.clone() for t in pools]
    for s, d in moves:
        for t, o in zip(pools, out):
            o[d] = t[s]
    return out


def _state(rng, rows, mb, nb, live):
    """Rows of random lengths on random pages, the first `live` of them in use."""
    free = list(range(nb))
    rng.shuffle(free)
    table, lens, refs = [[-1] * mb for _ in range(rows)], [0] * rows, [0] * nb
    for r in range(live):
        n = rng.randint(0, min(mb, len(free)))
        lens[r] = max(0, 16 * n - rng.choice([0, 0, rng.randint(0, 15)])) if n else 0
        for j in range((lens[r] + 15) // 16):
            table[r][j] = free.pop()
            refs[table[r][j]] = 1
    return table, lens, refs


FORKS = [
    # rows, max_blocks, num_blocks, live rows, forks, layers, hkv, P_K, P_V
    (4, 1, 5, 1, 1, 1, 1, 16, 16),
    (10, 7, 60, 5, 5, 2, 2, 64, 32),
    (40, 5, 50, 12, 28, 1, 3, 24, 96),       # parents forked many times, the pool runs out
    (300, 130, 9000, 100, 200, 1, 1, 48, 16),
    (2100, 3, 7000, 1000, 1100, 1, 1, 16, 16),   # more forks than planning threads
]


@pytest.mark.parametrize("rows,mb,nb,live,n,layers,hkv,pk,pv", FORKS)
@pytest.mark.parametrize("inplace", [False, True])
def test_fork(K, rows, mb, nb, live, n, layers, hkv, pk, pv, inplace):
    rng = random.Random(rows * 7 + mb)
    table, lens, refs = _state(rng, rows, mb, nb, live)
    parents = [rng.randrange(live) for _ in range(n)]
    children = rng.sample(range(live, rows), n)
    pools = _pools(nb, layers, hkv, pk, pv, rows)
    rt, rl, rr, moves, skipped, full = R.fork(table, lens, refs, parents, children)
    expect = _moved(pools, moves)
    K.tq_device_error()
    t, l, r = _i32(table), _i32(lens), _i32(refs)
    out = (t, l, r) if inplace else None
    before = [x.clone() for x in (t, l, r)]
    got = K.TQPagePools(pools).fork(t, l, r, _i32(parents), _i32(children), out=out)
    torch.cuda.synchronize()
    for a, b in zip(got, (rt, rl, rr)):
        assert torch.equal(a, _i32(b))
    if not inplace:
        assert all(torch.equal(a, b) for a, b in zip((t, l, r), before))
    for a, b in zip(pools, expect):
        assert torch.equal(a, b)
    assert skipped == 0
    assert K.tq_device_error()[1] == (K.TQ_DEVERR_POOL_FULL if full else 0)


def test_fork_of_the_largest_table(K):
    """As many rows as a call takes, forks at both ends of the table."""
    rows, nb = K.TQ_MAX_PAGE_ROWS, 40
    table, lens, refs = [[-1] for _ in range(rows)], [0] * rows, [0] * nb
    for r, page, length in ((0, 7, 5), (1, 3, 16), (rows - 2, 30, 9)):
        table[r], lens[r], refs[page] = [page], length, 1
    parents, children = [0, 1, rows - 2, 0], [rows - 1, rows // 2, 2, rows - 3]
    pools = _pools(nb, 1, 1, 16, 16, 3)
    rt, rl, rr, moves, _, _ = R.fork(table, lens, refs, parents, children)
    expect = _moved(pools, moves)
    K.tq_device_error()
    got = K.TQPagePools(pools).fork(_i32(table), _i32(lens), _i32(refs), _i32(parents), _i32(children))
    for a, b in zip(got, (rt, rl, rr)):
        assert torch.equal(a, _i32(b))
    assert all(torch.equal(a, b) for a, b in zip(pools, expect))
    assert K.tq_device_error() == (K.TQ_OK, 0)


def test_no_forks(K):
    """An empty list copies the tables, or does nothing in place."""
    rng = random.Random(5)
    t, l, r = (_i32(x) for x in _state(rng, 5, 3, 20, 3))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    h = K.TQPagePools(_pools(20, 1, 1, 16, 16, 1))
    for out in (None, (t, l, r)):
        got = h.fork(t, l, r, none, none, out=out)
        assert all(torch.equal(a, b) for a, b in zip(got, (t, l, r)))
    assert K.tq_device_error() == (K.TQ_OK, 0)


def test_fork_skips_and_flags_impossible_pairs(K):
    rng = random.Random(5)
    table, lens, refs = _state(rng, 12, 4, 40, 6)
    #  child named twice, child that is a parent, parent and child outside, one good one
    parents = [0, 1, 2, 99, 3, -1, 4]
    children = [7, 7, 4, 8, 12, 9, 10]
    pools = _pools(40, 1, 1, 16, 16, 1)
    rt, rl, rr, moves, skipped, _ = R.fork(table, lens, refs, parents, children)
    assert skipped == 6
    expect = _moved(pools, moves)
    K.tq_device_error()
    got = K.TQPagePools(pools).fork(_i32(table), _i32(lens), _i32(refs), _i32(parents), _i32(children))
    torch.cuda.synchronize()
    for a, b in zip(got, (rt, rl, rr)):
        assert torch.equal(a, _i32(b))
    assert all(torch.equal(a, b) for a, b in zip(pools, expect))
    assert K.tq_device_error() == (K.TQ_ERR_DEVICE, K.TQ_DEVERR_ROW_RANGE)


def test_fork_of_bad_tables_and_lengths_is_bounded(K):
    """Entries and lengths outside their ranges: dropped and flagged, nothing read outside."""
    pools = _pools(4, 1, 1, 16, 16, 2)
    table = [[7, 0, 1], [2, 99, -5], [-1, -1, -1], [-1, -1, -1], [0, 1, 9], [-1, -1, -1]]
    lens, refs = [33, 1000, 0, -4, 40, 0], [2, 2, 1, 0]
    K.tq_device_error()
    got = K.TQPagePools(pools).fork(_i32(table), _i32(lens), _i32(refs), _i32([0, 1, 4]), _i32([2, 3, 5]))
    torch.cuda.synchronize()
    # row 0: entry 7 dropped, page 0 shared, page 1 copied; row 1 clamped to 48
    # positions: page 2 shared, 99 and -5 dropped; row 4: 0, 1 shared, 9 dropped
    assert got[0].tolist() == [table[0], table[1], [-1, 0, 3], [2, -1, -1], table[4], [0, 1, -1]]
    assert got[1].tolist() == [33, 1000, 33, 48, 40, 40]
    assert got[2].tolist() == [4, 3, 2, 1]
    st, bits = K.tq_device_error()
    assert bits == K.TQ_DEVERR_BLOCK_RANGE | K.TQ_DEVERR_POS_RANGE


TRIMS = [(1, 1, 16, 0), (3, 9, 20, 4), (5, 33, 1, 0), (17, 64, 100, 17), (4, 8, 0, 0), (4, 8, None, 0), (60, 131, 900, 33)]


@pytest.mark.parametrize("rows,mb,window,sinks", TRIMS)
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("release", [False, True])
def test_trim(K, rows, mb, window, sinks, inplace, release):
    rng = random.Random(rows * mb)
    nb = rows * mb + 3
    table = [[rng.choice([-1, rng.randrange(nb)]) for _ in range(mb)] for _ in range(rows)]
    refs = [0] * nb
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    lens = [rng.randint(0, 16 * mb) for _ in range(rows)]
    rel = [rng.random() < 0.3 for _ in range(rows)] if release else None
    ref = R.trim(table, lens, refs, window, sinks, rel)
    t, l, r = _i32(table), _i32(lens), _i32(refs)
    mask = torch.tensor(rel, device="cuda") if release else None
    got = K.pages_trim(t, l, r, window=window, sinks=sinks, release=mask, out=(t, l, r) if inplace else None)
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, _i32(b))
    assert K.tq_device_error() == (K.TQ_OK, 0)


COMPACTS = [
    # rows, max_blocks, num_blocks, share used
    (1, 1, 1, 1.0), (1, 2, 1, 0.0), (3, 5, 33, 0.5), (8, 16, 200, 0.0), (8, 16, 200, 1.0), (9, 64, 4096, 0.3),
    (9, 64, 4097, 0.7), (30, 100, 8192, 0.9), (5, 50, 8193, 0.02), (5, 50, 40001, 0.5),
]


@pytest.mark.parametrize("rows,mb,nb,share", COMPACTS)
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(K, rows, mb, nb, share, inplace):
    rng = random.Random(nb)
    refs = [rng.randint(1, 3) if rng.random() < share else rng.choice([0, 0, -1]) for _ in range(nb)]
    used = [b for b, r in enumerate(refs) if r > 0]
    table = [[rng.choice(used) if used and rng.random() < 0.8 else rng.choice([-1, -7, rng.randrange(nb)])
              for _ in range(mb)] for _ in range(rows)]
    pools = _pools(nb, 1, 1, 24, 16, nb)
    rt, rr, rm, ru, moves = R.compact(table, refs)
    expect = [t.clone() for t in pools]
    if moves:
        s, d = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for t, o in zip(pools, expect):
            o[d] = t[s]
    t, r = _i32(table), _i32(refs)
    out = None
    if inplace:
        out = (t, r, torch.empty_like(r), torch.empty(1, dtype=torch.int32, device="cuda"))
    got = K.TQPagePools(pools).compact(t, r, out=out)
    torch.cuda.synchronize()
    for a, b in zip(got, (rt, rr, rm, [ru])):
        assert torch.equal(a, _i32(b))
    for a, b in zip(pools, expect):
        assert torch.equal(a, b)
    assert K.tq_device_error() == (K.TQ_OK, 0)


def test_compact_drops_and_flags_entries_past_the_pool(K):
    pools = _pools(3, 1, 1, 16, 16, 3)
    got = K.TQPagePools(pools).compact(_i32([[0, 2, 3, 1 << 30]]), _i32([0, 0, 1]))
    torch.cuda.synchronize()
    assert got[0].tolist() == [[-1, 0, -1, -1]] and got[1].tolist() == [1, 0, 0]
    assert got[2].tolist() == [-1, -1, 0] and got[3].tolist() == [1]
    assert K.tq_device_error() == (K.TQ_ERR_DEVICE, K.TQ_DEVERR_BLOCK_RANGE)


def test_large_pages_many_pools_and_replay(K):
    """Pages of several units in many pools (views of stacked layers), forked
    and compacted from a captured graph whose replay sees new tables."""
    nb, layers = 40, 9
    k = torch.randint(0, 256, (layers, nb, 16, 8, 64), device="cuda", dtype=torch.uint8)
    n = torch.randn(layers, nb, 16, 8, device="cuda")
    pools = [*k.unbind(0), *n.unbind(0)]
    h = K.TQPagePools(pools)
    rng = random.Random(11)
    state = _state(rng, 12, 4, nb, 6)
    t, l, r = (_i32(x) for x in state)
    p, c = _i32([0, 1, 2]), _i32([7, 9, 11])
    o1 = tuple(torch.empty_like(x) for x in (t, l, r))
    o2 = (torch.empty_like(t), torch.empty_like(r), torch.empty_like(r), torch.empty(1, dtype=torch.int32, device="cuda"))
    w1 = torch.empty(K.tq_pages_fork_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(K.tq_pages_compact_workspace_bytes(nb), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h.fork(t, l, r, p, c, out=o1, workspace=w1)
        h.compact(o1[0], o1[2], out=o2, workspace=w2)
    for seed in (12, 13):
        state = _state(random.Random(seed), 12, 4, nb, 6)
        for x, y in zip((t, l, r), state):
            x.copy_(_i32(y))
        ft, fl, fr, moves, _, _ = R.fork(*state, [0, 1, 2], [7, 9, 11])
        expect = _moved(pools, moves)
        ct, cr, cm, cu, moves = R.compact(ft, fr)
        expect = _moved(expect, moves)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*o1, *o2), (ft, fl, fr, ct, cr, cm, [cu])):
            assert torch.equal(a, _i32(b))
        for a, b in zip(pools, expect):
            assert torch.equal(a, b)
    assert K.tq_device_error() == (K.TQ_OK, 0)
