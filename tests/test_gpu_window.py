"""Windowed attention over packed caches against the oracle's decoded rows and
a plain 64-bit attention (needs a B200)."""

import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    import kv_cache_vector_turboquant_b200 as K

    return K


def _cache(K, shape, d, bits, seed, spread=0.2):
    """Packed rows of N(0,1) vectors of varied norms."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, d, generator=g, device="cuda")
    x = x * torch.exp(spread * torch.randn(*shape, 1, generator=g, device="cuda"))
    codec = K.TurboQuant(d, bits)
    return codec, *codec.encode(x.half())


def _pages(t, ctx, table_seed, spare=2):
    """[B, S, ...] rows -> (pool, table) with scattered pages."""
    B, S = t[0].shape[:2]
    mb = (S + 15) // 16
    perm = torch.randperm(B * mb + spare, generator=torch.Generator().manual_seed(table_seed))[:B * mb]
    pools = []
    for x in t:
        pad = torch.zeros(B, mb * 16, *x.shape[2:], dtype=x.dtype, device=x.device)
        pad[:, :S] = x
        pool = torch.zeros(B * mb + spare, 16, *x.shape[2:], dtype=x.dtype, device=x.device)
        pool[perm.cuda()] = pad.view(B * mb, 16, *x.shape[2:])
        pools.append(pool)
    return pools, perm.view(B, mb).int().cuda()


def _check(o, ref, tol):
    err = (o.cpu().double() - ref).norm(dim=-1)
    assert torch.isfinite(o).all()
    assert (err <= tol).all(), (err / tol.clamp(min=1e-30)).max().item()


CASES = [
    # d, kb, vb, hq, hkv, S, [(query tokens, context)], window, sinks
    (128, 4, 2, 32, 8, 70, [(1, 70), (1, 1), (1, 33)], None, 0),
    (128, 4, 2, 32, 8, 150, [(1, 150), (1, 17), (1, 64)], 40, 4),
    (128, 4, 2, 4, 1, 300, [(1, 300)], 1, 0),             # a window of the token itself
    (128, 4, 2, 4, 1, 300, [(1, 300), (1, 299)], 1, 1),
    (128, 4, 2, 4, 1, 300, [(1, 300)], 100, 200),         # sinks and window meet
    (128, 4, 2, 4, 1, 300, [(1, 300)], 100, 1000),        # every position a sink
    (128, 4, 4, 16, 4, 90, [(5, 90), (3, 60), (4, 4), (1, 90)], None, 0),
    (128, 3, 3, 6, 2, 90, [(5, 90), (0, 60), (7, 20)], 16, 3),
    (64, 2, 3, 5, 1, 100, [(2, 100), (9, 50)], 33, 17),
    (64, 3, 2, 12, 12, 47, [(1, 47), (2, 33)], 15, 0),
    (64, 4, 4, 9, 3, 64, [(1, 64), (1, 48), (1, 16)], 16, 16),
    (64, 3, 3, 1, 1, 33, [(33, 33)], None, 0),
    (256, 4, 2, 8, 1, 70, [(1, 70), (1, 64)], 30, 2),
    (256, 2, 4, 10, 2, 40, [(3, 40)], None, 0),
    (256, 3, 3, 4, 4, 35, [(2, 35), (2, 2)], 9, 1),
    (128, 2, 2, 13, 1, 40, [(3, 40)], 17, 5),             # odd group of query heads
    (128, 4, 2, 7, 7, 18, [(18, 18), (2, 9)], 5, 2),
    (128, 4, 3, 8, 2, 260, [(130, 260), (40, 41), (1, 200)], 60, 20),
    (64, 4, 2, 8, 1, 200, [(140, 200), (17, 17)], None, 0),
    (256, 4, 4, 4, 1, 150, [(70, 150)], 50, 3),
    # 40 to 128 query rows per kv head over long contexts
    (128, 4, 2, 32, 8, 1100, [(16, 1100), (11, 64), (1, 700), (0, 5), (16, 129)], None, 0),
    (128, 3, 4, 8, 1, 900, [(16, 900), (16, 16)], 700, 70),
    (64, 2, 2, 40, 1, 1500, [(3, 1500), (1, 65), (2, 1409)], None, 3),
    (128, 4, 3, 5, 1, 1029, [(25, 1029)], None, 0),
]


@pytest.mark.parametrize("d,kb,vb,hq,hkv,S,seqs,window,sinks", CASES)
@pytest.mark.parametrize("scale", [0.0, 0.7])
def test_matches_plain_attention(K, d, kb, vb, hq, hkv, S, seqs, window, sinks, scale):
    """Query scale 0 weighs every visible position the same: a position too
    many or too few shows against the small tolerance of that case."""
    B = len(seqs)
    kc, kp, kn = _cache(K, (B, S, hkv), d, kb, d + S)
    vc, vp, vn = _cache(K, (B, S, hkv), d, vb, d + S + 1)
    n = [a for a, _ in seqs]
    off = np.concatenate([[0], np.cumsum(n)])
    q = (scale * torch.randn(int(off[-1]), hq, d, generator=torch.Generator(device="cuda").manual_seed(S),
                             device="cuda")).half()
    ctx = torch.tensor([c for _, c in seqs], dtype=torch.int32, device="cuda")
    args = {"window": window, "sinks": sinks}
    if n != [1] * B:
        args |= {"q_offsets": torch.tensor(off, dtype=torch.int32, device="cuda"), "max_q": max(n)}
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, **args)
    # paged, with the entries that no query sees taken out
    (kq, knq, vq, vnq), table = _pages((kp, kn, vp, vn), ctx, S)
    for b, (m, c) in enumerate(seqs):
        seen = {t // 16 for i in range(m) for t in range(c - m + i + 1)
                if t < sinks or window is None or t > c - m + i - window}
        for j in set(range(table.shape[1])) - seen:
            table[b, j] = -1 if j % 2 else 1 << 30
    op = K.attend_window_paged(q, kc, vc, kq, knq, vq, vnq, table, ctx, **args)
    torch.cuda.synchronize()
    assert K.tq_device_error() == (K.TQ_OK, 0)
    for b, (m, c) in enumerate(seqs):
        if not m:
            continue
        kk = R.decode_rows(kp[b, :c], kn[b, :c], kb, d)
        vv = R.decode_rows(vp[b, :c], vn[b, :c], vb, d)
        ref, tol = R.attend(q[off[b]:off[b + 1]], kk, vv, c, window, sinks, kb, vb)
        _check(o[off[b]:off[b + 1]], ref, tol)
        _check(op[off[b]:off[b + 1]], ref, tol)


@pytest.mark.parametrize("n,S,window,sinks", [(1, 3000, 700, 33), (6, 2500, None, 0), (300, 2100, 500, 40)])
@pytest.mark.parametrize("d,kb,vb", [(128, 4, 2), (64, 3, 4), (256, 4, 4)])
def test_long_contexts_sampled(K, n, S, window, sinks, d, kb, vb):
    """Many blocks per split and, with 300 tokens, many query tiles; two heads of each group checked."""
    hq, hkv, B = 8, 2, 2
    kc, kp, kn = _cache(K, (B, S, hkv), d, kb, 5)
    vc, vp, vn = _cache(K, (B, S, hkv), d, vb, 6)
    q = (0.5 * torch.randn(B * n, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))).half()
    lens = [S, S - 777]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, window=window, sinks=sinks, q_offsets=off, max_q=n)
    heads, rows = [0, 3, 4, 7], sorted({0, n // 3, n - 1})
    for b in range(B):
        kk, vv = R.decode_rows(kp[b], kn[b], kb, d), R.decode_rows(vp[b], vn[b], vb, d)
        for i in rows:
            c = lens[b] - n + i + 1  # as a single query at that position
            ref, tol = R.attend(q[b * n + i][None, heads], kk[:, [0, 1]], vv[:, [0, 1]], c, window, sinks, kb, vb)
            _check(o[b * n + i][None, heads], ref, tol)
    assert K.tq_device_error() == (K.TQ_OK, 0)


def test_agrees_with_the_decode_step_attention(K):
    """One token, no window: the function of tq_attend_decode, whose levels
    are rounded to fp16 as they are (2^-12)."""
    d, B, S, hq, hkv = 128, 3, 500, 32, 8
    kc, kp, kn = _cache(K, (B, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (B, S, hkv), d, 2, 2)
    q = torch.randn(B, hq, d, device="cuda").half()
    ctx = torch.tensor([500, 3, 77], dtype=torch.int32, device="cuda")
    a = K.attend_decode(q, kc, vc, kp, kn, vp, vn, ctx)
    b = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx)
    # row error of the first: scores off by 2^-12 |q| |k| / sqrt(d) each way, values by 2^-12
    vmax = vn.max().item()
    ds = 2.0 ** -12 * q.float().norm(dim=-1).max().item() * kn.max().item() / d ** 0.5
    assert ((a.float() - b.float()).norm(dim=-1) <= (3 * ds + 2.0 ** -10) * vmax).all()


def test_empty_contexts_and_unseen_tokens(K):
    d, S, hq, hkv = 128, 40, 8, 2
    kc, kp, kn = _cache(K, (4, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (4, S, hkv), d, 2, 2)
    # sequences of 2, 0, 3 and 2 tokens; the third has fewer positions than tokens; tokens 7.. are in none
    q = torch.randn(10, hq, d, device="cuda").half()
    off = torch.tensor([0, 2, 2, 5, 7], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([40, 9, 1, 0], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, window=9, sinks=2, q_offsets=off, max_q=3, out=out)
    torch.cuda.synchronize()
    assert torch.all(out[2:4] == 0) and torch.all(out[5:7] == 0) and torch.all(out[7:] == 7.0)
    assert torch.all(out[4].float().abs().sum(-1) > 0) and not torch.any(out[:2] == 7.0)
    v0 = R.decode_rows(vp[2, :1], vn[2, :1], 2, d)  # position 0 alone
    for h in range(hq):
        assert (out[4, h].cpu().double() - v0[0, h // 4]).abs().max() <= 2.0 ** -11 * v0[0, h // 4].abs().max() * 1.1
    assert K.tq_device_error() == (K.TQ_OK, 0)
    ctx = torch.tensor([-5, 0, -1, 0], dtype=torch.int32, device="cuda")
    one = K.attend_window(q[:4], kc, vc, kp, kn, vp, vn, ctx)
    assert torch.all(one == 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_with_empty_and_short_contexts(K, d):
    """The same for sequences of many query tokens (one more than a row tile of
    some, an empty one between, more tokens than positions), with a replaced
    offset row behind them left alone."""
    S, hq, hkv, kb, vb = 150, 2, 2, 4, 3
    n, lens = [129, 0, 60, 45, 41], [150, 7, 13, 0, 41]
    B = len(n)
    kc, kp, kn = _cache(K, (B, S, hkv), d, kb, 1)
    vc, vp, vn = _cache(K, (B, S, hkv), d, vb, 2)
    off = np.concatenate([[0], np.cumsum(n)])
    q = (0.5 * torch.randn(int(off[-1]) + 3, hq, d, device="cuda")).half()
    out = torch.full_like(q, 7.0)
    K.attend_window(q, kc, vc, kp, kn, vp, vn, torch.tensor(lens, dtype=torch.int32, device="cuda"), window=20, sinks=3,
                    q_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_q=129, out=out)
    torch.cuda.synchronize()
    assert K.tq_device_error() == (K.TQ_OK, 0)
    assert torch.all(out[off[-1]:] == 7.0)
    for b in range(B):
        if not n[b]:
            continue
        kk, vv = R.decode_rows(kp[b], kn[b], kb, d), R.decode_rows(vp[b], vn[b], vb, d)
        ref, tol = R.attend(q[off[b]:off[b + 1]], kk, vv, lens[b], 20, 3, kb, vb)
        _check(out[off[b]:off[b + 1]], ref, tol)
    assert torch.all(out[off[2]:off[2] + 47] == 0) and torch.all(out[off[3]:off[4]] == 0)


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_whole_row_tiles_that_see_nothing(K, d, rows):
    """Unsplit calls whose row tiles are full and see no position: contexts of
    0 and tokens before position 0. Every element is zero, every time, and the
    tokens behind them are those of a call of their own."""
    S, hq, hkv, kb, vb, seen = 40, 2, 1, 4, 2, 9
    n = rows // 2
    kc, kp, kn = _cache(K, (1, S, hkv), d, kb, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, vb, 2)
    B = 148
    lens = [0 if b % 3 else seen for b in range(B)]  # sequences of 2 n tokens: the first n see nothing
    caches = [x.expand(B, *x.shape[1:]).contiguous() for x in (kp, kn, vp, vn)]
    assert K.tq_attend_window_workspace_bytes(2 * n * B, B, 2 * n, hq, hkv, d, S, 0, 0) == 0
    q = 10 * torch.randn(2 * n, hq, d, device="cuda").half()
    some = K.attend_window(q[-seen:].contiguous(), kc, vc, kp, kn, vp, vn,
                           torch.tensor([seen], dtype=torch.int32, device="cuda"),
                           q_offsets=torch.tensor([0, seen], dtype=torch.int32, device="cuda"), max_q=seen)
    kk, vv = R.decode_rows(kp[0, :seen], kn[0, :seen], kb, d), R.decode_rows(vp[0, :seen], vn[0, :seen], vb, d)
    ref, tol = R.attend(q[-seen:], kk, vv, seen, None, 0, kb, vb)
    _check(some, ref, tol)
    args = (torch.tensor(lens, dtype=torch.int32, device="cuda"), None, 0,
            2 * n * torch.arange(B + 1, dtype=torch.int32, device="cuda"), 2 * n)
    for _ in range(20):
        out = torch.full((B * 2 * n, hq, d), 7.0, dtype=torch.float16, device="cuda")
        K.attend_window(q.repeat(B, 1, 1), kc, vc, *caches, *args, out=out)
        o = out.view(B, 2 * n, hq, d)
        assert torch.all(o[:, :-seen] == 0)
        assert torch.all(o[1::3] == 0) and torch.all(o[2::3] == 0)
        _check(o[0, -seen:], ref, tol)
        assert torch.equal(o[::3], o[:1].expand_as(o[::3]))
    assert K.tq_device_error() == (K.TQ_OK, 0)


@pytest.mark.parametrize("d,n,g", [(128, 6, 8), (64, 9, 5), (256, 4, 8), (128, 5, 8)])
@pytest.mark.parametrize("B", [1, 64])
def test_between_the_kernels(K, d, n, g, B):
    """32 to 63 query rows per kv head, where the sizes choose the kernel: one
    sequence and many of the same one."""
    S, L, hkv = 1104, 1090, 2
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    q = torch.randn(n, hkv * g, d, device="cuda").half()
    caches = [x.expand(B, *x.shape[1:]).contiguous() for x in (kp, kn, vp, vn)]
    o = K.attend_window(q.repeat(B, 1, 1), kc, vc, *caches, torch.full((B,), L, dtype=torch.int32, device="cuda"),
                        q_offsets=n * torch.arange(B + 1, dtype=torch.int32, device="cuda"), max_q=n)
    kk, vv = R.decode_rows(kp[0], kn[0], 4, d), R.decode_rows(vp[0], vn[0], 2, d)
    ref, tol = R.attend(q, kk, vv, L, None, 0, 4, 2)
    o = o.view(B, n, hkv * g, d)
    _check(o[0], ref, tol)
    assert torch.equal(o, o[:1].expand_as(o))


@pytest.mark.parametrize("n", [1, 48])
def test_output_in_place_of_the_queries(K, n):
    d, S, hq, hkv = 128, 700, 8, 2
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 4, 2)
    q = torch.randn(n, hq, d, device="cuda").half()
    args = (kc, vc, kp, kn, vp, vn, torch.tensor([S], dtype=torch.int32, device="cuda"), 300, 4,
            torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    ref = K.attend_window(q, *args)
    K.attend_window(q, *args, out=q)
    assert torch.equal(q, ref)


def test_non_finite_norms_where_no_query_looks(K):
    """Norms of NaN and infinity behind the context, outside the window and in
    unread pages leave the results as they are."""
    d, S, hq, hkv = 128, 100, 8, 2
    kc, kp, kn = _cache(K, (2, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (2, S, hkv), d, 2, 2)
    q = torch.randn(2, hq, d, device="cuda").half()
    ctx = torch.tensor([90, 35], dtype=torch.int32, device="cuda")
    ref = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, window=20, sinks=3)
    for b, c in enumerate((90, 35)):
        for x in (kn, vn):
            x[b, c:] = float("nan")
            x[b, 3:c - 20] = float("inf")
            x[b, 5] = float("nan")
    got = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, window=20, sinks=3)
    assert torch.equal(ref, got)
    kn[0, 80, 1] = float("nan")  # seen by the second kv head's queries only
    got = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, window=20, sinks=3)
    assert torch.equal(ref[1], got[1]) and torch.equal(ref[0, :4], got[0, :4]) and got[0, 4:].isnan().all()


@pytest.mark.parametrize("d,n", [(128, 1), (64, 5), (128, 48), (256, 48), (128, 400)])
@pytest.mark.parametrize("big", [1e30, 3e38])
def test_huge_norms_where_no_query_looks(K, d, n, big):
    """Finite norms of any size at positions that no query sees, in blocks that
    some do: the results are those of the same cache with zeros there."""
    S, hq, hkv, window, sinks = 700, 4, 2, 43, 3
    L = S - 5
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    q = torch.randn(n, hq, d, device="cuda").half()
    args = (torch.tensor([L], dtype=torch.int32, device="cuda"), window, sinks,
            torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    got = []
    for hidden in (0.0, big):
        for x in (kn, vn):
            x[:, sinks:L - n - window + 1] = hidden
            x[:, L:] = hidden
        got.append(K.attend_window(q, kc, vc, kp, kn, vp, vn, *args))
    assert got[0].abs().max() > 0 and torch.equal(*got)


def test_a_huge_norm_leaves_earlier_row_tiles_as_they_were(K):
    """The last token's value norm lies in a block that rows of the first row
    tile (256 rows: tokens 0 to 127) see up to the position before it."""
    d, S, hq, hkv, n = 128, 640, 4, 2, 136
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    vn *= 1e-3
    q = torch.randn(n, hq, d, device="cuda").half()
    args = (torch.tensor([S], dtype=torch.int32, device="cuda"), None, 0,
            torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    ref = K.attend_window(q, kc, vc, kp, kn, vp, vn, *args)
    vn[0, -1] = 3e38
    got = K.attend_window(q, kc, vc, kp, kn, vp, vn, *args)
    assert ref.abs().max() > 0 and torch.equal(got[:128], ref[:128])
    assert not torch.equal(got[-1], ref[-1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n", [4, 64])
def test_non_finite_norms_reach_the_rows_that_see_them(K, n, bad):
    """A value norm that is not finite: NaN or infinite rows for the queries of
    its kv head that see the position, the others as they were (few and many
    query rows)."""
    d, S, hq, hkv, window, sinks = 128, 300, 4, 2, 40, 2
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    q = torch.randn(n, hq, d, device="cuda").half()
    args = (torch.tensor([S], dtype=torch.int32, device="cuda"), window, sinks,
            torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    ref = K.attend_window(q, kc, vc, kp, kn, vp, vn, *args)
    at = S - 42  # seen by the tokens at positions below at + 40
    vn[0, at, 1] = bad
    got = K.attend_window(q, kc, vc, kp, kn, vp, vn, *args)
    p = torch.arange(S - n, S, device="cuda")
    hit = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    hit[(p >= at) & (p - at < window), 2:] = True
    assert torch.equal(got[~hit], ref[~hit])
    assert not torch.isfinite(got[hit]).any(-1).any() if hit.any() else True
    assert hit.any() and not hit.all()


@pytest.mark.parametrize("n,S", [(1, 40), (1, 2000), (40, 100), (40, 3000)])
def test_a_nan_query_gives_its_own_rows_nan(K, n, S):
    """One and several splits, few and many query rows."""
    d, hq, hkv = 128, 4, 2
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    q = torch.randn(n, hq, d, device="cuda").half()
    q[n // 2, 1, 7] = float("nan")
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, torch.tensor([S], dtype=torch.int32, device="cuda"),
                        q_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)
    nan = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    nan[n // 2, 1] = True
    assert torch.equal(o.isnan().all(-1), nan) and torch.equal(o.isnan().any(-1), nan)


@pytest.mark.parametrize("k_norm,v_norm,q_size", [(1e6, 1e6, 1e-4), (1e-6, 1e-6, 100.0), (1e-30, 1e4, 1.0), (30.0, 1e-20, 1e-3)])
def test_norms_and_queries_of_any_size(K, k_norm, v_norm, q_size):
    """Norms far outside fp16 (stored as f32) neither overflow nor vanish:
    compared after the values are brought back to unit size in 64 bits."""
    d, S, hq, hkv, L = 128, 64, 4, 1, 50
    kc, kp, kn = _cache(K, (1, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (1, S, hkv), d, 2, 2)
    kn, vn = kn / kn.mean() * k_norm, vn / vn.mean() * v_norm
    q = (q_size * torch.randn(1, hq, d, device="cuda")).half()
    ctx = torch.tensor([L], dtype=torch.int32, device="cuda")
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx)
    kk, vv = R.decode_rows(kp[0, :L], kn[0, :L], 4, d), R.decode_rows(vp[0, :L], vn[0, :L], 2, d)
    ref, tol = R.attend(q, kk, vv, L, None, 0, 4, 2)
    if ref.abs().max() > 65504:
        assert torch.equal(torch.isinf(o.cpu()), ref.abs() >= 65520) or (ref.abs() > 65000).any()
        fine = (ref.abs() < 65000) & torch.isfinite(o.cpu())
        assert ((o.cpu().double() - ref).abs()[fine] <= tol.max()).all()
    else:
        _check(o, ref, tol)


def _check_to_infinity(o, ref, tol):
    """Results of any size: within the tolerance where fp16 holds the value,
    infinite with the value's sign above. An element of a row with tolerance tol
    is off by up to tol, so it is finite for certain where |value| + tol lies
    below 65520 (where fp16 rounds to infinity), infinite where |value| - tol
    lies above, and either one between (a row of 1e25 has elements that cancel
    to 0 exactly, and a tolerance of 1e22)."""
    o, size = o.cpu().double(), ref.abs()
    fits, over = size + tol[..., None] < 65520, size - tol[..., None] > 65520
    assert torch.isfinite(o[fits]).all()
    assert torch.equal(o[over], ref[over].sign() * float("inf"))
    err = torch.where(fits, o - ref, torch.zeros_like(ref)).norm(dim=-1)
    assert (err <= tol).all(), (err / tol.clamp(min=1e-30)).max().item()


@pytest.mark.parametrize("ratio", [1e4, 1e6, 1e10, 1e25, 1e27])
@pytest.mark.parametrize("n,hq,S", [(3, 2, 200), (3, 4, 3000), (64, 2, 200), (32, 2, 2000), (136, 4, 700)])
@pytest.mark.parametrize("d,kb,vb", [(128, 2, 4), (64, 2, 2), (256, 2, 3)])
def test_a_large_norm_leaves_the_rows_before_it_as_exact(K, d, kb, vb, n, hq, S, ratio):
    """A value norm larger than the others by `ratio` at a token in the middle:
    the rows of earlier tokens, in the same warp or row tile, do not see it and
    are as exact as without it. Few and many query rows, one split and several."""
    kc, kp, kn = _cache(K, (1, S, 2), d, kb, 1)
    vc, vp, vn = _cache(K, (1, S, 2), d, vb, 2)
    at = S - n + n // 2
    vn[0, at] = ratio * vn.mean()
    q = torch.randn(n, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).half()
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, torch.tensor([S], dtype=torch.int32, device="cuda"),
                        q_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)
    kk, vv = R.decode_rows(kp[0], kn[0], kb, d), R.decode_rows(vp[0], vn[0], vb, d)
    for i in sorted({0, 1, n // 2 - 1, n // 2, n - 1}):
        ref, tol = R.attend(q[i][None], kk, vv, S - n + i + 1, None, 0, kb, vb)
        _check_to_infinity(o[i][None], ref, tol)
        assert ref.abs().max() > 0.01
    assert K.tq_device_error() == (K.TQ_OK, 0)


@pytest.mark.parametrize("weightless", [True, False])
@pytest.mark.parametrize("n,S", [(1, 90), (4, 3000), (64, 90), (32, 2000)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_norms_at_small_weights(K, d, n, S, weightless):
    """Visible positions whose weight and norm differ by large factors: one of
    weight e^-45 whose norm is 2^40 times the others', and one that takes
    nearly all the weight (others e^-28) while the others' norms are 2^43 times
    its own (infinite rows for the tokens before it)."""
    hq, kb, vb, at = 2, 2, 4, 37
    g = torch.Generator(device="cuda").manual_seed(S + d)
    u = torch.randn(d, generator=g, device="cuda")
    u /= u.norm()
    x = torch.randn(1, S, 1, d, generator=g, device="cuda")
    x -= (x @ u)[..., None] * u  # other keys score near 0
    gap = -45.0 if weightless else 28.0
    x[0, at, 0] = gap * d ** 0.5 / 16 * u
    kc = K.TurboQuant(d, kb)
    kp, kn = kc.encode(x.half())
    vc, vp, vn = _cache(K, (1, S, 1), d, vb, 2)
    if weightless:
        vn[0, at] *= 2.0 ** 40
    else:
        vn *= 2.0 ** 33
        vn[0, at] = 2.0 ** -10 * d ** 0.5
    q = (16 * u + 0.05 * torch.randn(n, hq, d, generator=g, device="cuda")).half()
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, torch.tensor([S], dtype=torch.int32, device="cuda"),
                        q_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)
    kk, vv = R.decode_rows(kp[0], kn[0], kb, d), R.decode_rows(vp[0], vn[0], vb, d)
    ref, tol = R.attend(q, kk, vv, S, None, 0, kb, vb)
    sees = torch.arange(S - n, S) >= at
    assert 0.001 < ref[sees].abs().max() < 60000
    _check(o[sees.cuda()], ref[sees], tol[sees])
    _check_to_infinity(o, ref, tol)
    assert K.tq_device_error() == (K.TQ_OK, 0)


@pytest.mark.parametrize("k_norm,v_norm,q_size", [(1e6, 1e6, 1e-4), (1e-6, 1e-6, 100.0), (1e-30, 1e4, 1.0),
                                                  (30.0, 1e-20, 1e-3), (1e-3, 3e6, 1.0), (1e4, 2e5, 1e-3)])
@pytest.mark.parametrize("n,hq", [(1, 4), (5, 4), (64, 2)])
@pytest.mark.parametrize("d,kb,vb", [(64, 4, 3), (128, 4, 2), (256, 3, 4)])
def test_norms_of_any_size_up_to_infinity(K, d, kb, vb, n, hq, k_norm, v_norm, q_size):
    """Norms and queries of any size that every query looks at, few and many
    query rows: finite where fp16 holds the result, infinite above."""
    S, L = 100, 97
    kc, kp, kn = _cache(K, (1, S, 1), d, kb, 1)
    vc, vp, vn = _cache(K, (1, S, 1), d, vb, 2)
    kn, vn = kn / kn.mean() * k_norm, vn / vn.mean() * v_norm
    q = (q_size * torch.randn(n, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d))).half()
    o = K.attend_window(q, kc, vc, kp, kn, vp, vn, torch.tensor([L], dtype=torch.int32, device="cuda"),
                        q_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)
    kk, vv = R.decode_rows(kp[0, :L], kn[0, :L], kb, d), R.decode_rows(vp[0, :L], vn[0, :L], vb, d)
    ref, tol = R.attend(q, kk, vv, L, None, 0, kb, vb)
    _check_to_infinity(o, ref, tol)
    assert K.tq_device_error() == (K.TQ_OK, 0)


def test_offsets_and_lengths_out_of_range_are_flagged(K):
    d, S, hq, hkv = 64, 32, 2, 1
    kc, kp, kn = _cache(K, (3, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (3, S, hkv), d, 4, 2)
    q = torch.randn(6, hq, d, device="cuda").half()
    ctx = torch.tensor([32, 32, 32], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    ref = K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, q_offsets=good, max_q=2)
    assert K.tq_device_error() == (K.TQ_OK, 0)
    # decreasing, past the tokens, negative, more than max_q: those sequences
    # are left out. (The first: [0, 2), none, [1, 3): tokens 1 and 2 belong to
    # the last sequence too, so token 0 alone has one value.)
    for off, kept in (([0, 2, 1, 3], [0]), ([0, 2, 4, 7], [0, 1, 2, 3]), ([-1, 2, 4, 6], [2, 3, 4, 5]),
                      ([0, 2, 6, 6], [0, 1])):
        out = torch.full_like(q, 7.0)
        K.attend_window(q, kc, vc, kp, kn, vp, vn, ctx, q_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                        max_q=2, out=out)
        torch.cuda.synchronize()
        assert K.tq_device_error() == (K.TQ_ERR_DEVICE, K.TQ_DEVERR_ROW_RANGE)
        assert torch.equal(out[kept], ref[kept])
    long = torch.tensor([99, 32, 32], dtype=torch.int32, device="cuda")  # clamped to the cache
    got = K.attend_window(q, kc, vc, kp, kn, vp, vn, long, q_offsets=good, max_q=2)
    assert torch.equal(got, ref)
    assert K.tq_device_error() == (K.TQ_ERR_DEVICE, K.TQ_DEVERR_POS_RANGE)


def test_page_out_of_range_is_clamped_and_flagged(K):
    d, S, hq, hkv = 128, 64, 8, 2
    kc, kp, kn = _cache(K, (4, 16, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (4, 16, hkv), d, 2, 2)
    q = torch.randn(1, hq, d, device="cuda").half()
    ctx = torch.tensor([S], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 99, -3, 3]], dtype=torch.int32, device="cuda")
    same = torch.tensor([[0, 3, 0, 3]], dtype=torch.int32, device="cuda")
    got = K.attend_window_paged(q, kc, vc, kp, kn, vp, vn, table, ctx)
    torch.cuda.synchronize()
    assert K.tq_device_error() == (K.TQ_ERR_DEVICE, K.TQ_DEVERR_BLOCK_RANGE)
    assert torch.equal(got, K.attend_window_paged(q, kc, vc, kp, kn, vp, vn, same, ctx))


def test_repeats_streams_workspaces_and_graphs(K):
    """Bit-identical again, on another stream, with a given workspace of any
    contents, and from two captured graphs that share one workspace."""
    d, B, S, hq, hkv = 128, 2, 900, 16, 4
    kc, kp, kn = _cache(K, (B, S, hkv), d, 4, 1)
    vc, vp, vn = _cache(K, (B, S, hkv), d, 2, 2)
    q = torch.randn(B, hq, d, device="cuda").half()
    ctx = torch.tensor([900, 333], dtype=torch.int32, device="cuda")
    args = (kc, vc, kp, kn, vp, vn, ctx, 400, 16)
    ref = K.attend_window(q, *args)
    need = K.tq_attend_window_workspace_bytes(B, B, 1, hq, hkv, d, S, 400, 16)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    assert torch.equal(ref, K.attend_window(q, *args, workspace=ws))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = K.attend_window(q, *args, stream=s)
    s.synchronize()
    assert torch.equal(ref, other)
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.attend_window(q, *args, out=o, workspace=ws)
        graphs.append(g)
    for shorter in (False, True):
        if shorter:
            ctx.sub_(100)
            ref = K.attend_window(q, *args)
        for o in outs:
            o.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref, o) for o in outs)


def test_cache_past_2_to_the_31_bytes(K):
    """Rows whose byte offsets pass 32 bits: a pool of 3 GB whose last pages are used."""
    d, hkv, hq, nb = 256, 8, 8, 200000
    kc, vc = K.TurboQuant(d, 4), K.TurboQuant(d, 2)
    kp = torch.zeros(nb, 16, hkv, 128, dtype=torch.uint8, device="cuda")
    vp = torch.zeros(nb, 16, hkv, 64, dtype=torch.uint8, device="cuda")
    kn = torch.zeros(nb, 16, hkv, device="cuda")
    vn = torch.zeros(nb, 16, hkv, device="cuda")
    assert kp.numel() > 1 << 31
    last = torch.tensor([[nb - 1, nb - 2, nb - 3]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 3, 16, hkv, d, device="cuda").half()
    for i in range(3):
        kp[nb - 1 - i], kn[nb - 1 - i] = kc.encode(x[0, i])
        vp[nb - 1 - i], vn[nb - 1 - i] = vc.encode(x[1, i])
    q = torch.randn(1, hq, d, device="cuda").half()
    ctx = torch.tensor([45], dtype=torch.int32, device="cuda")
    got = K.attend_window_paged(q, kc, vc, kp, kn, vp, vn, last, ctx)
    low = torch.tensor([[2, 1, 0]], dtype=torch.int32, device="cuda")
    ref = K.attend_window_paged(q, kc, vc, *(t[nb - 3:].contiguous() for t in (kp, kn, vp, vn)), low, ctx)
    assert torch.equal(got, ref) and torch.isfinite(got).all() and got.abs().max() > 0
