"""The operators together, as a serving engine runs them (needs a B200):
norm and rotation, encode into pages, windowed attention, trimming, forking
and compacting between steps, against 64-bit attention over the decoded rows
of a plain copy of every sequence."""

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    import kv_cache_vector_turboquant_b200 as K

    return K


def test_a_refused_step_leaves_the_pools_as_they_were(K):
    d, hq, hkv, T = 64, 4, 2, 3
    kc, vc = K.TurboQuant(d, 4), K.TurboQuant(d, 2)
    layer = K.TQPagedAttention(kc, hq, v_tq=vc)
    pools = [torch.zeros(4, 16, hkv, kc.packed_bytes, dtype=torch.uint8, device="cuda"),
             torch.zeros(4, 16, hkv, device="cuda"),
             torch.zeros(4, 16, hkv, vc.packed_bytes, dtype=torch.uint8, device="cuda"),
             torch.zeros(4, 16, hkv, device="cuda")]
    q, k, v = (torch.randn(T, h, d, device="cuda").half() for h in (hq, hkv, hkv))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = {"positions": i32([0, 1, 2]), "slot_mapping": i32([0, 1, 2]), "k_packed": pools[0], "k_norms": pools[1],
            "v_packed": pools[2], "v_norms": pools[3], "block_tables": i32([[0]]), "context_lens": i32([3]),
            "q_offsets": i32([0, 3]), "max_q": 3}
    for bad in ({"window": 0}, {"sinks": -1}, {"q_offsets": None}, {"max_q": None}, {"context_lens": i32([3, 3])},
                {"context_lens": i32([3]).long()}, {"block_tables": i32([0])}, {"v_norms": pools[3][:3]},
                {"v_packed": pools[0]}, {"k_norms": pools[1].double()}, {"slot_mapping": i32([0, 1])},
                {"slot_mapping": i32([0, 1, 2]).long()}, {"slot_mapping": i32([0, 1, 2]).cpu()},
                {"context_lens": i32([3]).cpu()}, {"positions": i32([0, 1])}):
        with pytest.raises(ValueError):
            layer.step(q, k, v, **(good | bad))
        with pytest.raises(ValueError):
            layer.step(q, k, v.cpu(), **good)
        assert not any(p.any() for p in pools), bad
    o = layer.step(q, k, v, **good)
    assert torch.isfinite(o).all() and all(p[0, :3].any() for p in pools)


def test_prompt_decode_fork_trim_compact(K):
    d, hq, hkv, kb, vb, window, sinks = 64, 6, 2, 4, 3, 40, 5
    rows, mb, nb = 4, 12, 30
    kc, vc = K.TurboQuant(d, kb), K.TurboQuant(d, vb)
    pools = [torch.zeros(nb, 16, hkv, kc.packed_bytes, dtype=torch.uint8, device="cuda"),
             torch.zeros(nb, 16, hkv, device="cuda"),
             torch.zeros(nb, 16, hkv, vc.packed_bytes, dtype=torch.uint8, device="cuda"),
             torch.zeros(nb, 16, hkv, device="cuda")]
    handle = K.TQPagePools(pools)
    layer = K.TQPagedAttention(kc, hq, v_tq=vc)
    f, scale = K.rope_frequencies(d, scaling="ntk", factor=4.0)
    w = (1 + 0.1 * torch.randn(d, device="cuda")).half()
    table = torch.full((rows, mb), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    plain = {r: ([], []) for r in range(rows)}  # fp64 decoded keys and values of every position
    g = torch.Generator(device="cuda").manual_seed(3)

    def grow(r, n):
        """Pages for n more tokens of row r (host side), and their slots."""
        slots = []
        for t in range(int(lens[r]), int(lens[r]) + n):
            if t % 16 == 0:
                page = int((refs == 0).nonzero()[0])
                table[r, t // 16] = page
                refs[page] = 1
            slots.append(int(table[r, t // 16]) * 16 + t % 16)
        lens[r] += n
        return slots

    def step(counts):
        """counts: new tokens of every row; attends and checks them."""
        start = lens.tolist()
        slots = [s for r, n in enumerate(counts) for s in grow(r, n)]
        T = sum(counts)
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").half()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
        pos = torch.tensor([start[r] + i for r, n in enumerate(counts) for i in range(n)], dtype=torch.int32, device="cuda")
        off = torch.tensor([sum(counts[:r]) for r in range(rows + 1)], dtype=torch.int32, device="cuda")
        slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
        o = layer.step(q, k, v, pos, slot, *pools, table, lens, window=window, sinks=sinks, q_offsets=off,
                       max_q=max(counts), inv_freq=f, rope_scale=scale, q_weight=w, k_weight=w)
        rq, rk = K.qk_norm_rope(q, k, pos, f, rope_scale=scale, q_weight=w, k_weight=w)
        kk = R.decode_rows(*kc.encode(rk), kb, d)
        vv = R.decode_rows(*vc.encode(v.contiguous()), vb, d)
        for r, n in enumerate(counts):
            lo = int(off[r])
            plain[r][0].extend(kk[lo:lo + n])
            plain[r][1].extend(vv[lo:lo + n])
            if n:
                ref, tol = R.attend(rq[lo:lo + n], torch.stack(plain[r][0]), torch.stack(plain[r][1]), len(plain[r][0]),
                                    window, sinks, kb, vb)
                err = (o[lo:lo + n].cpu().double() - ref).norm(dim=-1)
                assert (err <= tol).all(), (r, (err / tol).max().item())

    step([70, 33, 0, 0])
    step([1, 1, 0, 0])
    table, lens, refs = handle.fork(table, lens, refs, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                    torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    for p, c in ((0, 2), (1, 3)):
        plain[c] = (list(plain[p][0]), list(plain[p][1]))
    step([1, 2, 3, 1])
    for _ in range(3):
        table, lens, refs = K.pages_trim(table, lens, refs, window=window, sinks=sinks)
        table, refs, remap, used = handle.compact(table, refs)
        assert int(used) == int((refs > 0).sum()) and torch.all(refs[int(used):] == 0)
        step([9, 1, 1, 17])
    table, lens, refs = K.pages_trim(table, lens, refs, release=torch.tensor([True, False, True, True], device="cuda"))
    assert lens.tolist()[0] == 0 and int((refs > 0).sum()) == int((table[1] >= 0).sum())
    plain.update({0: ([], []), 2: ([], []), 3: ([], [])})
    step([20, 1, 0, 5])
    assert K.tq_device_error() == (K.TQ_OK, 0)
