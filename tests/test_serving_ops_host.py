"""Refusals and host arithmetic of the operators around the packed cache,
without a GPU: every refusal happens before a CUDA call."""

import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def K():
    import kv_cache_vector_turboquant_b200 as K

    return K


def _raises(fn, text):
    with pytest.raises(ValueError, match=text):
        fn()


def test_norm_rope_refusals(K):
    q, k = torch.zeros(5, 4, 128, dtype=torch.float16), torch.zeros(5, 2, 128, dtype=torch.float16)
    pos = torch.zeros(5, dtype=torch.int32)
    f, _ = K.rope_frequencies(128, device="cpu")
    w = torch.ones(128)
    f_ = K.qk_norm_rope
    _raises(lambda: f_(q, k, pos, f), "CUDA")
    _raises(lambda: f_(q[0], k, pos, f), "Hq")
    _raises(lambda: f_(q, k[:4], pos, f), "same T")
    _raises(lambda: f_(q[..., :96], k[..., :96], pos), "head_dim")
    _raises(lambda: f_(q.float(), k, pos, f), "float16")
    _raises(lambda: f_(q, k.bfloat16(), pos, f), "float16")
    _raises(lambda: f_(q, k, pos.long(), f), "positions: dtype")
    _raises(lambda: f_(q, k, pos[:4], f), "positions: 5 elements")
    _raises(lambda: f_(q, k, pos, f.float()), "inv_freq: dtype")
    _raises(lambda: f_(q, k, pos, torch.zeros(65, dtype=torch.float64)), "at most 64")
    _raises(lambda: f_(q, k, pos, f, q_weight=w[:64]), "q_weight: 128")
    _raises(lambda: f_(q, k, pos, f, q_weight=w, k_weight=w.half()), "same dtype")
    _raises(lambda: f_(q, k, pos, f, q_weight=w.bfloat16()), "q_weight: dtype")
    _raises(lambda: f_(q, k, pos, f, eps=-1.0), "eps")
    _raises(lambda: f_(q, k, pos, f, eps=float("nan")), "eps")
    _raises(lambda: f_(q, k, pos, f, out=(q, k.float())), "out k: dtype")
    _raises(lambda: f_(q, k, pos, f, out=(q[:4], k)), "out q: shape")
    same = k.clone()
    _raises(lambda: f_(k, k.clone(), pos, f, out=(same, same)), "shares memory")
    _raises(lambda: f_(k.clone(), k, pos, f, out=(k, torch.empty_like(k))), "shares memory")
    slab = torch.zeros(5 * 4 * 128 + 8, dtype=torch.float16)
    _raises(lambda: f_(slab[:2560].view(5, 4, 128), k, pos, f, out=(slab[8:].view(5, 4, 128), same)), "shares memory")
    _raises(lambda: f_(q.bfloat16(), k.bfloat16(), pos, f, out=(q, k)), "CUDA")
    _raises(lambda: f_(q, k, pos, f, out=(q, k)), "CUDA")  # in place is fine
    _raises(lambda: f_(q, k, pos, f, out=(q, same), k_weight=same.view(-1)[:128]), "shares memory")
    wide = torch.zeros(5, 4, 132, dtype=torch.float16)[..., :128]
    _raises(lambda: f_(wide, k, pos, f), "strides")
    off = torch.zeros(5 * 4 * 128 + 1, dtype=torch.float16)[1:].view(5, 4, 128)
    _raises(lambda: f_(off, k, pos, f), "16-byte")
    _raises(lambda: f_(q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, f), "dense rows")


def test_norm_rope_strides_of_single_elements(K):
    """The stride of a dimension of one element is never used: any will do,
    and a view that differs in it alone is the same tensor."""
    pos, f = torch.zeros(1, dtype=torch.int32), K.rope_frequencies(128, device="cpu")[0]
    wide = torch.zeros(3, 6 * 128 + 5, dtype=torch.float16)
    q, k = wide.as_strided((1, 4, 128), (773, 128, 1)), wide.as_strided((1, 2, 128), (773, 128, 1), 512)
    assert q.stride(0) % 8 and q.is_contiguous()
    _raises(lambda: K.qk_norm_rope(q, k, pos, f), "CUDA")
    one = torch.zeros(5, 8, 132, dtype=torch.float16)[:, :1, :128]  # one head, token strides of 8 x 132
    assert one.stride(0) % 8 == 0 and one.stride(1) % 8
    _raises(lambda: K.qk_norm_rope(one, one.clone(), torch.zeros(5, dtype=torch.int32), f), "CUDA")
    # in place, through a view whose strides differ only where there is one element
    _raises(lambda: K.qk_norm_rope(q, k, pos, f, out=(q.as_strided((1, 4, 128), (512, 128, 1)), k)), "CUDA")
    _raises(lambda: K.qk_norm_rope(wide.as_strided((2, 4, 128), (773, 128, 1)), k.expand(2, 2, 128),
                                   torch.zeros(2, dtype=torch.int32), f), "strides")


def test_frequencies(K):
    f, s = K.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and s == 1.0
    assert f[0] == 1.0 and math.isclose(f[31].item(), 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, s = K.rope_frequencies(64, 10000.0, "linear", 4.0, device="cpu")
    assert torch.allclose(lin * 4, f, rtol=1e-14, atol=0) and s == 1.0
    ntk, _ = K.rope_frequencies(64, 10000.0, "ntk", 4.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[31].item() * 4, f[31].item(), rel_tol=1e-12)
    yarn, s = K.rope_frequencies(64, 10000.0, "yarn", 4.0, original_len=4096, device="cpu")
    assert math.isclose(s, 1 + 0.1 * math.log(4.0))
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns > 64], f[turns > 64])          # fast ones kept
    assert torch.allclose(yarn[turns < 0.5] * 4, f[turns < 0.5])  # slow ones stretched
    assert (yarn <= f).all() and (yarn * 4 >= f * (1 - 1e-12)).all()
    for bad in (lambda: K.rope_frequencies(3), lambda: K.rope_frequencies(64, scaling="other"),
                lambda: K.rope_frequencies(64, scaling="linear", factor=0.5),
                lambda: K.rope_frequencies(2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("rot,base,length,factor,fast,slow", [
    (64, 1e4, 4096, 4.0, 32.0, 1.0), (128, 1e4, 32768, 4.0, 32.0, 1.0), (128, 5e5, 8192, 8.0, 32.0, 1.0),
    # the slowest frequency turns more than beta_slow times
    (128, 1e4, 131072, 4.0, 32.0, 1.0), (64, 1e4, 65536, 8.0, 32.0, 1.0), (20, 1e4, 32768, 8.0, 32.0, 1.0),
    (64, 1e4, 1 << 20, 2.0, 64.0, 2.0), (2, 1e4, 4096, 2.0, 32.0, 1.0),
    # more than beta_fast times, and none of them: all kept
    (64, 100.0, 1 << 20, 4.0, 32.0, 1.0),
    # the fastest one turns less often than beta_fast, less often than beta_slow
    (64, 1e4, 100, 4.0, 32.0, 1.0), (64, 1e4, 3, 4.0, 32.0, 1.0), (64, 1e4, 1, 4.0, 32.0, 1.0)])
def test_yarn_follows_the_published_rule(K, rot, base, length, factor, fast, slow):
    """The ramp between the indices at which a frequency turns `fast` and
    `slow` times within `length`, rounded outward and kept within
    [0, rot - 1], written out for every index."""
    got, s = K.rope_frequencies(rot, base, "yarn", factor, length, fast, slow, device="cpu")
    assert math.isclose(s, 1 + 0.1 * math.log(factor))

    def index(turns):  # base^(-2 i / rot) length = 2 pi turns
        return rot / 2 * math.log(length / (2 * math.pi * turns), base)

    first, last = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if length * f / (2 * math.pi) < slow and i >= index(slow) + 1:
            expect = f / factor
        elif length * f / (2 * math.pi) > fast and i <= first:
            expect = f
        elif last <= 0:  # even the fastest frequency turns less than `slow` times
            expect = f / factor
        else:
            share = min(max((i - first) / (last - first), 0.0), 1.0) if last > first else 0.0
            expect = f / factor * share + f * (1 - share)
        assert math.isclose(got[i].item(), expect, rel_tol=1e-12), i
        if length * f / (2 * math.pi) > fast:
            assert math.isclose(got[i].item(), f, rel_tol=1e-12)


def test_window_refusals(K):
    kc, vc = K.TurboQuant(128, 4), K.TurboQuant(128, 2)
    B, S, hkv, hq = 2, 32, 2, 8
    q = torch.zeros(B, hq, 128, dtype=torch.float16)
    kp, vp = torch.zeros(B, S, hkv, 64, dtype=torch.uint8), torch.zeros(B, S, hkv, 32, dtype=torch.uint8)
    kn, vn = torch.zeros(B, S, hkv), torch.zeros(B, S, hkv)
    ctx, off = torch.zeros(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    f = K.attend_window
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx), "CUDA")
    _raises(lambda: f(q.bfloat16(), kc, vc, kp, kn, vp, vn, ctx), "q: dtype")
    _raises(lambda: f(q[:, :7].contiguous(), kc, vc, kp, kn, vp, vn, ctx), "multiple of 2")
    _raises(lambda: f(q, kc, K.TurboQuant(64, 2), kp, kn, vp, vn, ctx), "same head_dim")
    _raises(lambda: f(q, kc, vc, vp, kn, vp, vn, ctx), "k_packed: shape")
    _raises(lambda: f(q, kc, vc, kp, kn[:1], vp, vn, ctx), "k_norms: shape")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn.double(), ctx), "v_norms: dtype")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx.long()), "context_lens: dtype")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, window=0), "window")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, sinks=-1), "sinks")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, window=2.5), "window")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, window=1 << 70), "window")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, q_offsets=off, max_q="2"), "max_q")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, [0, 0]), "context_lens: a torch tensor")
    _raises(lambda: f(torch.cat([q, q]), kc, vc, kp, kn, vp, vn, ctx), "one token per sequence")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, max_q=2), "one token per sequence")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, q_offsets=off), "max_q")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, q_offsets=off[:2], max_q=1), "q_offsets: 3")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, out=q.float()), "out: dtype")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, workspace=kn), "workspace: dtype")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, out=q), "CUDA")  # in place is fine
    slab = torch.zeros(q.numel() + 128, dtype=torch.float16)
    part = slab[:q.numel()].view(q.shape)
    _raises(lambda: f(part, kc, vc, kp, kn, vp, vn, ctx, out=slab[128:].view(q.shape)), "out: shares memory")
    ws = slab.view(torch.uint8)
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, out=part, workspace=ws), "out: shares memory")
    _raises(lambda: f(part, kc, vc, kp, kn, vp, vn, ctx, workspace=ws), "workspace: shares memory")
    _raises(lambda: f(q, kc, vc, kp, kn, vp, vn, ctx, workspace=kp.view(-1)[:64]), "workspace: shares memory")
    pool = [t.reshape(B * S // 16, 16, *t.shape[2:]) for t in (kp, kn, vp, vn)]
    bt = torch.zeros(B, S // 16, dtype=torch.int32)
    p = K.attend_window_paged
    _raises(lambda: p(q, kc, vc, *pool, bt, ctx), "CUDA")
    _raises(lambda: p(q, kc, vc, *pool, bt.long(), ctx), "block_tables: dtype")
    _raises(lambda: p(q, kc, vc, pool[0].reshape(2, 32, 2, 64), *pool[1:], bt, ctx), "16 positions")
    _raises(lambda: p(q, kc, vc, *pool, bt, ctx[:1]), "context_lens")
    layer = K.TQPagedAttention(kc, hq, v_tq=vc)
    key = torch.zeros(B, hkv, 128, dtype=torch.float16)
    _raises(lambda: layer.step(q[:, :4], key, key, ctx, ctx, *pool, bt, ctx), "num_query_heads")
    _raises(lambda: layer.step(q, key, key[:1], ctx, ctx, *pool, bt, ctx), "value")
    _raises(lambda: layer.step(q, key, key, ctx, ctx, *pool, bt, ctx), "CUDA")


def test_gradients_are_refused_not_dropped(K):
    """No call here has a backward pass: what requires a gradient is refused
    while gradients are recorded, and taken otherwise."""
    q, k = torch.zeros(2, 4, 128, dtype=torch.float16), torch.zeros(2, 2, 128, dtype=torch.float16)
    pos, w = torch.zeros(2, dtype=torch.int32), torch.nn.Parameter(torch.ones(128))
    f = K.rope_frequencies(128, device="cpu")[0]
    grad = lambda t: t.clone().requires_grad_()  # noqa: E731
    f_ = K.qk_norm_rope
    for name, call in (("q", lambda: f_(grad(q), k, pos, f)), ("k", lambda: f_(q, grad(k), pos, f)),
                       ("q_weight", lambda: f_(q, k, pos, f, q_weight=w)),
                       ("k_weight", lambda: f_(q, k, pos, f, k_weight=w)),
                       ("inv_freq", lambda: f_(q, k, pos, grad(f))),
                       ("out k", lambda: f_(q, k, pos, f, out=(q, grad(k))))):
        _raises(call, f"^{name}: requires a gradient")
        with torch.no_grad():
            _raises(call, "CUDA")
    _raises(lambda: f_(q, k, pos, f, q_weight=w.detach()), "CUDA")
    kc, vc = K.TurboQuant(128, 4), K.TurboQuant(128, 2)
    kp, vp = torch.zeros(2, 16, 2, 64, dtype=torch.uint8), torch.zeros(2, 16, 2, 32, dtype=torch.uint8)
    kn, vn = torch.zeros(2, 16, 2), torch.zeros(2, 16, 2)
    a = K.attend_window
    for name, call in (("q", lambda: a(grad(q), kc, vc, kp, kn, vp, vn, pos)),
                       ("k_norms", lambda: a(q, kc, vc, kp, grad(kn), vp, vn, pos)),
                       ("v_norms", lambda: a(q, kc, vc, kp, kn, vp, grad(vn), pos)),
                       ("q", lambda: K.attend_window_paged(grad(q), kc, vc, kp, kn, vp, vn, pos[:, None], pos)),
                       ("value", lambda: K.TQPagedAttention(kc, 4, v_tq=vc).step(
                           q, k, grad(k), pos, pos, kp, kn, vp, vn, pos[:, None], pos))):
        _raises(call, f"^{name}: requires a gradient")
        with torch.no_grad():
            _raises(call, "CUDA")


def test_page_refusals(K):
    t, n, r = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    f = K.pages_trim
    _raises(lambda: f(t, n, r, window=5), "CUDA")
    _raises(lambda: f(t.long(), n, r), "block_tables: dtype")
    _raises(lambda: f(t[0], n, r), r"\[rows, max_blocks\]")
    _raises(lambda: f(t[:, :0], n, r), "max_blocks")
    _raises(lambda: f(t, n[:2], r), "context_lens: 3")
    _raises(lambda: f(t, n, r[:0]), "refs")
    _raises(lambda: f(t, n, r, window=-1), "window")
    _raises(lambda: f(t, n, r, sinks=-1), "sinks")
    _raises(lambda: f(t, n, r, release=n), "release: dtype")
    _raises(lambda: f(t, n, r, out=(t[:2], n[:2], r)), "out: shape")
    _raises(lambda: f(t, n, r, out=(t, n, r[:5])), "out: shape")
    _raises(lambda: f(t, n, r, out=(t, n, r)), "CUDA")
    both = torch.zeros(20, dtype=torch.int32)
    _raises(lambda: f(t, n, r, out=(both[:12].view(3, 4), both[11:14], r.clone())), "shares memory")
    _raises(lambda: f(both[:12].view(3, 4), n, r, out=(both[1:13].view(3, 4), n, r)), "shares memory")
    _raises(lambda: f(t, n, r, out=(t.clone(), t[0, :3], r)), "shares memory")
    P = K.TQPagePools
    pool = torch.zeros(9, 16, 2, 16, dtype=torch.uint8)
    _raises(lambda: P([]), "pools")
    _raises(lambda: P([pool]), "CUDA")
    _raises(lambda: P([pool, pool[:8]]), "9 pages")
    _raises(lambda: P([pool[:, :8]]), "contiguous")
    _raises(lambda: P([torch.zeros(9, 24, dtype=torch.uint8)]), "multiple of 16")
    _raises(lambda: P([torch.zeros(9 * 32 + 8, dtype=torch.uint8)[8:].view(9, 32)]), "aligned")
    _raises(lambda: P([pool, pool[:]]), "overlap")
    _raises(lambda: P([torch.zeros(9, 16, dtype=torch.uint8) for _ in range(513)]), "512")


def test_page_calls_refuse_shared_memory(K):
    """Workspaces, tables and outputs of fork and compact that share memory
    with one another or with a pool (host tensors; every refusal comes before
    the one of their device)."""
    ops, i32 = K._calls(), torch.int32
    pool = torch.zeros(9, 16, 2, 16, dtype=torch.uint8)
    a = (K.PagePool * 1)()
    a[0].base, a[0].block_bytes = pool.data_ptr(), 512
    mine = (ctypes.addressof(a), 1, 9, 0)

    def fork(t=None, n=None, r=None, p=None, c=None, out=None, ws=None):
        new = lambda x, *s: torch.zeros(*s, dtype=i32) if x is None else x  # noqa: E731
        return lambda: ops.pages_fork(*mine, new(t, 3, 4), new(n, 3), new(r, 9), new(p, 2), new(c, 2), out, ws)

    def compact(t=None, r=None, out=None, ws=None):
        new = lambda x, *s: torch.zeros(*s, dtype=i32) if x is None else x  # noqa: E731
        return lambda: ops.pages_compact(*mine, new(t, 3, 4), new(r, 9), out, ws)

    slab = torch.zeros(4096, dtype=torch.uint8)
    word = lambda at, *s: slab[at:at + 4 * math.prod(s)].view(i32).view(*s)  # noqa: E731
    for call in (fork(), compact(), fork(ws=slab), compact(ws=slab), fork(t=word(0, 3, 4), ws=slab[48:])):
        _raises(call, "CUDA")  # nothing shared
    out = (torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(9, dtype=i32))
    for call in (fork(t=word(0, 3, 4), ws=slab), fork(n=word(64, 3), ws=slab), fork(r=word(64, 9), ws=slab),
                 fork(p=word(64, 2), ws=slab), fork(c=word(0, 2), ws=slab[4:]),
                 fork(out=(word(0, 3, 4), *out[1:]), ws=slab[44:]), fork(out=(out[0], word(0, 3), out[2]), ws=slab),
                 fork(out=(*out[:2], word(4060, 9)), ws=slab[:4064]),
                 compact(t=word(0, 3, 4), ws=slab), compact(r=word(64, 9), ws=slab),
                 compact(out=(word(0, 3, 4), out[2], torch.zeros(9, dtype=i32), torch.zeros(1, dtype=i32)), ws=slab),
                 compact(out=(out[0], out[2], word(64, 9), torch.zeros(1, dtype=i32)), ws=slab),
                 compact(out=(out[0], out[2], torch.zeros(9, dtype=i32), word(64, 1)), ws=slab)):
        _raises(call, "workspace: shares memory with another")
    inside = lambda *s: pool.view(-1)[-4 * math.prod(s):].view(i32).view(*s)  # noqa: E731
    for call, name in ((fork(t=inside(3, 4)), "block_tables"), (fork(n=inside(3)), "context_lens"),
                       (fork(r=inside(9)), "refs"), (fork(p=inside(2)), "parents"), (fork(c=inside(2)), "children"),
                       (fork(ws=pool.view(-1)[16:]), "workspace"), (fork(out=(inside(3, 4), *out[1:])), "out"),
                       (fork(out=(out[0], inside(3), out[2])), "out"), (fork(out=(*out[:2], inside(9))), "out"),
                       (compact(t=inside(3, 4)), "block_tables"), (compact(r=inside(9)), "refs"),
                       (compact(ws=pool.view(-1)[16:]), "workspace"),
                       (compact(out=(out[0], out[2], inside(9), torch.zeros(1, dtype=i32))), "out remap"),
                       (compact(out=(out[0], out[2], torch.zeros(9, dtype=i32), inside(1))), "out used")):
        _raises(call, f"^{name}: shares memory with pool 0")


def test_abi_refusals(K):
    """The C entry points with host pointers that are never followed."""
    L = K._binding._lib
    buf = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(buf) + 63) & ~63
    kc, vc, small = K.tq_create(128, 4), K.tq_create(128, 2), K.tq_create(64, 2)

    def nr(dtype=0, n=4, hq=2, hkv=1, d=128, strides=(256, 128, 128, 128), rot=64, eps=1e-6, q=p, qo=p, freq=p):
        return L.tq_qk_norm_rope(q, p, dtype, n, hq, hkv, d, *strides, p, freq, rot, 0, 1.0, None, None, 0, eps, qo, p, None)

    assert nr(n=0, q=None) == K.TQ_OK
    assert nr(d=96) == nr(dtype=2) == K.TQ_ERR_UNSUPPORTED
    assert nr(n=-1) == nr(hq=0) == nr(hkv=0) == nr(rot=63) == nr(rot=130) == nr(eps=-1.0) == K.TQ_ERR_INVALID_ARG
    assert nr(eps=float("nan")) == nr(eps=float("inf")) == nr(q=None) == nr(freq=None) == K.TQ_ERR_INVALID_ARG
    assert nr(q=p + 8) == nr(qo=p + 2) == nr(strides=(256, 128, 132, 128)) == nr(freq=p + 4) == K.TQ_ERR_ALIGNMENT

    def aw(k=kc, v=vc, q=p, T=2, B=2, off=None, mq=1, hq=4, hkv=2, S=64, win=0, sinks=0, ws=p, wsn=1 << 40, ctx=p):
        return L.tq_attend_window(k.handle if k else None, v.handle, q, T, B, off, mq, hq, hkv, p, p, p, p, S, ctx, win,
                                  sinks, p, ws, wsn, None)

    assert aw(T=0, B=0, q=None) == K.TQ_OK and aw(T=0, off=p, q=None) == K.TQ_OK
    assert aw(k=None) == aw(v=small) == aw(hq=3) == aw(hkv=0) == aw(S=0) == aw(sinks=-1) == K.TQ_ERR_INVALID_ARG
    assert aw(T=3) == aw(mq=2) == aw(mq=0) == aw(q=None) == aw(ctx=None) == aw(T=-1) == K.TQ_ERR_INVALID_ARG
    assert aw(S=1 << 31) == aw(T=65536, B=65536) == aw(hq=1 << 17, hkv=1 << 17) == K.TQ_ERR_UNSUPPORTED
    assert aw(q=p + 2) == aw(ctx=p + 2) == aw(off=p + 2, mq=2) == aw(ws=p + 4) == K.TQ_ERR_ALIGNMENT
    assert aw(ws=None) == aw(wsn=16) == K.TQ_ERR_WORKSPACE
    ws = K.tq_attend_window_workspace_bytes
    assert ws(2, 2, 1, 4, 2, 128, 64, 0, 0) > 0 and ws(2, 2, 1, 4, 3, 128, 64, 0, 0) == ws(0, 2, 1, 4, 2, 128, 64, 0, 0) == 0
    # the window bounds the splits, and so the workspace
    assert ws(2, 2, 1, 4, 2, 128, 1 << 20, 100, 4) < ws(2, 2, 1, 4, 2, 128, 1 << 20, 0, 0)
    assert ws(2, 2, 1, 4, 2, 128, 1 << 20, (1 << 63) - 1, (1 << 63) - 1) == ws(2, 2, 1, 4, 2, 128, 1 << 20, 0, 0)

    def pg(nb=8, bt=p, mb=2, win=1, sinks=0):
        return L.tq_pages_trim(bt, p, p, p, p, p, 3, mb, nb, win, sinks, None, None)

    assert pg(nb=0) == pg(bt=None) == pg(mb=0) == pg(sinks=-1) == K.TQ_ERR_INVALID_ARG
    assert pg(nb=1 << 27) == pg(mb=1 << 28) == K.TQ_ERR_UNSUPPORTED and pg(bt=p + 2) == K.TQ_ERR_ALIGNMENT

    def fk(base=p, size=32, n=2, rows=3, ws=p, wsn=1 << 20, npool=1):
        a = (K.PagePool * 1)()
        a[0].base, a[0].block_bytes = base, size
        return L.tq_pages_fork(a, npool, 8, p, p, p, p, p, p, rows, 2, p, p, n, ws, wsn, None)

    assert fk(base=None) == fk(size=0) == fk(n=4) == fk(n=-1) == fk(rows=0) == K.TQ_ERR_INVALID_ARG
    assert fk(rows=1 << 18) == fk(npool=513) == fk(size=1 << 31) == K.TQ_ERR_UNSUPPORTED
    assert fk(base=p + 8) == fk(size=24) == K.TQ_ERR_ALIGNMENT
    assert fk(ws=None) == fk(wsn=15) == K.TQ_ERR_WORKSPACE
    assert K.tq_pages_fork_workspace_bytes(0) == K.tq_pages_compact_workspace_bytes(0) == 0


def test_plain_page_operations_agree_with_a_walk(K):
    """The list implementations that the GPU tests compare with, by hand."""
    import serving_ref as R

    t, n, r, moves, skipped, full = R.fork([[3, 1], [-1, -1], [-1, -1]], [20, 0, 0], [0, 1, 0, 1], [0, 0], [1, 2])
    assert t == [[3, 1], [3, 0], [3, 2]] and n == [20, 20, 20] and r == [1, 1, 1, 3]
    assert moves == [(1, 0), (1, 2)] and (skipped, full) == (0, 0)
    t, n, r = R.trim([[0, 1, 2, 3]], [50], [1, 1, 1, 1], 17, 4, None)
    assert t == [[0, -1, 2, 3]] and r == [1, 0, 1, 1]  # page 1 ends at 32 <= 50 - 17; page 2 at 48
    t, n, r = R.trim([[0, 1, 2, 3]], [50], [1, 1, 1, 1], 2, 4, None)
    assert t == [[0, -1, -1, 3]] and r == [1, 0, 0, 1]
    assert R.compact([[4, 0, 2]], [0, 1, 0, 1, 2]) == ([[2, -1, -1]], [0 + 1, 1, 2, 0, 0], [-1, 1, -1, 0, 2], 3, [(3, 0), (4, 2)])
