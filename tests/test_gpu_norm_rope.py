"""Norm and rotation of query and key heads against the formula in 64 bits
(needs a B200)."""

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    import kv_cache_vector_turboquant_b200 as K

    return K


def _qkv(T, hq, hkv, d, dtype, seed):
    """Queries and keys as views of one projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
    return x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))


def _close(got, ref, tol):
    assert got.dtype == torch.float16 and got.shape == ref.shape
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()


CASES = [
    # T, hq, hkv, d, rot, interleaved, norm, dtype, positions up to
    (1, 32, 8, 128, 128, False, True, torch.float16, 1 << 17),
    (1, 1, 1, 64, 2, False, True, torch.bfloat16, 5),
    (3, 5, 1, 64, 64, True, False, torch.bfloat16, 1 << 20),
    (7, 4, 4, 256, 64, False, True, torch.float16, 1 << 20),
    (5, 7, 1, 128, 20, False, True, torch.float16, 4096),    # half of 10: not a multiple of 8
    (5, 7, 1, 256, 250, False, True, torch.bfloat16, 4096),
    (5, 7, 1, 128, 36, True, True, torch.float16, 4096),
    (9, 3, 3, 64, 0, False, True, torch.float16, 4096),      # norm only
    (331, 2, 1, 128, 128, False, True, torch.float16, 1 << 17),
    (2600, 2, 1, 64, 48, True, True, torch.bfloat16, 1 << 17),   # tokens share a CTA
    (1500, 3, 2, 256, 48, False, False, torch.float16, 1 << 17),
    (640, 71, 9, 64, 32, False, True, torch.float16, 1 << 17),
]


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,norm,dtype,far", CASES)
@pytest.mark.parametrize("w32", [False, True])
def test_matches_formula(K, T, hq, hkv, d, rot, inter, norm, dtype, far, w32):
    q, k = _qkv(T, hq, hkv, d, dtype, T + d)
    g = torch.Generator(device="cuda").manual_seed(rot)
    pos = torch.randint(-far, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    wt = torch.float32 if w32 else dtype
    qw = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt) if norm else None
    kw = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt) if norm else None
    f, scale = (K.rope_frequencies(rot, 10000.0, "yarn", 8.0) if rot > 2 else
                (torch.ones(1, dtype=torch.float64, device="cuda"), 1.25) if rot else (None, 1.0))
    qo, ko = K.qk_norm_rope(q, k, pos, f, interleaved=inter, rope_scale=scale, q_weight=qw, k_weight=kw, eps=1e-5)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        _close(got, *R.rope(x, w, pos, f, inter, scale, 1e-5))


def test_one_weight_only_and_zero_rows(K):
    q, k = _qkv(6, 2, 2, 128, torch.float16, 1)
    q = q.clone()
    q[2] = 0
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    f, _ = K.rope_frequencies(128)
    w = torch.full((128,), 2.0, device="cuda")
    qo, ko = K.qk_norm_rope(q, k, pos, f, q_weight=w)
    assert torch.all(qo[2] == 0)
    _close(qo, *R.rope(q, w, pos, f, False, 1.0, 1e-6))
    _close(ko, *R.rope(k, None, pos, f, False, 1.0, 1e-6))


def test_in_place_strides_and_streams(K):
    q, k = _qkv(50, 4, 2, 128, torch.float16, 3)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    f, _ = K.rope_frequencies(64)
    ref = K.qk_norm_rope(q, k, pos, f)
    qc, kc = q.contiguous(), k.contiguous()
    K.qk_norm_rope(qc, kc, pos, f, out=(qc, kc))
    assert torch.equal(qc, ref[0]) and torch.equal(kc, ref[1])
    # heads outside, tokens inside: [H, T, d] storage
    qt, kt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k))
    got = K.qk_norm_rope(qt, kt, pos, f)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = K.qk_norm_rope(q, k, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_single_elements_of_any_stride(K):
    """One token, and one head, of a buffer whose stride there is not a
    multiple of 8 (it is never used), also in place."""
    f, _ = K.rope_frequencies(128)
    w = 1 + 0.1 * torch.randn(128, device="cuda")
    wide = torch.randn(3, 6 * 128 + 5, device="cuda").half()
    one = torch.randn(5, 8, 132, device="cuda").half()[:, :1, :128]
    for q, k in ((wide.as_strided((1, 4, 128), (773, 128, 1)), wide.as_strided((1, 2, 128), (773, 128, 1), 512)),
                 (one, torch.randn(5, 2, 128, device="cuda").half())):
        pos = 7 + torch.arange(q.shape[0], dtype=torch.int32, device="cuda")
        got = K.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
        _close(got[0], *R.rope(q, w, pos, f, False, 1.0, 1e-6))
        _close(got[1], *R.rope(k, w, pos, f, False, 1.0, 1e-6))
        if q.is_contiguous():
            K.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w, out=(q, k))
            assert torch.equal(q, got[0]) and torch.equal(k, got[1])


def test_empty_and_non_finite(K):
    q, k = _qkv(0, 4, 2, 128, torch.float16, 3)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    qo, ko = K.qk_norm_rope(q, k, pos)
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
    q, k = _qkv(3, 4, 2, 128, torch.float16, 4)
    q = q.clone()
    q[1, 2, 5] = float("nan")
    q[2, 0, 7] = float("inf")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    f, _ = K.rope_frequencies(128)
    w = torch.ones(128, device="cuda")
    qo, ko = K.qk_norm_rope(q, k, pos, f, q_weight=w)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True  # only the rows that hold them
    assert torch.equal(qo.isnan().any(-1), bad) and torch.isfinite(ko).all()


def test_captured_and_replayed(K):
    q, k = _qkv(16, 32, 8, 128, torch.bfloat16, 9)
    q, k = q.clone(), k.clone()
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    f, _ = K.rope_frequencies(128)
    out = (torch.empty(16, 32, 128, dtype=torch.float16, device="cuda"),
           torch.empty(16, 8, 128, dtype=torch.float16, device="cuda"))
    K.qk_norm_rope(q, k, pos, f, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.qk_norm_rope(q, k, pos, f, out=out)
    q.mul_(0.5)
    pos.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    ref = K.qk_norm_rope(q, k, pos, f)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
