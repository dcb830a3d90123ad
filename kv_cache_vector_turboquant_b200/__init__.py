"""TurboQuant KV-cache codec for NVIDIA B200 (sm_100a).

The compute path is the CUDA library ``libtq.so`` behind the C ABI of
``include/tq.h``; this package is its ctypes binding plus a small convenience
layer with the call shapes of the "aither-kvcache" page ("Quick Start --
TurboQuant", "API Reference": ``TurboQuant(head_dim, bits, seed=42)``,
``encode(x) -> (packed, norms)``, ``decode(packed, norms)``,
``compression_ratio()``). PyTorch supplies device memory and streams only.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib

from ._binding import (  # noqa: F401
    LIB_PATH,
    TQ_BF16,
    TQ_DEVERR_BLOCK_RANGE,
    TQ_DEVERR_POOL_FULL,
    TQ_DEVERR_POS_RANGE,
    TQ_DEVERR_ROW_RANGE,
    TQ_DEVERR_SLOT_RANGE,
    TQ_DEVERR_SMEM_LAYOUT,
    TQ_DEVERR_TIMEOUT,
    TQ_ERR_ALIGNMENT,
    TQ_ERR_CUDA,
    TQ_ERR_DEVICE,
    TQ_ERR_INVALID_ARG,
    TQ_ERR_NOMEM,
    TQ_ERR_TIMEOUT,
    TQ_ERR_UNSUPPORTED,
    TQ_ERR_WORKSPACE,
    TQ_F16,
    TQ_MAX_PAGE_POOLS,
    TQ_MAX_PAGE_ROWS,
    TQ_OK,
    TQ_PAGE_BLOCK,
    Ctx,
    PagePool,
    TQError,
    TQ_ATTEND_STATIC_SCRATCH_BYTES,
    tq_attend_decode,
    tq_attend_decode_paged,
    tq_attend_decode_static,
    tq_attend_window,
    tq_attend_window_paged,
    tq_attend_window_workspace_bytes,
    tq_attend_workspace_bytes,
    tq_create,
    tq_decode,
    tq_check_device_error,
    tq_device_error,
    tq_encode,
    tq_encode_append,
    tq_encode_append_kv,
    tq_encode_os,
    tq_decode_os,
    tq_encode_slots,
    tq_get_tables,
    tq_pages_compact,
    tq_pages_compact_workspace_bytes,
    tq_pages_fork,
    tq_pages_fork_workspace_bytes,
    tq_pages_trim,
    tq_qk_norm_rope,
    tq_status_string,
    tq_tensor_core_check,
)


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check(t, name: str, dtypes, shape=None, numel=None) -> None:
    """Type, dtype, layout and size of a tensor argument; the device is
    checked separately (_on_device), after every size check."""
    try:  # the common case first: a call of a decode step makes a dozen of these
        if (t.dtype is dtypes and t.is_contiguous() and (shape is None or t.shape == shape)
                and (numel is None or t.numel() == numel)):
            return
    except AttributeError:
        pass
    import torch

    _require(isinstance(t, torch.Tensor), f"{name}: a torch tensor")
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    _require(t.dtype in dtypes, f"{name}: dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    _require(t.is_contiguous(), f"{name}: contiguous")
    if shape is not None:
        _require(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel is not None:
        _require(t.numel() == numel, f"{name}: {numel} elements, got {t.numel()}")


def _on_device(**tensors) -> None:
    """Every kernel reads and writes device memory: host tensors are refused
    here, before a pointer reaches the library."""
    for name, t in tensors.items():
        _require(t.is_cuda, f"{name}: a CUDA tensor")


@contextlib.contextmanager
def _launching(device, stream):
    """Make `device` current and, where a stream is given, that stream: what
    is allocated inside then belongs to the stream that uses it."""
    import torch

    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            _require(stream.device == device, f"stream: one of {device}, got {stream.device}")
            with torch.cuda.stream(stream):
                yield


def _one_device(names, tensors) -> int:
    """Index of the CUDA device that holds all the tensors (Nones are left out)."""
    dev = tensors[0].get_device()
    if dev >= 0:
        for t in tensors:
            if t is not None and t.get_device() != dev:
                break
        else:
            return dev
    for name, t in zip(names, tensors):
        if t is not None:
            _require(t.is_cuda, f"{name}: a CUDA tensor")
            _require(t.get_device() == dev, f"{name}: on {tensors[0].device} like the other tensors, got {t.device}")
    return dev


@functools.cache
def _calls():
    """The compiled checks and calls of the operators around the cache."""
    import torch  # noqa: F401  (the extension is linked against its libraries)

    try:
        return importlib.import_module("._ops", __name__)
    except ImportError as e:
        raise ImportError("_ops.so is missing or does not fit the installed torch; build it with "
                          "`python kv_cache_vector_turboquant_b200/build.py`") from e


def _on_stream(stream, name, t, call, *args):
    """`call` inside `stream`, one of the device that holds the tensor `t`."""
    import torch

    _require(isinstance(t, torch.Tensor) and t.is_cuda, f"{name}: a CUDA tensor")
    with _launching(t.device, stream):
        return call(*args)


class TurboQuant:
    """One codec (head_dim, bits, seed) on the current CUDA device."""

    def __init__(self, head_dim: int = 128, bits: int = 4, seed: int = 42):
        self.ctx = tq_create(head_dim, bits, seed)
        self.head_dim, self.bits, self.seed = head_dim, bits, seed
        self.packed_bytes = self.ctx.packed_bytes

    def compression_ratio(self) -> float:
        """fp16 bytes over stored bytes (packed codes + f32 norm) per vector."""
        return 2.0 * self.head_dim / (self.packed_bytes + 4)

    def memory_report(self, seq_len: int, num_layers: int = 32, num_kv_heads: int = 8) -> dict:
        """KV-cache bytes of one sequence of `seq_len` tokens over `num_layers`
        layers of `num_kv_heads` kv heads (K and V), fp16 against this codec
        (packed codes plus one f32 norm per vector)."""
        vectors = 2 * int(num_layers) * int(num_kv_heads) * int(seq_len)
        fp16 = vectors * 2 * self.head_dim
        packed = vectors * (self.packed_bytes + 4)
        return {"vectors": vectors, "fp16_bytes": fp16, "packed_bytes": packed, "saved_bytes": fp16 - packed,
                "compression_ratio": fp16 / packed, "bits": self.bits, "head_dim": self.head_dim}

    def validate(self, num_vectors: int = 10000, seed: int = 0) -> dict:
        """Encode and decode `num_vectors` seeded N(0,1) fp16 vectors on the
        current device and report the reconstruction: mean relative squared
        error ||x - x_hat||^2 / ||x||^2, mean cosine similarity, and the
        largest relative error of the stored norms."""
        import torch

        g = torch.Generator(device="cuda").manual_seed(int(seed))
        x = torch.randn(int(num_vectors), self.head_dim, generator=g, device="cuda").to(torch.float16)
        packed, norms = self.encode(x)
        xh = self.decode(packed, norms).float()
        xf = x.float()
        nx = xf.norm(dim=1)
        rel = ((xf - xh).pow(2).sum(dim=1) / nx.pow(2)).mean().item()
        cos = torch.nn.functional.cosine_similarity(xf, xh, dim=1).mean().item()
        nerr = ((norms - xf.double().norm(dim=1).float()).abs() / nx).max().item()
        return {"num_vectors": int(num_vectors), "mse_relative": rel, "cosine": cos, "max_norm_rel_err": nerr,
                "bits": self.bits, "head_dim": self.head_dim}

    def benchmark(self, num_vectors: int = 32768, reps: int = 20) -> dict:
        """Device time of one encode and one decode of `num_vectors` vectors
        (CUDA events around `reps` back-to-back calls after a warm-up), with
        the fp16-equivalent throughput (2 * head_dim bytes per vector)."""
        import torch

        x = torch.randn(int(num_vectors), self.head_dim, device="cuda").to(torch.float16)
        packed, norms = self.encode(x)
        out = self.decode(packed, norms)
        res = {"num_vectors": int(num_vectors), "bits": self.bits, "head_dim": self.head_dim}
        for name, fn in (("encode", lambda: self.encode(x, out=(packed, norms))),
                         ("decode", lambda: self.decode(packed, norms, out=out))):
            for _ in range(3):
                fn()
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            for _ in range(int(reps)):
                fn()
            e1.record()
            torch.cuda.synchronize()
            t = e0.elapsed_time(e1) / int(reps) / 1e3
            res[f"{name}_us"] = t * 1e6
            res[f"{name}_GBps"] = 2.0 * self.head_dim * int(num_vectors) / t / 1e9
        return res

    def encode(self, x, out=None, stream=None):
        """[..., d] fp16 CUDA tensor -> ([..., d*b/8] uint8, [...] float32)."""
        import torch

        _require(x.is_cuda and x.dtype == torch.float16 and x.is_contiguous(), "x: contiguous fp16 CUDA tensor")
        _require(x.shape[-1] == self.head_dim, "last dim must be head_dim")
        lead = tuple(x.shape[:-1])
        n = x.numel() // self.head_dim
        if out is None:
            packed = torch.empty(lead + (self.packed_bytes,), dtype=torch.uint8, device=x.device)
            norms = torch.empty(lead, dtype=torch.float32, device=x.device)
        else:
            packed, norms = out
            _check(packed, "out packed", torch.uint8, numel=n * self.packed_bytes)
            _check(norms, "out norms", torch.float32, numel=n)
            _on_device(packed=packed, norms=norms)
        tq_encode(self.ctx, x, n, packed, norms, stream)
        return packed, norms

    def decode(self, packed, norms, out=None, stream=None):
        """([..., d*b/8] uint8, [...] float32) -> [..., d] fp16."""
        import torch

        _require(packed.is_cuda and packed.dtype == torch.uint8 and packed.is_contiguous(), "packed: uint8 CUDA")
        _require(packed.shape[-1] == self.packed_bytes, "last dim of packed must be head_dim*bits/8")
        _require(norms.dtype == torch.float32 and norms.is_contiguous(), "norms: contiguous float32")
        lead = tuple(packed.shape[:-1])
        n = packed.numel() // self.packed_bytes
        _require(norms.numel() == n, "norms must have one entry per vector")
        x = out if out is not None else torch.empty(lead + (self.head_dim,), dtype=torch.float16,
                                                    device=packed.device)
        _check(x, "out", torch.float16, numel=n * self.head_dim)
        _on_device(norms=norms, out=x)
        tq_decode(self.ctx, packed, norms, n, x, stream)
        return x

    def encode_append(self, x, cache_packed, cache_norms, slot, stream=None):
        """Write one token per sequence: x [n_seq, h, d] into cache slot[s]."""
        import torch

        _require(x.dim() == 3 and x.shape[-1] == self.head_dim, "x: [n_seq, h, head_dim]")
        n_seq, h, d = x.shape
        _require(cache_packed.dim() == 4, "cache_packed: [n_seq, s_max, h, P]")
        s_max = cache_packed.shape[1]
        _check(x, "x", torch.float16)
        _check(cache_packed, "cache_packed", torch.uint8, shape=(n_seq, s_max, h, self.packed_bytes))
        _check(cache_norms, "cache_norms", torch.float32, shape=(n_seq, s_max, h))
        _check(slot, "slot", torch.int32, numel=n_seq)
        _on_device(x=x, cache_packed=cache_packed, cache_norms=cache_norms, slot=slot)
        tq_encode_append(self.ctx, x, n_seq, h, cache_packed, cache_norms, s_max, slot, stream)

    def encode_append_kv(self, k, v, k_cache, k_norms, v_cache, v_norms, slot, stream=None):
        """Write the key and the value of one token per sequence in one launch:
        k, v [n_seq, h, d] into slot[s] of their caches [n_seq, s_max, h, P]."""
        import torch

        _require(k.dim() == 3 and k.shape[-1] == self.head_dim and tuple(v.shape) == tuple(k.shape),
                 "k, v: [n_seq, h, head_dim]")
        n_seq, h, d = k.shape
        _require(k_cache.dim() == 4, "k_cache: [n_seq, s_max, h, P]")
        s_max = k_cache.shape[1]
        for name, t in (("k", k), ("v", v)):
            _check(t, name, torch.float16)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _check(t, name, torch.uint8, shape=(n_seq, s_max, h, self.packed_bytes))
        for name, t in (("k_norms", k_norms), ("v_norms", v_norms)):
            _check(t, name, torch.float32, shape=(n_seq, s_max, h))
        _check(slot, "slot", torch.int32, numel=n_seq)
        _on_device(k=k, v=v, k_cache=k_cache, v_cache=v_cache, k_norms=k_norms, v_norms=v_norms, slot=slot)
        tq_encode_append_kv(self.ctx, k, v, n_seq, h, k_cache, k_norms, v_cache, v_norms, s_max, slot, stream)

    def encode_os(self, x, stream=None):
        """Offset + fp16-scale variant: x [..., d] fp16 -> (packed [..., P]
        uint8, side [...] int32 = fp16 offset | fp16 scale << 16)."""
        import torch

        _require(x.shape[-1] == self.head_dim, "last dim must be head_dim")
        _check(x, "x", torch.float16)
        _on_device(x=x)
        lead = x.shape[:-1]
        n = x.numel() // self.head_dim
        packed = torch.empty(*lead, self.packed_bytes, dtype=torch.uint8, device=x.device)
        side = torch.empty(lead, dtype=torch.int32, device=x.device)
        tq_encode_os(self.ctx, x, n, packed, side, stream)
        return packed, side

    def decode_os(self, packed, side, stream=None):
        import torch

        _require(packed.shape[-1] == self.packed_bytes, "last dim of packed must be head_dim*bits/8")
        lead = packed.shape[:-1]
        n = packed.numel() // self.packed_bytes
        _check(packed, "packed", torch.uint8)
        _check(side, "side", (torch.int32, torch.uint32), numel=n)
        _on_device(packed=packed, side=side)
        out = torch.empty(*lead, self.head_dim, dtype=torch.float16, device=packed.device)
        tq_decode_os(self.ctx, packed, side, n, out, stream)
        return out

    def encode_slots(self, x, cache_packed, cache_norms, slot_mapping, stream=None):
        """Encode-on-write: x [n_tok, h, d] into slot slot_mapping[t] of a pool
        cache_packed [num_slots, h, P] (or a paged pool [num_blocks, 16, h, P]),
        cache_norms likewise; negative slots are skipped."""
        import torch

        _require(x.dim() == 3 and x.shape[-1] == self.head_dim, "x: [n_tok, h, head_dim]")
        n_tok, h, d = x.shape
        _require(cache_packed.shape[-2] == h and cache_packed.shape[-1] == self.packed_bytes, "cache layout")
        num_slots = cache_packed.numel() // (h * self.packed_bytes)
        _check(x, "x", torch.float16)
        _check(cache_packed, "cache_packed", torch.uint8)
        _check(cache_norms, "cache_norms", torch.float32, numel=num_slots * h)
        _check(slot_mapping, "slot_mapping", torch.int32, numel=n_tok)
        _on_device(x=x, cache_packed=cache_packed, cache_norms=cache_norms, slot_mapping=slot_mapping)
        tq_encode_slots(self.ctx, x, n_tok, h, cache_packed, cache_norms, num_slots, slot_mapping, stream)


def attend_decode(q, k_codec: TurboQuant, v_codec: TurboQuant, k_packed, k_norms, v_packed, v_norms,
                  positions, out=None, workspace=None, stream=None):
    """One decode step of attention over packed caches.

    q [B, Hq, d] fp16; k_packed [B, S, Hkv, Pk] uint8; k_norms [B, S, Hkv] f32;
    v likewise; positions [B] int32 (valid cache length per sequence).
    Returns o [B, Hq, d] fp16.
    """
    import torch

    _require(q.dim() == 3 and k_packed.dim() == 4, "q: [B, Hq, d]; k_packed: [B, S, Hkv, Pk]")
    B, hq, d = q.shape
    s_max, hkv = k_packed.shape[1], k_packed.shape[2]
    _check(q, "q", torch.float16)
    _check(k_packed, "k_packed", torch.uint8, shape=(B, s_max, hkv, k_codec.packed_bytes))
    _check(v_packed, "v_packed", torch.uint8, shape=(B, s_max, hkv, v_codec.packed_bytes))
    _check(k_norms, "k_norms", torch.float32, shape=(B, s_max, hkv))
    _check(v_norms, "v_norms", torch.float32, shape=(B, s_max, hkv))
    _check(positions, "positions", torch.int32, numel=B)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", torch.float16, shape=(B, hq, d))
    ws_bytes = tq_attend_workspace_bytes(B, hq, d, s_max)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8)
    _on_device(q=q, k_packed=k_packed, v_packed=v_packed, k_norms=k_norms, v_norms=v_norms, positions=positions,
               out=out, workspace=workspace)
    tq_attend_decode(k_codec.ctx, v_codec.ctx, q, B, hq, hkv, k_packed, k_norms, v_packed, v_norms, s_max,
                     positions, out, workspace, workspace.numel(), stream)
    return out


class TQPagedAttention:
    """Decode-step attention over paged packed caches, in the form of the
    pages' `TQPagedAttention(tq, num_query_heads).forward(...)`: `tq` codes
    the keys and, unless `v_tq` is given, the values too."""

    def __init__(self, tq: TurboQuant, num_query_heads: int, v_tq: TurboQuant = None):
        self.k_codec, self.v_codec = tq, (v_tq if v_tq is not None else tq)
        self.num_query_heads = int(num_query_heads)

    def forward(self, query, k_packed, k_norms, v_packed, v_norms, block_tables, context_lens, out=None,
                workspace=None, stream=None):
        """query [B, num_query_heads, head_dim] fp16; caches [num_blocks, 16,
        Hkv, P]; block_tables [B, max_blocks] int32; context_lens [B] int32.
        Returns [B, num_query_heads, head_dim] fp16."""
        _require(query.dim() == 3 and query.shape[1] == self.num_query_heads,
                 "query must be [B, num_query_heads, head_dim]")
        return attend_decode_paged(query, self.k_codec, self.v_codec, k_packed, k_norms, v_packed, v_norms,
                                   block_tables, context_lens, out=out, workspace=workspace, stream=stream)

    __call__ = forward

    def step(self, query, key, value, positions, slot_mapping, k_packed, k_norms, v_packed, v_norms, block_tables,
             context_lens, window=None, sinks=0, q_offsets=None, max_q=None, inv_freq=None, interleaved=False,
             rope_scale=1.0, q_weight=None, k_weight=None, eps=1e-6, stream=None):
        """One layer's attention for the new tokens of a batch, from their
        projections on: `qk_norm_rope` of query [T, num_query_heads, d] and
        key [T, Hkv, d] at `positions` [T], `encode_slots` of keys and values
        [T, Hkv, d] fp16 to slot_mapping [T] of the pools, then
        `attend_window_paged`. The tables and context_lens include the new
        tokens. Returns [T, num_query_heads, d] fp16. Arguments are refused
        before anything is written to the pools."""
        import torch

        _require(query.dim() == 3 and query.shape[1] == self.num_query_heads,
                 "query must be [T, num_query_heads, head_dim]")
        _require(value.dim() == 3 and value.shape == key.shape, "value: the key's shape")
        _require(not (value.requires_grad and torch.is_grad_enabled()),
                 "value: requires a gradient, which this call does not compute (detach it, or call under "
                 "torch.no_grad())")
        q, k = qk_norm_rope(query, key, positions, inv_freq, interleaved=interleaved, rope_scale=rope_scale,
                            q_weight=q_weight, k_weight=k_weight, eps=eps, stream=stream)
        _require(value.device == q.device, f"value: on {q.device} like the query, got {value.device}")
        _check(slot_mapping, "slot_mapping", torch.int32, numel=key.shape[0])
        _require(slot_mapping.device == q.device, f"slot_mapping: on {q.device} like the query, got {slot_mapping.device}")
        _calls().check_attend_window(q, self.k_codec.ctx.address, self.v_codec.ctx.address, k_packed, k_norms,
                                     v_packed, v_norms, True, block_tables, context_lens, window, sinks, q_offsets,
                                     max_q, None, None)
        with _launching(q.device, stream):
            value = value.half().contiguous()
            self.k_codec.encode_slots(k, k_packed, k_norms, slot_mapping)
            self.v_codec.encode_slots(value, v_packed, v_norms, slot_mapping)
        return attend_window_paged(q, self.k_codec, self.v_codec, k_packed, k_norms, v_packed, v_norms, block_tables,
                                   context_lens, window=window, sinks=sinks, q_offsets=q_offsets, max_q=max_q,
                                   stream=stream)


def attend_decode_paged(q, k_codec: TurboQuant, v_codec: TurboQuant, k_cache, k_norms, v_cache, v_norms,
                        block_tables, context_lens, out=None, workspace=None, stream=None):
    """One decode step of attention over paged packed caches.

    q [B, Hq, d] fp16; k_cache [num_blocks, 16, Hkv, Pk] uint8; k_norms
    [num_blocks, 16, Hkv] f32; v likewise; block_tables [B, max_blocks] int32
    (block of positions [16 j, 16 j + 16) of sequence b); context_lens [B]
    int32. Returns o [B, Hq, d] fp16.
    """
    import torch

    _require(q.dim() == 3 and k_cache.dim() == 4 and block_tables.dim() == 2,
             "q: [B, Hq, d]; k_cache: [num_blocks, 16, Hkv, Pk]; block_tables: [B, max_blocks]")
    B, hq, d = q.shape
    num_blocks, blk, hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    _require(blk == TQ_PAGE_BLOCK, f"cache blocks must hold {TQ_PAGE_BLOCK} positions")
    max_blocks = block_tables.shape[1]
    _check(q, "q", torch.float16)
    _check(k_cache, "k_cache", torch.uint8, shape=(num_blocks, blk, hkv, k_codec.packed_bytes))
    _check(v_cache, "v_cache", torch.uint8, shape=(num_blocks, blk, hkv, v_codec.packed_bytes))
    _check(k_norms, "k_norms", torch.float32, shape=(num_blocks, blk, hkv))
    _check(v_norms, "v_norms", torch.float32, shape=(num_blocks, blk, hkv))
    _check(block_tables, "block_tables", torch.int32, shape=(B, max_blocks))
    _check(context_lens, "context_lens", torch.int32, numel=B)
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", torch.float16, shape=(B, hq, d))
    ws_bytes = tq_attend_workspace_bytes(B, hq, d, max_blocks * TQ_PAGE_BLOCK)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8)
    _on_device(q=q, k_cache=k_cache, v_cache=v_cache, k_norms=k_norms, v_norms=v_norms, block_tables=block_tables,
               context_lens=context_lens, out=out, workspace=workspace)
    tq_attend_decode_paged(k_codec.ctx, v_codec.ctx, q, B, hq, hkv, k_cache, k_norms, v_cache, v_norms, num_blocks,
                           block_tables, max_blocks, context_lens, out, workspace, workspace.numel(), stream)
    return out


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq [rot_dim / 2] float64 on `device`, rope_scale) for
    `qk_norm_rope`: f_i = base^(-2 i / rot_dim), stretched by `factor` for
    contexts beyond the `original_len` positions of training.

    scaling: None; "linear" (every frequency divided by factor); "ntk" (the
    base grows so that the lowest frequency is divided by factor and the
    highest kept); "yarn" (frequencies of more than beta_fast turns within
    original_len kept, of fewer than beta_slow divided by factor, between them
    a linear ramp over the index, whose ends are rounded outward to whole
    indices within 0 ... rot_dim - 1, and rope_scale 1 + 0.1 ln(factor)).
    """
    import math

    import torch

    _require(rot_dim >= 2 and rot_dim % 2 == 0, "rot_dim: even, at least 2")
    _require(scaling in (None, "linear", "ntk", "yarn"), "scaling: None, 'linear', 'ntk' or 'yarn'")
    _require(factor >= 1.0 and base > 1.0 and original_len > 0, "factor >= 1, base > 1, original_len > 0")
    _require(scaling != "ntk" or rot_dim > 2, "ntk: rot_dim of at least 4")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = float(base) ** (-2 * i / rot_dim)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        _require(beta_fast > beta_slow > 0, "beta_fast > beta_slow > 0")
        # the ramp runs over the index i, between those at which a frequency turns beta_fast and beta_slow times;
        # its upper end may lie behind the last index (every frequency turns more than beta_slow times)
        at = [rot_dim * math.log(original_len / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow)]
        hi = min(math.ceil(at[1]), rot_dim - 1)
        lo = min(max(math.floor(at[0]), 0), hi - 1)
        ramp = ((i - lo) / (hi - lo)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(device), scale


def qk_norm_rope(q, k, positions, inv_freq=None, *, interleaved: bool = False, rope_scale: float = 1.0,
                 q_weight=None, k_weight=None, eps: float = 1e-6, out=None, stream=None):
    """Norm of every query and key head and rotation by position.

    q [T, Hq, d], k [T, Hkv, d] fp16 or bf16 (views of one projection's output
    are fine: rows dense, strides multiples of 8); positions [T] int32;
    inv_freq [rot / 2] float64 (`rope_frequencies`), None for no rotation;
    interleaved pairs (2i, 2i + 1) or half layout (i, i + rot / 2); weights [d]
    in q's dtype or float32, None for no norm of that tensor. Returns (q, k)
    fp16 [T, H, d]: keys as `encode_slots` takes them, queries as the attention
    calls do. `out` = (q_out, k_out), which may be q and k where they are
    contiguous fp16, and share no memory with the inputs otherwise. Forward
    only: tensors that require a gradient are refused while one is recorded.
    """
    args = (q, k, positions, inv_freq, interleaved, rope_scale, q_weight, k_weight, eps, out)
    if stream is not None:
        return _on_stream(stream, "q", q, _calls().qk_norm_rope, *args)
    return _calls().qk_norm_rope(*args)


def attend_window(q, k_codec: TurboQuant, v_codec: TurboQuant, k_packed, k_norms, v_packed, v_norms, context_lens,
                  window=None, sinks: int = 0, q_offsets=None, max_q=None, out=None, workspace=None, stream=None):
    """Causal attention of one or more query tokens per sequence over packed
    caches, within the last `window` positions (None: all) and the first
    `sinks`.

    q [T, Hq, d] fp16; caches [B, S, Hkv, P] uint8 and norms [B, S, Hkv] f32 as
    `attend_decode`; context_lens [B] int32, the query tokens included (their
    keys and values are in the cache); q_offsets [B + 1] int32: sequence b's
    tokens are q[q_offsets[b]:q_offsets[b + 1]], at most max_q of them (None:
    one token per sequence). Returns o [T, Hq, d] fp16 (rows of tokens in no
    sequence are not written). `out` may be q itself and shares no memory with
    anything else. Forward only, as `qk_norm_rope`.

    Sums and scores are float32; codebook levels enter the products as fp16
    (within 7e-5 of a level at 4 bits, 1.5e-5 at 3, 1.7e-6 at 2), queries and
    weights times norms as two fp16 parts (22 bits). One kernel and one number
    of splits serve the whole call, chosen from max_q: prompt chunks and single
    tokens of one batch are faster in two calls.
    """
    args = (q, k_codec.ctx.address, v_codec.ctx.address, k_packed, k_norms, v_packed, v_norms, False, None,
            context_lens, window, sinks, q_offsets, max_q, out, workspace)
    if stream is not None:
        return _on_stream(stream, "q", q, _calls().attend_window, *args)
    return _calls().attend_window(*args)


def attend_window_paged(q, k_codec: TurboQuant, v_codec: TurboQuant, k_cache, k_norms, v_cache, v_norms,
                        block_tables, context_lens, window=None, sinks: int = 0, q_offsets=None, max_q=None,
                        out=None, workspace=None, stream=None):
    """`attend_window` over paged caches: pools [num_blocks, 16, Hkv, P] and
    block_tables [B, max_blocks] int32 as `attend_decode_paged`. Table entries
    of pages that no query sees are not read, so they may be negative
    (`pages_trim`)."""
    args = (q, k_codec.ctx.address, v_codec.ctx.address, k_cache, k_norms, v_cache, v_norms, True, block_tables,
            context_lens, window, sinks, q_offsets, max_q, out, workspace)
    if stream is not None:
        return _on_stream(stream, "q", q, _calls().attend_window, *args)
    return _calls().attend_window(*args)


def pages_trim(block_tables, context_lens, refs, window=None, sinks: int = 0, release=None, out=None, stream=None):
    """Give pages back: all pages of rows with release[row] true (their length
    becomes 0), and of the others those that no query of `attend_window_paged`
    with this window and sinks sees any more (window None: none of them; 0: a
    window of no positions, every whole page behind the sinks).

    block_tables [rows, max_blocks], context_lens [rows], refs [num_blocks]
    int32; release [rows] bool or uint8, or None. Returns new (block_tables,
    context_lens, refs), written to `out` where given (its tensors may be the
    inputs themselves).
    """
    args = (block_tables, context_lens, refs, window, sinks, release, out)
    if stream is not None:
        return _on_stream(stream, "refs", refs, _calls().pages_trim, *args)
    return _calls().pages_trim(*args)


class TQPagePools:
    """The pools of a paged cache that share one page numbering: codes and
    norms, keys and values, of every layer. `tensors`: contiguous CUDA tensors
    [num_blocks, ...] on one device, each page a multiple of 16 bytes (views of
    stacked layers are fine). Holds references to them."""

    def __init__(self, tensors):
        import torch

        tensors = list(tensors)
        _require(0 < len(tensors) <= TQ_MAX_PAGE_POOLS, f"pools: 1 to {TQ_MAX_PAGE_POOLS} tensors, got {len(tensors)}")
        for i, t in enumerate(tensors):
            _require(isinstance(t, torch.Tensor) and t.dim() >= 1 and t.numel() > 0, f"pool {i}: a tensor with pages")
            _require(t.is_contiguous(), f"pool {i}: contiguous")
            _require(t.shape[0] == tensors[0].shape[0], f"pool {i}: {tensors[0].shape[0]} pages, got {t.shape[0]}")
            _require(t.data_ptr() % 16 == 0, f"pool {i}: 16-byte aligned")
            size = t.numel() // t.shape[0] * t.element_size()
            _require(size % 16 == 0, f"pool {i}: pages of a multiple of 16 bytes, got {size}")
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors)
        _require(all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), "pools: tensors that do not overlap")
        self._dev = _one_device([f"pool {i}" for i in range(len(tensors))], tensors)
        self.tensors = tensors
        self.num_blocks = tensors[0].shape[0]
        self._array = (PagePool * len(tensors))()
        for i, t in enumerate(tensors):
            self._array[i].base = t.data_ptr()
            self._array[i].block_bytes = t.numel() // t.shape[0] * t.element_size()
        self._mine = (ctypes.addressof(self._array), len(tensors), self.num_blocks, self._dev)

    def fork(self, block_tables, context_lens, refs, parents, children, out=None, workspace=None, stream=None):
        """Make row children[i] a copy of row parents[i]: the parent's full
        pages are shared, a partly filled last page is copied to the lowest
        free page. parents, children [n] int32; other tensors as `pages_trim`.
        A child's former pages are not given back (`pages_trim` first). No
        tensor shares memory with a pool, `workspace` with none at all. Returns
        (block_tables, context_lens, refs)."""
        args = (*self._mine, block_tables, context_lens, refs, parents, children, out, workspace)
        if stream is not None:
            return _on_stream(stream, "refs", refs, _calls().pages_fork, *args)
        return _calls().pages_fork(*args)

    def compact(self, block_tables, refs, out=None, workspace=None, stream=None):
        """Move the used pages (refs > 0) to the front of the pools. Returns
        (block_tables, refs, remap, used): the tables with the new page
        numbers, the moved counts, the new number of every page (-1: free) and
        the number of used pages [1] int32. `out` = (block_tables, refs, remap,
        used); the first two may be the inputs themselves."""
        args = (*self._mine, block_tables, refs, out, workspace)
        if stream is not None:
            return _on_stream(stream, "refs", refs, _calls().pages_compact, *args)
        return _calls().pages_compact(*args)
