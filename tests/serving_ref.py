"""Plain 64-bit implementations of the operators around the packed cache
(norm and rotation of query and key heads, windowed attention, page
operations), and the tolerances of their fp16 outputs.

Tolerances. A rounding to fp16 is off by at most 2^-11 of the value (2^-25
below 2^-14), one to f32 by 2^-24.

* Norm and rotation: sums of squares are 8 terms in a lane and up to 5 tree
  levels, so the mean is off by less than 14 x 2^-24 and its root by half of
  that; root, quotient, weight and product add five roundings, the angle in
  turns one (times 2 pi), sine and cosine two, the rotation three: below
  32 x 2^-24 = 2^-19 of scale (|y_a| + |y_b|) together.
* Attention: the matrix operands are the levels rounded to fp16 after a common
  factor, off by at most EPS_LEVEL[bits] of a level, the query to 2^-21. A score
  is then off by ds = (EPS_LEVEL[K bits] + 2^-20) |q| |k| / sqrt(d) (Cauchy), a
  normalised weight by 2 ds + 2^-18 of itself (exponential, f32 sums), so the
  2-norm of an output row's error is at most
  2^-11 |o| + (EPS_LEVEL[V bits] + 2 max ds + 2^-17) sum_t p_t |v_t| + sqrt(d) 2^-25.
"""

import math

import torch

import oracle as O

EPS_LEVEL = {2: 1.7e-6, 3: 1.5e-5, 4: 7.0e-5}


def rope(x, weight, positions, inv_freq, interleaved, scale, eps):
    """(fp64 result, tolerance) of the norm and rotation of x [T, H, d]."""
    y = x.double()
    d = y.shape[-1]
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
    out, mag = y.clone(), y.abs()
    if inv_freq is not None:
        half = inv_freq.numel()
        ang = (positions.double()[:, None] * inv_freq)[:, None]
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ya, yb = y[..., a], y[..., b]
        out[..., a] = scale * (ya * ang.cos() - yb * ang.sin())
        out[..., b] = scale * (yb * ang.cos() + ya * ang.sin())
        both = abs(scale) * (ya.abs() + yb.abs())
        mag[..., a], mag[..., b] = both, both
    assert out.shape[-1] == d
    return out, out.abs() * 2.0 ** -11 + mag * 2.0 ** -19 + 2.0 ** -25


def decode_rows(packed, norms, bits, d, seed=42):
    """fp64 rows of packed codes (CUDA or CPU tensors) by the oracle."""
    return torch.from_numpy(O.decode_f64(packed.cpu().numpy(), norms.cpu().numpy(), bits, seed, d))


def attend(q, k, v, ctx, window, sinks, kb, vb):
    """One sequence: q [n, hq, d] fp16, k, v [L, hkv, d] fp64 (L >= ctx) ->
    (o [n, hq, d] fp64, row tolerance [n, hq] of the 2-norm of the error)."""
    q = q.cpu().double()
    n, hq, d = q.shape
    g = hq // k.shape[1]
    o = torch.zeros(n, hq, d, dtype=torch.float64)
    tol = torch.zeros(n, hq, dtype=torch.float64)
    for i in range(n):
        p = ctx - n + i
        t = [t for t in range(0, p + 1) if t < sinks or window is None or t > p - window]
        if not t:
            continue
        for h in range(hq):
            kk, vv = k[t, h // g], v[t, h // g]
            s = kk @ q[i, h] / math.sqrt(d)
            w = torch.softmax(s, 0)
            o[i, h] = w @ vv
            ds = (EPS_LEVEL[kb] + 2.0 ** -20) * q[i, h].norm() * kk.norm(dim=1).max() / math.sqrt(d)
            tol[i, h] = (2.0 ** -11 * o[i, h].norm() + (EPS_LEVEL[vb] + 2 * ds + 2.0 ** -17) * (w @ vv.norm(dim=1))
                         + math.sqrt(d) * 2.0 ** -25)
    return o, tol


def fork(table, lens, refs, parents, children):
    """(table, lens, refs, [(src, dst)], skipped, full) of a fork, on lists."""
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    old, old_lens, moves, skipped, full = [list(r) for r in table], list(lens), [], 0, 0
    free = [b for b, r in enumerate(refs) if r <= 0]
    rows, mb = len(table), len(table[0])
    for p, c in zip(parents, children):
        bad = not (0 <= p < rows and 0 <= c < rows) or list(children).count(c) > 1 or c in parents
        if bad:
            skipped += 1
            continue
        length = max(0, min(old_lens[p], 16 * mb))
        whole, row, fresh = length // 16, [-1] * mb, None
        last = old[p][whole] if length % 16 else -1
        if 0 <= last < len(refs):
            if not free:
                full += 1
                table[c], lens[c] = row, 0
                continue
            fresh = free.pop(0)
        for j in range(whole):
            if 0 <= old[p][j] < len(refs):
                row[j] = old[p][j]
                refs[row[j]] += 1
        if fresh is not None:
            row[whole] = fresh
            refs[fresh] = 1
            moves.append((last, fresh))
        table[c], lens[c] = row, length
    return table, lens, refs, moves, skipped, full


def trim(table, lens, refs, window, sinks, release):
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    for r, row in enumerate(table):
        length = min(lens[r], 16 * len(row))
        for j, e in enumerate(row):
            gone = release is not None and release[r]
            gone = gone or (window is not None and 16 * j >= sinks and 16 * j + 16 <= length - window)
            if gone and e >= 0:
                if e < len(refs):
                    refs[e] -= 1
                row[j] = -1
        if release is not None and release[r]:
            lens[r] = 0
    return table, lens, refs


def compact(table, refs):
    """(table, refs, remap, used, [(src, dst)])"""
    used = sum(r > 0 for r in refs)
    src = [b for b, r in enumerate(refs) if r > 0 and b >= used]
    dst = [b for b, r in enumerate(refs) if r <= 0 and b < used]
    remap = [b if r > 0 else -1 for b, r in enumerate(refs)]
    out = [r if r > 0 and b < used else 0 for b, r in enumerate(refs)]
    for s, d in zip(src, dst):
        remap[s] = d
        out[d] = refs[s]
    table = [[remap[e] if 0 <= e < len(refs) else -1 for e in row] for row in table]
    return table, out, remap, used, list(zip(src, dst))
