"""Plain 64-bit definitions of the cache operators (rotary append, exact
attention with token weights, eviction), on CPU tensors, and seeded inputs for
their tests.  Test infrastructure only."""
import math

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def paged(lens, page, Hkv, d, dtype, seed, *, spare=3, stale=float("nan"), width=None):
    """A paged cache for sequences of these lengths: (k, v [pages, Hkv, page,
    d], table [B, width]).  Rows no sequence holds, in used pages and in the
    `spare` unused ones, are `stale`; unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    blocks = [-(-max(0, n) // page) for n in lens]
    total = sum(blocks) + spare
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(lens), width or max(max(blocks), 1)), -1, dtype=torch.int32)
    k = torch.full((total, Hkv, page, d), stale, dtype=torch.float32)
    v = torch.full((total, Hkv, page, d), stale, dtype=torch.float32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :blocks[b]] = perm[at:at + blocks[b]].to(torch.int32)
        at += blocks[b]
        t = torch.arange(max(0, n))
        pg, row = table[b, t // page].long(), t % page
        k[pg, :, row] = torch.randn(len(t), Hkv, d, generator=g)
        v[pg, :, row] = torch.randn(len(t), Hkv, d, generator=g)
    return k.to(DT[dtype]), v.to(DT[dtype]), table


def rows(cache, table, b, h, n):
    """The first n rows of kv-head h of sequence b, [n, d] in 64 bits."""
    t = torch.arange(n)
    page = cache.shape[2]
    return cache[table[b, t // page].long(), h, t % page].double()


def attend(q, k, v, table, lens, scale=None):
    """out [B, Hq, d], lse [B, Hq], weights (list of [Hkv, n] sums over the
    group's heads) and, for the error bounds, size = scale * max_t sum
    |q||k|, top = max_t |x_t| and spread = sum_t w_t |v_t| per head."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = torch.zeros(B, Hq, d, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    size, top = torch.zeros(B, Hq, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    spread = torch.zeros(B, Hq, d, dtype=torch.float64)
    weights = []
    for b, n in enumerate(lens):
        n = max(0, int(n))
        wb = torch.zeros(Hkv, n, dtype=torch.float64)
        for h in range(Hkv):
            if n == 0:
                continue
            kk, vv = rows(k, table, b, h, n), rows(v, table, b, h, n)
            qq = q[b, h * G:(h + 1) * G].double()
            x = scale * (qq @ kk.T)
            hs = slice(h * G, (h + 1) * G)
            lse[b, hs] = torch.logsumexp(x, -1)
            w = torch.exp(x - lse[b, hs, None])
            out[b, hs] = w @ vv
            wb[h] = w.sum(0)
            size[b, hs] = scale * (qq.abs() @ kk.abs().T).amax(-1)
            top[b, hs] = x.abs().amax(-1)
            spread[b, hs] = w @ vv.abs()
        weights.append(wb)
    return out, lse, weights, size, top, spread


def logit_error(d, size, top, lse):
    """Bound on a logit's error (natural units) in the kernels: d fp32
    accumulation steps of at most 2^-23 of the magnitude sum (the matrix
    units may truncate), and rounding of the scaling, the differences to the
    maximum and the log-sum-exp (at most four halves of 2^-22 of their sizes)."""
    finite = torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    return (d + 2) * 2.0 ** -23 * size + 2.0 ** -22 * (top + finite)


def weight_error(d, n, size, top, lse):
    """Relative bound on a softmax weight: the logit's and the log-sum-exp's
    errors, ex2's 2^-21 and n fp32 additions in the sum."""
    return 2 * logit_error(d, size, top, lse) + 2.0 ** -20 + n * 2.0 ** -24


def turn_by(f, positions, amplitude=1.0):
    angle = np.multiply.outer(np.asarray(positions, dtype=np.float64), np.asarray(f, dtype=np.float64))
    return torch.from_numpy(amplitude * np.cos(angle)), torch.from_numpy(amplitude * np.sin(angle))


def rotate(x, cos, sin, rot, layout):
    """x [T, H, d] turned by [T, rot/2] cosines and sines, 64 bits."""
    y = x.double().clone()
    i = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    j = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    a, b = x.double()[..., i], x.double()[..., j]
    y[..., i] = a * cos[:, None] - b * sin[:, None]
    y[..., j] = a * sin[:, None] + b * cos[:, None]
    return y


def evict_kept(mass, n_tokens, budget, sink, recent):
    """Ascending kept rows of one unit; mass a 1-D float array."""
    n = max(0, int(n_tokens))
    keep = min(n, budget)
    if keep == n:
        return list(range(n))
    safe = [t for t in range(n) if t < sink or t >= n - recent]
    rest = [t for t in range(n) if not (t < sink or t >= n - recent)]
    val = lambda t: -math.inf if math.isnan(mass[t]) else float(mass[t])   # noqa: E731
    nan = lambda t: 1 if math.isnan(mass[t]) else 0                        # noqa: E731
    rest.sort(key=lambda t: (nan(t), -val(t), t))
    return sorted((safe + rest)[:keep])
