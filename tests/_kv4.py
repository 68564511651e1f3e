"""The 4-bit K/V cache in plain numpy and torch, for the tests: its format from
the definition (IEEE fp32 divisions, nearest code with ties to even), and the
attention over it in 64 bits."""

import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
# every E4M3 code's value: 0x7F / 0xFF are NaN
E4M3 = np.array([(-1.0) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if (c >> 3 & 15) == 0 else
                                       (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                 if (c & 127) != 127 else np.nan for c in range(256)])


def nearest(values, x):
    """Index of the nearest of ascending values, ties to the even index, the
    last one where x is larger."""
    i = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo, hi = x - values[i - 1], values[i] - x
    return np.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)


def quantize(x, s):
    """Codes [.., D] and scale codes [.., D/16] of x [.., D] (fp32 holding BF16
    values, no NaN) at the fp32 scale s."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = np.float32(s)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        top = np.abs(g).max(-1) / (np.float32(6) * s)
        sc = nearest(E4M3[:127], top.astype(np.float64)).astype(np.uint8)
        by = (E4M3[sc].astype(np.float32) * s)[..., None]
        t = np.where(by > 0, g / by, np.float32(0)).astype(np.float64)
        code = nearest(E2M1, np.abs(t)).astype(np.uint8) | (np.signbit(t).astype(np.uint8) << 3)
    return code.reshape(x.shape), sc


def regions(cache):
    """K codes, V codes, K scales, V scales of cache bytes [.., 18 D]."""
    d = cache.shape[-1] // 18
    cut = [8 * d, 16 * d, 17 * d]
    a, b, c, e = (cache[..., lo:hi] for lo, hi in zip([0] + cut, cut + [18 * d]))
    return tuple(x.reshape(*cache.shape[:-1], 16, x.shape[-1] // 16) for x in (a, b, c, e))


def values(code_bytes, scale_bytes, s):
    """fp64 values of bytes of codes [.., D/2] and scales [.., D/16] (torch)."""
    lut = torch.tensor(np.concatenate([E2M1, -E2M1]), device=code_bytes.device)
    e4 = torch.tensor(E4M3, device=code_bytes.device)
    c = code_bytes.long()
    v = lut[torch.stack([c & 15, c >> 4], -1).flatten(-2)]
    return v * e4[scale_bytes.long()].repeat_interleave(16, -1) * float(s)


def attention(q, cu_q, kv_lens, table, cache, s_k, s_v, scale, causal):
    """(out, lse, spread, reach) in fp64: spread = sum_j p_j |v_j| and reach =
    max_j scale |q| . |k_j| bound the errors of the fp32 computation.  Rows
    outside every request are NaN in out.  Pages that the cache lacks are not
    seen."""
    pages, heads, strips, _ = cache.shape
    page, dim = 16 * strips, cache.shape[3] // 18
    total, hq, _ = q.shape
    g = hq // heads
    new = dict(dtype=torch.float64, device=q.device)
    out = torch.full(q.shape, math.nan, **new)
    lse = torch.full((total, hq), math.nan, **new)
    spread, reach = torch.zeros(q.shape, **new), torch.zeros((total, hq), **new)
    cu = cu_q.tolist()
    for b, kv in enumerate(kv_lens.tolist()):
        lo, hi = min(max(cu[b], 0), total), min(cu[b + 1], total)
        n, kv = max(hi - lo, 0), min(max(kv, 0), page * table.shape[1])
        if n == 0:
            continue
        ids = table[b, :-(-kv // page)].long()
        there = (ids >= 0) & (ids < pages)
        x = cache[ids.clamp(0, max(pages - 1, 0))] if kv else cache[:0]
        kc, vc, ks, vs = regions(x)
        i = torch.arange(n, device=q.device)[:, None]
        j = torch.arange(kv, device=q.device)[None]
        sees = there.repeat_interleave(page)[:kv][None].expand(n, -1)
        if causal:
            sees = sees & (j <= kv - n + i)
        for h in range(heads):
            k = values(kc[:, h], ks[:, h], s_k).flatten(0, -2)[:kv]
            v = values(vc[:, h], vs[:, h], s_v).flatten(0, -2)[:kv]
            v = torch.where(there.repeat_interleave(page)[:kv, None], v, torch.zeros_like(v))
            for r in range(h * g, (h + 1) * g):
                qq = q[lo:hi, r].double()
                z = (qq @ k.t() * scale).masked_fill(~sees, -math.inf)
                p = torch.where(sees.any(1, keepdim=True), torch.softmax(z, 1), torch.zeros_like(z))
                out[lo:hi, r] = p @ v
                spread[lo:hi, r] = p @ v.abs()
                lse[lo:hi, r] = torch.logsumexp(z, 1) if kv else -math.inf
                if kv:
                    reach[lo:hi, r] = ((qq.abs() @ k.abs().t()) * abs(scale) * sees).amax(1)
    return out, lse, spread, reach
