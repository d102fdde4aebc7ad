"""Plain implementations in 64 bits of the rotary and paged-cache operators, and the error
bounds their tests use (CPU only).

Bounds.  u = eps / 2 of the element type is the relative error of one rounding.
Rotation: y is a sum of two products of 16-bit inputs with a sine and a cosine.  The angle's
fraction of a turn is rounded to 2^-26 turns at most (4e-7 rad once the top 32 bits are
taken), sincospif is good to 2^-22, the fp32 products and the sum to 2^-23: together below
1e-6 of |x1| + |x2|, times the magnitude.  The result is rounded once: u |y|.
Attention: the weights are rounded to the element type and divided by the sum of the rounded
weights, so the output moves by at most u / (1 - u) sum_j p_j |v_j - O|; in fp16 weights below
2^-14 of a weight of 1 also move by up to 2^-25 each, the largest weight of a row being at
least 2^-8 after the rescale's slack of 2^8; scores carry an fp32 accumulation error of at
most d 2^-23 scale sum |q k|, which moves a weight relatively by the same; the sums of
weights and of P V, the exponentials and the merge are fp32 (2e-5 of sum p |v| covers them for
the lengths here).  The output is rounded once: u |O|."""
import math

import numpy as np
import torch


def inv_freq(rot, base=10000.0, scaling="none", factor=1.0, length=None):
    i = np.arange(rot // 2)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((length * f / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        return (1 - g) * f / factor + g * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, positions, rot, layout, f, mag, sign=1.0):
    """x [B, h, N, d] (torch, any type), positions [B, N]; returns (y, bound without u |y|)."""
    x = x.double().numpy()
    a = positions.double().numpy()[:, None, :, None] * f
    c, s = np.cos(a) * mag, np.sin(a) * mag * sign
    y, e = x.copy(), np.zeros_like(x)
    if layout == "half":
        i1, i2 = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i1, i2 = slice(0, rot, 2), slice(1, rot, 2)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    e[..., i1] = e[..., i2] = 1e-6 * mag * (abs(x1) + abs(x2))
    return y, e


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(y, dtype):
    """Largest error of rounding y to the type (its smallest step included)."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return half_step(dtype) * np.abs(y) + tiny / 2


def gather(cache, table, slots):
    """[Hk, n, d] of one sequence's slots."""
    page = cache.shape[2]
    return cache[table[slots // page].long(), :, slots % page].transpose(0, 1)


def paged(q, k_cache, v_cache, table, cache_len, new_len, tree, scale, heads=None):
    """(o, lse, bound of o without rounding, bound of lse), all float64 numpy; of `heads`
    only, where given."""
    B, H, T, d = q.shape
    Hk = k_cache.shape[1]
    dtype = q.dtype
    u = half_step(dtype)
    o, ob = np.zeros((B, H, T, d)), np.zeros((B, H, T, d))
    lse, lb = np.full((B, H, T), -np.inf), np.zeros((B, H, T))
    for b in range(B):
        past, n = int(cache_len[b]), T if new_len is None else int(new_len[b])
        if n == 0:
            continue
        slots = torch.arange(past + n)
        seen = np.ones((n, past + n), bool)
        if tree is None:
            seen[:, past:] = np.tril(np.ones((n, n), bool))
        else:
            m = tree if tree.dim() == 2 else tree[b]
            seen[:, past:] = m[:n, :n].numpy() != 0
        K = gather(k_cache, table[b], slots).double().numpy()
        V = gather(v_cache, table[b], slots).double().numpy()
        for h in (range(H) if heads is None else heads):
            k, v = K[h // (H // Hk)], V[h // (H // Hk)]
            qq = q[b, h, :n].double().numpy()
            with np.errstate(all="ignore"):
                z = np.where(seen, scale * qq @ k.T, -np.inf)
                top = z.max(axis=1, keepdims=True)
                p = np.where(seen, np.exp(z - np.where(np.isinf(top), 0, top)), 0.0)
                total = p.sum(axis=1, keepdims=True)
                w = p / np.where(total > 0, total, 1)
                acc = np.abs(scale) * np.where(seen, np.abs(qq) @ np.abs(k).T, 0).max(axis=1, keepdims=True)
                for t in range(n):
                    s = seen[t]
                    if not s.any():
                        continue
                    x = w[t, s] @ v[s]
                    o[b, h, t] = x
                    spread = w[t, s] @ np.abs(v[s] - x)
                    es = d * 2.0 ** -23 * acc[t, 0]
                    ob[b, h, t] = (1.01 * u + 2 * es) * spread + 2e-5 * (w[t, s] @ np.abs(v[s]))
                    if dtype == torch.float16:
                        ob[b, h, t] += s.sum() * 2.0 ** -25 * 2.0 ** 8 / max(total[t, 0], 1.0) * \
                            np.abs(v[s] - x).max()
                    lse[b, h, t] = top[t, 0] + np.log(total[t, 0])
                    lb[b, h, t] = es + 2.0 ** -19 * (1 + abs(lse[b, h, t]))
    return o, lse, ob, lb


def check(name, got, want, bound):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    inf = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN in other places"
    assert np.array_equal(got[inf & ~np.isnan(want)], want[inf & ~np.isnan(want)]), name
    diff = np.abs(got[~inf] - want[~inf])
    off = diff - np.broadcast_to(bound, want.shape)[~inf]
    assert off.size == 0 or off.max() <= 0, \
        f"{name}: {diff.max():.3g} off, {off.max():.3g} beyond the bound"
