"""Plain restatement of the operators of a generation step (projections with 4-bit weights, beam selection, reordering
of cached beams) for the tests: numpy, in 64 bits, written from include/csa2.h.  Nothing of the library runs here."""
import numpy as np
import torch

PAGE = 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3(byte):
    """Values of E4M3 bytes."""
    b = np.asarray(byte, np.int64)
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(b & 128, -mag, mag)


def weights(codes, scales):
    """W [n][k] of codes [n][k / 2] and scales [n][k / 16]."""
    n = codes.shape[0]
    w = np.empty((n, codes.shape[1] * 2))
    w[:, 0::2], w[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    return (w.reshape(n, -1, 16) * e4m3(scales)[..., None]).reshape(n, -1)


def linear(x, w, alpha, bias=None):
    """(y, a bound on |fp32 y - y|): products of bf16 x and the weights are exact; sums of 8 or 16 products are added
    in fp32, off by up to two steps of 2^-24 of what has been summed so far, some k / 8 times, and a few more where
    parts join; x as f16 relative to its row's largest is off by 2^-40 of that where it is small; the sum times alpha
    plus bias is rounded once (2^-24 of the result and of the bias)."""
    y = alpha * (x @ w.T)
    mag = abs(alpha) * (np.abs(x) @ np.abs(w).T)
    most = np.abs(x).max(1, keepdims=True, initial=0.0)
    tol = (x.shape[1] / 8 + 64) * 2.0 ** -23 * mag + 2.0 ** -40 * abs(alpha) * most * np.abs(w).sum(1)
    if bias is not None:
        y = y + bias
        tol = tol + 2.0 ** -24 * np.abs(bias)
    return y, tol + 2.0 ** -24 * np.abs(y) + 1e-37


def beam_select(logits, cum, take, done=None, end=0):
    """(scores [g][take], parents, tokens, lse, bound on |lse - exact|) of logits [g * k][v]: an exponential is off by
    2^-22 of itself (one exp2) and its argument by two steps of 2^-24, so it by that times its distance; a lane adds 64 of
    them in fp32."""
    groups, k = cum.shape
    x = np.asarray(logits, np.float64).reshape(groups, k, -1)
    x = np.where(np.isnan(x) | (x == np.inf), -np.inf, x)
    cum = np.where(np.isnan(cum) | (cum == np.inf), -np.inf, np.asarray(cum, np.float64))
    v = x.shape[-1]
    top = x.max(-1, keepdims=True)
    some = top > -np.inf
    d = np.where(np.isfinite(x), x, 0) - np.where(some, top, 0)
    e = np.where(np.isfinite(x), np.exp(d), 0)
    total = e.sum(-1)
    logs = np.log(np.where(total > 0, total, 1))
    lse = np.where(some[..., 0], np.where(some, top, 0)[..., 0] + logs, -np.inf)
    off = np.where(total > 0, (e * (2.0 ** -22 + 2.0 ** -22 * np.abs(d))).sum(-1) / np.where(total > 0, total, 1), 0)
    off = off + 66 * 2.0 ** -24
    # (relative to the largest: beside logits near fp32's lowest the other terms would be lost)
    s = np.where(np.isfinite(x), d, -np.inf) + cum[..., None] - logs[..., None]
    if done is not None:
        for g, b in zip(*np.nonzero(done)):
            s[g, b], lse[g, b], off[g, b] = -np.inf, 0.0, 0.0
            s[g, b, end] = cum[g, b]
    scores, parents, tokens = np.full((groups, take), -np.inf), np.full((groups, take), -1), np.full((groups, take), -1)
    for g in range(groups):
        flat = s[g].ravel()
        at = np.argsort(-flat, kind="stable")[:take]
        at = at[flat[at] > -np.inf]
        n = len(at)
        scores[g, :n], parents[g, :n], tokens[g, :n] = flat[at], g * k + at // v, at % v
    return scores, parents, tokens, lse.reshape(-1), off.reshape(-1)


def reorder(table, parents, length, beams):
    """(new table, copies (group's) as (from page, to page, slots)) of one call; length [groups]."""
    new, copies = table.copy(), []
    for g in range(table.shape[0] // beams):
        mine = range(g * beams, (g + 1) * beams)
        n, rest = divmod(int(length[g]), PAGE)
        keeper = {}
        for i in mine:
            if parents[i] >= 0 and (parents[i] not in keeper or parents[i] == i):
                keeper[parents[i]] = i
        free = [i for i in mine if i not in keeper]
        for i in mine:
            p = parents[i]
            if p >= 0:
                new[i, :n] = table[p, :n]
            if p >= 0 and keeper[p] == i:
                if rest:
                    new[i, n] = table[p, n]
                continue
            take = free.pop(0)
            if rest:
                new[i, n] = table[take, n]
                if p >= 0:
                    copies.append((table[p, n], table[take, n], rest))
    return new, copies


def bf16_tensor(x):
    return torch.from_numpy(np.asarray(x, np.float64)).float().to(torch.bfloat16)
