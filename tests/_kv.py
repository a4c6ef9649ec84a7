"""Plain restatement of the paged key / value operators for the tests: numpy, attention in fp64, encodings by the
oracle's codecs, written from include/csa2.h.  Nothing of the library runs here."""
import math

import numpy as np
import torch

import compressed_sparse_attention_07_gb300 as csa
import oracle

PAGE = 64


def bf16(x):
    """Values of x rounded to bf16 (nearest even), as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().to(torch.bfloat16).double().numpy()


def normal(rng, *shape, std=1.0):
    return bf16(rng.standard_normal(shape) * std)


def fp4_round(x):
    """(stored values, codes [..., D/2], scales [..., D/16]) of rows x in FP4."""
    D, lead = x.shape[-1], x.shape[:-1]
    if x.size == 0:
        return np.zeros(x.shape), np.zeros(lead + (D // 2,), np.uint8), np.zeros(lead + (D // 16,), np.uint8)
    codes, scales = oracle.fp4_encode(np.asarray(x, np.float64).reshape(1, -1))  # groups of 16 stand alone
    val = oracle.fp4_decode(codes, scales)
    return val.reshape(x.shape), codes.reshape(*lead, D // 2), scales.reshape(*lead, D // 16)


def rope_rows(n, dims, theta=1e4):
    half = dims // 2
    a = np.arange(n)[:, None] * theta ** (-np.arange(half) / half)
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def rotate(x, table, pos, dims, half):
    """Rows x [T][H][D] at positions pos: products and sums rounded to fp32 one by one."""
    out = x.astype(np.float32)
    if dims:
        c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
        a, b = ((out[..., : dims // 2], out[..., dims // 2: dims]) if half
                else (out[..., 0:dims:2], out[..., 1:dims:2]))
        u, w = (a * c).astype(np.float32) - b * s, (a * s).astype(np.float32) + b * c
        if half:
            out[..., : dims // 2], out[..., dims // 2: dims] = u, w
        else:
            out[..., 0:dims:2], out[..., 1:dims:2] = u, w
    return out


def fill(cache, cfg, b, kind, x, start=0):
    """Write rows x [n][H][D] of sequence b (already values of the cache's type) into its pages at start .. start + n."""
    table = cache.block_table.cpu().numpy()
    data = cache.k_data if kind == "k" else cache.v_data
    scales = cache.k_scales if kind == "k" else cache.v_scales
    n, dev = x.shape[0], data.device
    j = np.arange(start, start + n)
    page, slot = torch.from_numpy(table[b, j // PAGE].astype(np.int64)).to(dev), torch.from_numpy(j % PAGE).to(dev)
    if cfg.cache_dtype == csa.CACHE_FP4:
        _, codes, sc = fp4_round(x)
        data[page, :, slot] = torch.from_numpy(codes).to(dev)
        scales[page, :, slot] = torch.from_numpy(sc).to(dev)
    else:
        v = torch.from_numpy(x).float().to(torch.bfloat16).to(dev)
        data[page, :, :, slot] = v.reshape(n, cfg.kv_heads, cfg.head_dim // 8, 8)


def read(cache, cfg, b, kind, n):
    """Rows [n][H][D] of sequence b as fp64 values, by the documented layout; and FP4's codes and scales."""
    table = cache.block_table.cpu().numpy()
    data = (cache.k_data if kind == "k" else cache.v_data).cpu()
    scales = cache.k_scales if kind == "k" else cache.v_scales
    j = np.arange(n)
    page, slot = table[b, j // PAGE], j % PAGE
    if cfg.cache_dtype == csa.CACHE_FP4:
        codes = data.numpy()[page, :, slot]
        sc = scales.cpu().numpy()[page, :, slot]
        val = oracle.fp4_decode(codes.reshape(1, -1), sc.reshape(1, -1)) if n else np.zeros(0)
        return val.reshape(n, cfg.kv_heads, cfg.head_dim), codes, sc
    v = data.double().numpy()[page, :, :, slot]
    return v.reshape(n, cfg.kv_heads, cfg.head_dim), None, None


def attend(q, k, v, scale, causal, window=0):
    """One sequence: q [n][Hq][D], k, v [m][H][D] in fp64 -> out, lse, and for the tolerances sum p |v| and, over
    the seen keys, the largest scale sum |q||k| and scale max |q| sum |k|."""
    n, hq, D = q.shape
    m, h = k.shape[:2]
    out, lse = np.zeros((n, hq, D)), np.full((n, hq), -np.inf)
    mag, dot, big = np.zeros((n, hq, D)), np.zeros((n, hq)), np.zeros((n, hq))
    pos = m - n + np.arange(n)
    see = np.ones((n, m), bool)
    if causal:
        see = np.arange(m) <= pos[:, None]
        if window:
            see &= np.arange(m) > pos[:, None] - window
    for a in range(hq):
        kk, vv = k[:, a * h // hq], v[:, a * h // hq]
        x = np.where(see, q[:, a] @ kk.T * scale, -np.inf)
        some = see.any(1)
        if not some.any():
            continue
        top = x[some].max(1, keepdims=True)
        p = np.exp(x[some] - top)
        l = p.sum(1, keepdims=True)
        out[some, a], lse[some, a] = p @ vv / l, (top + np.log(l))[:, 0]
        mag[some, a] = p @ np.abs(vv) / l
        dot[some, a] = np.where(see, np.abs(q[:, a]) @ np.abs(kk).T, 0)[some].max(1) * abs(scale)
        big[some, a] = (np.abs(q[:, a]).max(1, keepdims=True) * np.where(see, np.abs(kk).sum(1), 0))[some].max(1) * abs(scale)
    return out, lse, mag, dot, big


def tolerances(cfg, keys, out, lse, mag, dot, big):
    """Bounds on |out - exact| and |lse - exact| by counting roundings (u32 = 2^-24):
    - a logit is a sum of head_dim products in fp32, then scaled and the maximum subtracted in fp32: off by
      (head_dim + 8) u32 of the sum of magnitudes; over FP4 its query is an f16 relative to the row's largest channel
      (channels below 2^-14 of it are off by up to 2^-25 of it).  That moves every weight by that relative amount, and
      the weights' sum by as much;
    - a weight is one exp2 (2^-22) and one rounding to the second product's operand type: f16 (2^-11, or 2^-25
      absolute below 2^-14) for FP4 caches, bf16 (2^-8) else;
    - weights and products are added in fp32: keys u32 of the sum of magnitudes, and once more for the maximum's
      changes and the parts' join;
    - the output is rounded once to bf16 (2^-8)."""
    u32 = 2.0 ** -24
    logit = (cfg.head_dim + 8) * u32 * dot + 2.0 ** -24 * big
    weight = 2.0 ** -11 if cfg.cache_dtype == csa.CACHE_FP4 else 2.0 ** -8
    rel = weight + 2.0 ** -22 + 2 * np.expm1(logit) + (2 * keys + 64) * u32
    tol = 2.0 ** -8 * np.abs(out) + mag * (rel[..., None] if np.ndim(rel) else rel) * (1 + 2.0 ** -7)
    tol = tol + keys * 2.0 ** -25 * 8 * mag.max(initial=0.0) + 1e-30
    return tol, logit + 2.0 ** -21 + (2 * keys + 64) * u32 + 4 * u32 * np.abs(np.where(np.isfinite(lse), lse, 0)) + dot * 8 * u32


# ---- sharp checks of long sequences, in torch (on whatever device the rows are)

def attend_sums(q, k, v, scale, causal):
    """One sequence in fp64: q [n][Hq][D], k, v [m][H][D] -> out, sqrt(sum p^2 v^2), the same with min(p, 2^-25 of the
    row's largest p) for p [n][Hq][D], and the largest scale sum |q||k| over the seen keys [n][Hq]."""
    n, hq, D = q.shape
    m, h = k.shape[:2]
    out, root, low = (torch.zeros(n, hq, D, dtype=torch.float64, device=q.device) for _ in range(3))
    dot = torch.zeros(n, hq, dtype=torch.float64, device=q.device)
    see = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        see = torch.arange(m, device=q.device) <= (m - n + torch.arange(n, device=q.device))[:, None]
    for a in range(hq):
        kk, vv, qq = (x[:, i].double() for x, i in ((k, a * h // hq), (v, a * h // hq), (q, a)))
        p = torch.softmax((qq @ kk.T * scale).masked_fill(~see, -math.inf), 1)
        out[:, a], root[:, a] = p @ vv, (p ** 2 @ vv ** 2).sqrt()
        low[:, a] = (torch.minimum(p, 2.0 ** -25 * p.amax(1, keepdim=True)) ** 2 @ vv ** 2).sqrt()
        dot[:, a] = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(~see, 0).amax(1)
    return out, root, low, dot


def far(cfg, keys, got, out, root, low, dot):
    """How far `got` is from `out` in units of what roundings allow: (the farthest value, the farthest row by the root of
    its mean square).  Below 1 where a row's channels lie within 2^14 of one another.

    A weight is off by at most w of itself (rounded to f16 or bf16, an exp2, its logit of fp32 sums) or, rounded to f16,
    by 2^-25 of the row's largest; a value of the output by half a step of bf16, 2^-8 of itself; the fp32 sums by two
    steps of 2^-24 in each of some keys / 8 additions, of what has been summed so far (4 root and the output at most).
    Weights are rounded apart from one another, so that their errors, each within w p |v|, go either way: by Hoeffding
    their sum passes 7 sqrt(sum (w p v)^2) once in 2e10.  Errors of rounding spread evenly over an interval have a root
    of the mean square of its half / sqrt(3); over a row's 64 or 128 channels the mean is not four times its expectation."""
    u32 = 2.0 ** -24
    w = 2.0 ** -22 + 2 * torch.expm1((cfg.head_dim + 10) * u32 * dot)[..., None]
    if cfg.cache_dtype == csa.CACHE_FP4:
        off = (w + 2.0 ** -11) * root + low
    else:
        off = (w + 2.0 ** -8) * root
    sums = (keys / 8 + 64) * 2 * u32 * (4 * root + out.abs())
    err = (got.double() - out).abs()
    each = err / (2.0 ** -8 * out.abs() + (1 + 2.0 ** -8) * (7 * off + sums) + 1e-30)
    mean = (off ** 2 + (2.0 ** -8 * out) ** 2).mean(-1) / 3
    rms = err.square().mean(-1).sqrt() / (2 * mean.sqrt() + sums.square().mean(-1).sqrt() + 1e-30)
    return each.max().item(), rms.max().item()
