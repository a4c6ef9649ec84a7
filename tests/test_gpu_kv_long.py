"""Attention over long paged caches on the GPU, compared closely enough to see a single page lost or misplaced: by the
mean square of random values, and by queries that pick out one key each."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_07_gb300 as csa
from tests import _kv

pytestmark = pytest.mark.gpu

FP4, BF16 = csa.CACHE_FP4, csa.CACHE_BF16

# (query heads, kv heads, channels, new tokens, keys): up to 8, 16 and 32 rows of a kv head; up to 64 and 128, which share
# a tile's two places; 256 and more; the last wave of row tiles divided; pages decoded ahead
SHAPES = [(4, 4, 64, [1], [9000]), (16, 1, 128, [1], [6007]), (30, 1, 64, [1, 1, 1], [9000, 64, 6007]),
          (8, 2, 128, [7, 3], [6007, 5000]), (40, 1, 64, [1, 1], [9000, 4000]), (16, 2, 128, [5], [6007]),
          (48, 2, 64, [4], [9001]), (8, 2, 128, [70], [6007]), (6, 2, 64, [200, 90], [5003, 9000]),
          (256, 16, 64, [208], [2700]), (128, 1, 64, [40], [3001]), (128, 1, 128, [33], [3001])]


def _cache(cfg, keys, seed):
    """A cache with its rows as the kernels see them, [sum keys][kv heads][channels] on the GPU."""
    pages = len(keys) * -(-max(keys) // 64)
    order = np.random.default_rng(seed).permutation(pages + 3)[:pages]
    cache = csa.KVCache(cfg, len(keys), max(keys), page_order=order, spare_pages=3)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [torch.randn(sum(keys), cfg.kv_heads, cfg.head_dim, generator=g, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    stored = [torch.empty_like(x) for x in rows]
    cu = torch.tensor([0] + list(np.cumsum(keys)), dtype=torch.int32, device="cuda")
    csa.kv_append(cfg, *rows, cu, torch.zeros(len(keys), dtype=torch.int64, device="cuda"), cache, k_out=stored[0],
                  v_out=stored[1])
    return cache, stored


def _call(cfg, cache, q, nq, keys, cross, workspace, scale):
    cu = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device="cuda")
    lens = torch.tensor(keys, dtype=torch.int32, device="cuda")
    need = csa.kv_workspace_bytes(cfg, len(nq), sum(nq), max(nq), max(keys)) if workspace else 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    out, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    (csa.kv_cross_attend if cross else csa.kv_attend)(cfg, q, cu, cache, lens, max(nq), max(keys), out, scale=scale,
                                                     workspace=ws, status=st)
    assert int(st.item()) == 0
    return out


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("workspace", [False, True])
def test_mean_square_of_long_sums(dtype, shape, cross, workspace):
    hq, hkv, dim, nq, keys = shape
    cfg = csa.KVCfg(hq, hkv, dim, dtype, rope_dims=0)
    cache, (k, v) = _cache(cfg, keys, dim + hq)
    g = torch.Generator(device="cuda").manual_seed(hq)
    q = torch.randn(sum(nq), hq, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    out = _call(cfg, cache, q, nq, keys, cross, workspace, dim ** -0.5)
    t = m = 0
    for n, keys_b in zip(nq, keys):
        want = _kv.attend_sums(q[t:t + n], k[m:m + keys_b], v[m:m + keys_b], dim ** -0.5, not cross)
        each, rms = _kv.far(cfg, keys_b, out[t:t + n], *want)
        assert each < 1 and rms < 1, "%.3g and %.3g of what roundings allow" % (each, rms)
        t, m = t + n, m + keys_b


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("workspace", [False, True])
def test_every_page_answers(dtype, shape, cross, workspace):
    """Queries along one key each, so that all others weigh less than 2^-20 together: the first and the last key of every
    page, and keys between, are picked out of either kv head in turn."""
    hq, hkv, dim, nq, keys = shape
    cfg, group = csa.KVCfg(hq, hkv, dim, dtype, rope_dims=0), hq // hkv
    cache, (k, v) = _cache(cfg, keys, dim + hq)
    rng = np.random.default_rng(hq)
    first = np.concatenate([[0], np.cumsum(keys)])
    marks = []
    for n, m in zip(nq, keys):
        last = m if cross else m - n + 1  # every row sees these
        at = np.arange(0, last, 64)
        marks.append(np.unique(np.concatenate([at, np.minimum(at + 63, last - 1), rng.integers(0, last, len(at))])))
    scale = 1.0  # logits 4 |k|^2 against 4 k k': some sqrt(D) = 8 deviations of a product apart, of 4 sqrt(D) each
    calls = max(-(-len(x) // (n * group)) for x, n in zip(marks, nq))
    for c in range(calls):
        q = torch.empty(sum(nq), hq, dim, dtype=torch.bfloat16, device="cuda")
        want = torch.empty_like(q)
        t = 0
        for b, n in enumerate(nq):
            pick = marks[b][(c * n * group + np.arange(n * group)) % len(marks[b])].reshape(n, 1, group)
            pick = torch.from_numpy(np.broadcast_to(first[b] + pick, (n, hkv, group)).reshape(n, hq).copy()).cuda()
            head = torch.arange(hq, device="cuda") // group
            q[t:t + n], want[t:t + n] = k[pick, head] * 4, v[pick, head]
            t += n
        out = _call(cfg, cache, q, nq, keys, cross, workspace, scale)
        # values are exact in bf16: what is left is the weight's rounding (2^-8, in f16 2^-11; the sum of weights has it
        # unrounded), the output's (2^-8), both of the value, and the others' 2^-20 of values up to 6
        far = (out.double() - want.double()).abs() / (2.01 * 2.0 ** -8 * want.double().abs() + 2.0 ** -17)
        assert far.max().item() <= 1, "%.3g" % far.max().item()


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,group,nq", [(64, 8, 1), (128, 32, 1), (64, 4, 10), (128, 2, 200)])
def test_a_million_keys(dtype, dim, group, nq):
    cfg, keys, cross = csa.KVCfg(group, 1, dim, dtype, rope_dims=0), 1000003, nq > 1
    cache, (k, v) = _cache(cfg, [keys], dim + nq)
    g = torch.Generator(device="cuda").manual_seed(nq)
    q = torch.randn(nq, group, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    some = min(nq, 8)  # rows that are compared in full, the last ones
    out = _call(cfg, cache, q, [nq], [keys], cross, True, dim ** -0.5)
    want = _kv.attend_sums(q[nq - some:], k, v, dim ** -0.5, not cross)
    each, rms = _kv.far(cfg, keys, out[nq - some:], *want)
    assert each < 1 and rms < 1, "%.3g and %.3g of what roundings allow" % (each, rms)
    at = np.random.default_rng(dim).integers(0, keys - nq, nq * group)
    at[:3] = 0, keys - nq, keys // 2 // 64 * 64
    at = torch.from_numpy(at.reshape(nq, group)).cuda()
    picked = _call(cfg, cache, k[at, 0] * 4, [nq], [keys], cross, True, 1.0)
    value = v[at, 0].double()
    assert ((picked.double() - value).abs() <= 2.01 * 2.0 ** -8 * value.abs() + 2.0 ** -17).all()
