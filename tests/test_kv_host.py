"""The paged key / value operators without a GPU: page sizes, refusals (each call below fails validation, so nothing is
launched) and the plain restatement that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import compressed_sparse_attention_07_gb300 as csa
from tests import _kv

FAKE = 0x10000  # never dereferenced


def _cache(**kw):
    d = dict(k_data=FAKE, k_scales=FAKE, v_data=FAKE, v_scales=FAKE, block_table=FAKE, max_pages=4, num_pages=8)
    d.update(kw)
    return csa._KVCacheDesc(**d)


def _append(cfg=None, cache=None, **kw):
    cfg = csa.KVCfg() if cfg is None else cfg
    a = dict(B=1, T=4, q=FAKE, qs=64 * 128, k=FAKE, ks=1024, v=FAKE, vs=1024, cu=FAKE, pos0=FAKE, rope=FAKE, rows=64,
             q_out=FAKE, os=64 * 128, k_out=None, v_out=None, status=None)
    a.update(kw)
    c = _cache() if cache is None else cache
    return csa.load().csa2_kv_append(
        C.byref(cfg), a["B"], a["T"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["pos0"], a["rope"],
        a["rows"], C.byref(c), a["q_out"], a["os"], a["k_out"], a["v_out"], a["status"], None)


def _attend(cfg=None, cache=None, cross=False, **kw):
    cfg = csa.KVCfg() if cfg is None else cfg
    a = dict(B=1, T=4, q=FAKE, qs=64 * 128, cu=FAKE, kv_len=FAKE, max_q=4, max_kv=256, scale=1.0, out=FAKE, os=64 * 128,
             lse=None, ws=None, wn=0, status=None)
    a.update(kw)
    c = _cache() if cache is None else cache
    f = csa.load().csa2_kv_cross_attend if cross else csa.load().csa2_kv_attend
    return f(C.byref(cfg), a["B"], a["T"], a["q"], a["qs"], a["cu"], C.byref(c), a["kv_len"], a["max_q"], a["max_kv"],
             a["scale"], a["out"], a["os"], a["lse"], a["ws"], a["wn"], a["status"], None)


def _cfg(**kw):
    c = csa.KVCfg()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("bad,code", [
    (dict(n_heads=63), 1), (dict(n_heads=0), 1), (dict(kv_heads=0), 1), (dict(n_heads=2048), 2), (dict(head_dim=96), 2),
    (dict(head_dim=256), 2), (dict(cache_dtype=csa.CACHE_FP4_S32), 1), (dict(window=-1), 1), (dict(rope_dims=8), 1),
    (dict(rope_dims=144), 1), (dict(rope_style=2), 1), (dict(reserved=1), 1)])
def test_configurations_refused(bad, code):
    c = _cfg(**bad)
    assert _append(c) == code
    assert _attend(c) == code
    assert _attend(c, cross=True) == code
    lib = csa.load()
    assert lib.csa2_kv_page_bytes(C.byref(c), 0) == 0
    assert csa.kv_workspace_bytes(c, 1, 1, 1, 64) == 0


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(rows=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(ks=1016), dict(vs=1020),
    dict(vs=1028), dict(cu=None), dict(pos0=None), dict(pos0=FAKE + 4), dict(q=None), dict(q_out=None),
    dict(q=FAKE + 2), dict(qs=64 * 128 - 8), dict(os=64 * 128 - 8), dict(rope=None), dict(rope=FAKE + 8),
    dict(k_out=FAKE + 8), dict(v_out=FAKE + 2), dict(status=FAKE + 1)])
def test_append_arguments_refused(bad):
    assert _append(**bad) == 1


@pytest.mark.parametrize("bad", [
    dict(k_data=None), dict(v_data=None), dict(k_scales=None), dict(v_scales=None), dict(block_table=None),
    dict(max_pages=0), dict(num_pages=0), dict(k_data=FAKE + 8), dict(v_scales=FAKE + 4), dict(block_table=FAKE + 2),
    dict(max_pages=1 << 26)])
def test_caches_refused(bad):
    c = _cache(**bad)
    assert _append(cache=c) == 1
    assert _attend(cache=c) == 1


def test_rope_goes_with_the_table():
    assert _append(_cfg(rope_dims=0)) == 1  # a table, and nothing to rotate


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(cu=None), 1), (dict(kv_len=None), 1), (dict(q=FAKE + 4), 1), (dict(out=FAKE + 8), 1), (dict(qs=8), 1),
    (dict(os=64 * 128 + 4), 1), (dict(lse=FAKE + 2), 1), (dict(ws=FAKE + 16, wn=1 << 20), 1), (dict(ws=None, wn=64), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(max_kv=257), 4), (dict(B=65536), 2)])
def test_attend_arguments_refused(bad, code):
    assert _attend(**bad) == code
    assert _attend(cross=True, **bad) == code


def test_cross_attention_has_no_window():
    assert _attend(_cfg(window=4), cross=True) == 1


def test_empty_calls_do_nothing():
    assert _append(B=0, k=None) == 0
    assert _append(T=0, k=None) == 0
    for cross in (False, True):
        assert _attend(B=0, q=None, cross=cross) == 0
        assert _attend(T=0, q=None, cross=cross) == 0
        assert _attend(max_q=0, q=None, cross=cross) == 0


def test_page_bytes():
    lib = csa.load()
    for dim in (64, 128):
        c = _cfg(kv_heads=8, head_dim=dim)
        assert lib.csa2_kv_page_bytes(C.byref(c), 0) == 8 * 64 * dim // 2
        assert lib.csa2_kv_page_bytes(C.byref(c), 1) == 8 * 64 * dim // 16
        c.cache_dtype = csa.CACHE_BF16
        assert lib.csa2_kv_page_bytes(C.byref(c), 0) == 8 * 64 * dim * 2
        assert lib.csa2_kv_page_bytes(C.byref(c), 1) == 0
        assert lib.csa2_kv_page_bytes(C.byref(c), 2) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    cfg = csa.KVCfg(n_heads=4, kv_heads=2, head_dim=64, rope_dims=0)
    pages = torch.zeros(3, 2, 64, 32, dtype=torch.uint8)
    scales = torch.zeros(3, 2, 64, 4, dtype=torch.uint8)
    table = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):  # on the host
        csa.KVCache.over(cfg, pages, pages, table, scales, scales)
    with pytest.raises(ValueError):  # FP4 without scales
        csa.KVCache.over(cfg, pages, pages, table)
    with pytest.raises(ValueError):  # another head_dim
        csa.KVCache.over(csa.KVCfg(n_heads=4, kv_heads=2, head_dim=128), pages, pages, table, scales, scales)
    with pytest.raises(ValueError):
        csa.KVCache.over(csa.KVCfg(head_dim=80), pages, pages, table, scales, scales)


def test_rope_table_matches_the_plain_one():
    got = csa.rope_table(300, 64, 1e4, device="cpu").numpy()
    # cos and sin of the same fp64 angles, each rounded once to fp32 (half a step is 2^-25 below 1), the angles
    # themselves off by a few steps of 2^-53 of up to 300
    assert np.abs(got - _kv.rope_rows(300, 64)).max() <= 2.0 ** -24


def test_plain_attention_is_a_weighted_mean():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((5, 2, 64)), rng.standard_normal((5, 2, 64))
    out, lse = _kv.attend(q, k, v, 0.1, causal=True)[:2]
    for i in range(3):
        for h in range(4):
            n = 5 - 3 + i + 1
            w = np.exp(0.1 * (k[:n, h // 2] @ q[i, h]))
            assert np.allclose(out[i, h], (w[:, None] * v[:n, h // 2]).sum(0) / w.sum())
            assert np.isclose(lse[i, h], np.log(w.sum()))
    out, lse = _kv.attend(q, k[:0], v[:0], 0.1, causal=False)[:2]
    assert (out == 0).all() and (lse == -np.inf).all()
    one, _ = _kv.attend(q, k, v, 0.1, causal=True, window=1)[:2]
    assert np.allclose(one[1, 3], v[3, 1])


def test_plain_rotation_keeps_lengths_and_both_styles_agree():
    rng = np.random.default_rng(2)
    x = _kv.normal(rng, 5, 2, 128)
    t, pos = _kv.rope_rows(40, 96), np.array([0, 3, 7, 20, 39])
    y = _kv.rotate(x, t, pos, 96, False).astype(np.float64)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
    assert (y[..., 96:] == x[..., 96:]).all() and (y[0] == x[0]).all()
    halves = np.concatenate([x[..., 0:96:2], x[..., 1:96:2], x[..., 96:]], -1)
    z = _kv.rotate(halves, t, pos, 96, True)
    assert (z[..., :48] == y[..., 0:96:2].astype(np.float32)).all() and (z[..., 48:96] == y[..., 1:96:2].astype(np.float32)).all()


def test_more_row_tiles_than_a_grid_holds_are_refused():
    c = _cfg(n_heads=1024, kv_heads=1024)
    many = dict(B=65535, T=2 ** 31 - 1, max_q=10 ** 6, qs=1024 * 128, os=1024 * 128)
    assert _attend(c, **many) == 2
    assert _attend(c, cross=True, **many) == 2


@pytest.mark.parametrize("dtype,tokens,batch,keys,ahead", [
    (csa.CACHE_FP4, 512, 1, 16384, True), (csa.CACHE_FP4, 511, 1, 16384, False), (csa.CACHE_BF16, 512, 1, 16384, False),
    (csa.CACHE_FP4, 512, 1, 16385, True), (csa.CACHE_FP4, 2048, 33, 16384, False)])
def test_workspace_holds_pages_decoded_ahead(dtype, tokens, batch, keys, ahead):
    # 64 over 8 heads of 128: 4096 rows read a key from 512 tokens on; 2 GB hold 32 sequences of 16384 keys
    c = csa.KVCfg(64, 8, 128, dtype)
    pages = batch * -(-keys // 64) * 8 * 2 * 64 * 128 * 2
    need = csa.kv_workspace_bytes(c, batch, tokens * batch, tokens, keys)
    parts = tokens * batch * 64 * 129 * 4  # the rest is whole parts of every row
    assert (need - (pages if ahead else 0)) % parts == 0 and (not ahead or need >= pages)
    # the same rows, mostly one sequence's: the mean decides
    if ahead:
        assert csa.kv_workspace_bytes(c, 100, tokens + 99, tokens, keys) % ((tokens + 99) * 64 * 129 * 4) == 0


def _rounded_attention(cfg, q, k, v, scale):
    """Attention with the roundings that the kernels make and no others: weights to f16 or bf16, the output to bf16."""
    h, hq = k.shape[1], q.shape[1]
    out = torch.empty(q.shape, dtype=torch.bfloat16)
    for a in range(hq):
        x = q[:, a] @ k[:, a * h // hq].T * scale
        p = torch.exp(x - x.amax(1, keepdim=True))
        r = p.to(torch.float16 if cfg.cache_dtype == csa.CACHE_FP4 else torch.bfloat16).double()
        out[:, a] = (r @ v[:, a * h // hq] / p.sum(1, keepdim=True)).to(torch.bfloat16)
    return out


@pytest.mark.parametrize("dtype", [csa.CACHE_FP4, csa.CACHE_BF16])
@pytest.mark.parametrize("dim,keys", [(64, 6007), (128, 9000)])
def test_long_comparison_sees_a_lost_page(dtype, dim, keys):
    """The comparison for long sequences lets roundings pass, and sees 16 values lost among 6000 and 9000 keys, a page
    taken from another place and a part of the keys counted twice."""
    rng = np.random.default_rng(dim)
    cfg = csa.KVCfg(4, 2, dim, dtype)
    q = torch.from_numpy(_kv.normal(rng, 3, 4, dim))
    k, v = (torch.from_numpy(_kv.fp4_round(x)[0] if dtype == csa.CACHE_FP4 else x)
            for x in (_kv.normal(rng, keys, 2, dim) for _ in "kv"))
    scale = dim ** -0.5
    want = _kv.attend_sums(q, k, v, scale, False)
    plain = _kv.attend(q.numpy(), k.numpy(), v.numpy(), scale, False)[0]
    assert np.allclose(want[0].numpy(), plain, rtol=1e-9, atol=1e-12)
    each, rms = _kv.far(cfg, keys, _rounded_attention(cfg, q, k, v, scale), *want)
    assert each < 1 and rms < 1
    at = keys // 2 // 64 * 64
    for lost in (slice(at, at + 64), slice(at, at + 16), slice(keys - 16, keys)):
        w = v.clone()
        w[lost] = 0
        assert _kv.far(cfg, keys, _rounded_attention(cfg, q, k, w, scale), *want)[1] > 1
    w = v.clone()
    w[at:at + 64] = v[64:128]
    assert _kv.far(cfg, keys, _rounded_attention(cfg, q, k, w, scale), *want)[1] > 1
    twice = _rounded_attention(cfg, q, torch.cat((k, k[:256])), torch.cat((v, v[:256])), scale)
    assert _kv.far(cfg, keys, twice, *want)[1] > 1


@pytest.mark.parametrize("tokens,keys", [(2048, 16384), (2048, 18432), (4000, 131072), (8192, 32768), (1999, 100000)])
@pytest.mark.parametrize("dtype", [csa.CACHE_FP4, csa.CACHE_BF16])
def test_workspace_holds_the_divided_tiles_alone(tokens, keys, dtype):
    # 64 over 8 heads of 128, 256 rows a tile: fewer row tiles than the GPU has SMs are divided, in 64 parts at most;
    # partial outputs of every row would be 33 KB a token and part
    c = csa.KVCfg(64, 8, 128, dtype)
    pages = -(-keys // 64) * 8 * 2 * 64 * 128 * 2 if dtype == csa.CACHE_FP4 else 0
    need = csa.kv_workspace_bytes(c, 1, tokens, tokens, keys) - (pages if pages <= 2 << 30 else 0)
    assert 0 <= need <= max(64 << 20, 64 * 160 * 256 * 129 * 4)
    every = tokens * 64 * 129 * 4
    assert need <= 64 << 20 or need < every


@pytest.mark.parametrize("batch,tokens,max_q,keys", [(1, 2048, 2048, 18432), (3, 900, 700, 5000), (48, 48, 1, 16384),
                                                     (8, 40, 5, 32768), (2, 300, 290, 9000)])
def test_workspace_grows_with_no_size_left_out(batch, tokens, max_q, keys):
    """Multiples of a row's partial outputs, whichever way they stand."""
    c = csa.KVCfg(64, 8, 128, csa.CACHE_BF16)
    assert csa.kv_workspace_bytes(c, batch, tokens, max_q, keys) % (129 * 4) == 0
