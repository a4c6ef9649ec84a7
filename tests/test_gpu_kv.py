"""Paged key / value operators on the GPU against their plain restatement in fp64."""
import math

import numpy as np
import pytest
import torch

import compressed_sparse_attention_07_gb300 as csa
from tests import _kv

pytestmark = pytest.mark.gpu

FP4, BF16 = csa.CACHE_FP4, csa.CACHE_BF16
HALF, INTER = csa.ROPE_HALF, csa.ROPE_INTERLEAVED


def _dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(dtype)


def _cu(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _cache(cfg, batch, capacity, seed=0):
    pages = batch * max(1, -(-capacity // 64))
    order = np.random.default_rng(seed).permutation(pages + 3)[:pages]
    return csa.KVCache(cfg, batch, capacity, page_order=order, spare_pages=3)


def _noise(cache):
    """Every bit pattern into the pages: E4M3 NaNs among the scales, NaN and infinities among bf16 values."""
    for t in (cache.k_data, cache.v_data, cache.k_scales, cache.v_scales):
        if t is not None:
            t.view(torch.uint8).random_(0, 256)
    for t in (cache.k_scales, cache.v_scales):
        if t is not None:
            t.view(-1)[::3] = 0x7F
    if cache.k_scales is None:
        for t in (cache.k_data, cache.v_data):
            t.view(-1)[::5] = float("nan")
            t.view(-1)[1::5] = float("inf")


# ----------------------------------------------------------------- append --

@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv,rope,style", [
    (64, 1, 1, 64, INTER), (64, 6, 3, 32, HALF), (128, 28, 4, 128, HALF), (128, 8, 8, 64, INTER), (128, 16, 1, 96, HALF),
    (64, 4, 2, 16, HALF), (128, 5, 5, 0, INTER)])
def test_append_matches(dtype, dim, hq, hkv, rope, style):
    _append_case(dtype, dim, hq, hkv, rope, style, [3, 0, 1, 70, 64], [0, 5, 63, 60, 128])


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv,rope,style", [
    (64, 3, 1, 64, INTER), (64, 200, 2, 32, HALF), (128, 112, 1, 128, HALF), (128, 7, 1, 64, INTER), (128, 0, 2, 0, INTER)])
def test_append_of_many_tokens(dtype, dim, hq, hkv, rope, style):
    # more rows than one piece of a token holds, and tokens without queries
    _append_case(dtype, dim, hq, hkv, rope, style, [901, 0, 1, 400, 64], [0, 5, 63, 60, 128])


def _append_case(dtype, dim, hq, hkv, rope, style, lengths, starts):
    rng = np.random.default_rng(dim + hq + rope)
    cfg = csa.KVCfg(hq or hkv, hkv, dim, dtype, rope_dims=rope, rope_style=style)
    cache = _cache(cfg, 5, max(a + b for a, b in zip(lengths, starts)))
    _noise(cache)
    before = [t.clone() for t in (cache.k_data, cache.v_data)]
    T = sum(lengths)
    rows = _kv.normal(rng, T + 4, hq + 2 * hkv + 1, dim)  # a projection's rows, wider than what is taken of them
    rows[0, -2, :16] = 0.0                                # a group of zeros (scale code 0) among the values
    wide = _dev(rows)
    q, k, v = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:hq + 2 * hkv]
    q_out = torch.full((T + 4, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out, v_out = (torch.full((T + 4, hkv, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    st = _status()
    table = csa.rope_table(1000, rope) if rope else None
    csa.kv_append(cfg, k, v, _cu(lengths), torch.tensor(starts, device="cuda"), cache, rope=table, q=q if hq else None,
                  q_out=q_out if hq else None, k_out=k_out, v_out=v_out, status=st)
    assert int(st.item()) == 0
    pos = np.concatenate([np.arange(n) + s for n, s in zip(lengths, starts)])
    host = table.cpu().numpy() if rope else None
    x = rows[:T].astype(np.float64)
    want_q = _kv.rotate(x[:, :hq], host, pos, rope, style == HALF)
    want_k = _kv.rotate(x[:, hq:hq + hkv], host, pos, rope, style == HALF)
    want_v = x[:, hq + hkv:hq + 2 * hkv]
    if hq:
        assert torch.equal(q_out[:T].cpu(), torch.from_numpy(want_q).to(torch.bfloat16))
    assert (q_out[T:] == 7).all() and (k_out[T:] == 7).all() and (v_out[T:] == 7).all()
    t0 = 0
    for b, (n, s) in enumerate(zip(lengths, starts)):
        for kind, want, plain in (("k", want_k, k_out), ("v", want_v, v_out)):
            w = want[t0:t0 + n]
            val, codes, sc = _kv.fp4_round(w) if dtype == FP4 else (_kv.bf16(w), None, None)
            got, gcodes, gsc = _kv.read(cache, cfg, b, kind, s + n)
            assert np.array_equal(got[s:], val)
            assert np.array_equal(plain[t0:t0 + n].double().cpu().numpy(), val)
            if dtype == FP4:
                assert np.array_equal(gcodes[s:], codes) and np.array_equal(gsc[s:], sc)
        t0 += n
    # nothing else changed: the written slots put back, the pages are as they were
    tab = cache.block_table.cpu().numpy()
    for t, old in zip((cache.k_data, cache.v_data), before):
        for b, (n, s) in enumerate(zip(lengths, starts)):
            for j in range(s, s + n):
                at = (tab[b, j // 64], slice(None), j % 64) if dtype == FP4 else (tab[b, j // 64], slice(None), slice(None), j % 64)
                t[at] = old[at]
        assert torch.equal(t.view(torch.uint8), old.view(torch.uint8))


def test_append_in_place_and_without_queries():
    rng = np.random.default_rng(3)
    cfg = csa.KVCfg(8, 2, 128, FP4, rope_dims=128, rope_style=HALF)
    table = csa.rope_table(64, 128)
    q, k, v = (_dev(_kv.normal(rng, 9, h, 128)) for h in (8, 2, 2))
    a, b = _cache(cfg, 1, 64), _cache(cfg, 1, 64)
    pos0 = torch.tensor([11], device="cuda")
    q_out = torch.empty_like(q)
    csa.kv_append(cfg, k, v, _cu([9]), pos0, a, rope=table, q=q, q_out=q_out)
    csa.kv_append(cfg, k, v, _cu([9]), pos0, b, rope=table)
    same = q.clone()
    csa.kv_append(cfg, k, v, _cu([9]), pos0, b, rope=table, q=same, q_out=same)
    assert torch.equal(same, q_out)
    assert torch.equal(a.k_data, b.k_data) and torch.equal(a.v_scales, b.v_scales)


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_append_of_what_is_not_finite(dtype):
    cfg = csa.KVCfg(2, 1, 64, dtype, rope_dims=0)
    cache = _cache(cfg, 1, 64)
    k = torch.full((2, 1, 64), 6.0, dtype=torch.bfloat16, device="cuda")  # scale 1, code 6
    v = k.clone()
    v[0, 0, 3], v[0, 0, 20], v[1, 0, 40] = float("inf"), float("nan"), float("-inf")
    st = _status()
    out = torch.empty_like(v)
    csa.kv_append(cfg, k, v, _cu([2]), torch.zeros(1, dtype=torch.int64, device="cuda"), cache, v_out=out, status=st)
    assert csa.status_string(int(st.item())) == csa.status_string(19)
    assert torch.isfinite(out.float()).all() and out[0, 0, 3] > 1000 and out[1, 0, 40] < -1000
    assert out[0, 0, 20] == 0 and out[0, 0, 21] == 6 and out[0, 0, 50] == 6
    assert np.isfinite(_kv.read(cache, cfg, 0, "v", 2)[0]).all()


def test_append_reports_places_out_of_bounds():
    cfg = csa.KVCfg(2, 1, 64, FP4, rope_dims=64)
    x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    for code, starts, lens, rows, page in ((17, [62, 0], [3, 1], 300, None), (17, [-1, 0], [3, 1], 300, None),
                                           (17, [9, 0], [3, 1], 10, None), (16, [0, 0], [3, 1], 300, 77),
                                           (16, [0, 0], [3, 1], 300, -1), (17, [0, 0], [3, 2], 300, None)):
        cache = csa.KVCache(cfg, 2, 64)
        if page is not None:
            cache.block_table[0, 0] = page
        st = _status()
        csa.kv_append(cfg, x, x, _cu(lens), torch.tensor(starts, device="cuda"), cache, rope=csa.rope_table(rows, 64),
                      status=st)
        assert int(st.item()) == code
        # the other sequence is written (unless its own rows reach past T)
        assert bool(cache.k_data[1].any()) == (lens[1] == 1)
        if page is not None or starts[0] == 0:
            assert bool(cache.k_data[0].any()) == (page is None)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("hq,dim", [(4, 64), (90, 128)])
def test_append_of_many_tokens_beside_a_bad_place(hq, dim, dtype):
    # rows ahead of the first sequence and behind the last, and one without a place, beside rows that are written
    rng = np.random.default_rng(hq)
    cfg = csa.KVCfg(hq, 1, dim, dtype, rope_dims=dim)
    lens, first, T = [1, 698, 3, 601], 5, 1320
    cu = torch.tensor(np.cumsum([first] + lens), dtype=torch.int32, device="cuda")
    q, k, v = (_dev(_kv.normal(rng, T, h, dim)) for h in (hq, 1, 1))
    got = []
    for start in (0, -1):
        cache, st = csa.KVCache(cfg, 4, 768), _status()
        out = torch.full_like(q, 7.0)
        csa.kv_append(cfg, k, v, cu, torch.tensor([3, start, 9, 60], device="cuda"), cache, rope=csa.rope_table(1024, dim),
                      q=q, q_out=out, status=st)
        assert int(st.item()) == (17 if start else 0)
        got.append((cache, out))
    (good, out), (some, part) = got
    lo, hi = first + 1, first + 1 + lens[1]
    assert (part[lo] == 7).all() and torch.equal(part[:lo], out[:lo]) and torch.equal(part[hi:], out[hi:])
    assert (out[:first] == 7).all() and (out[first + sum(lens):] == 7).all() and not (out[lo] == 7).all()
    # position -1 is the only one without a place: the rows behind it stand at 0, 1, ..
    alone, own = csa.KVCache(cfg, 1, 768), q[lo + 1:hi].clone()
    csa.kv_append(cfg, k[lo + 1:hi], v[lo + 1:hi], _cu([lens[1] - 1]), torch.zeros(1, dtype=torch.int64, device="cuda"), alone,
                  rope=csa.rope_table(1024, dim), q=own, q_out=own)
    assert torch.equal(part[lo + 1:hi], own)
    table = good.block_table.long()
    for kind in ("k_data", "v_data"):
        a, b = getattr(good, kind), getattr(some, kind)
        assert all(torch.equal(a[table[i]], b[table[i]]) for i in (0, 2, 3))
        assert torch.equal(b[table[1]], getattr(alone, kind)[alone.block_table[0].long()])


# -------------------------------------------------------------- attention --

def _attend_case(cfg, nq, kv, cross=False, seed=0, workspace=True, std=1.0, scale=None, pad=0, wide=0, slack=0,
                 noise=True, capture=False):
    rng = np.random.default_rng(seed)
    B, D, T = len(nq), cfg.head_dim, sum(nq)
    cache = _cache(cfg, B, max(max(kv), 1) + 70, seed)
    if noise:
        _noise(cache)
    ks, vs = [], []
    for b, n in enumerate(kv):
        for kind, into in (("k", ks), ("v", vs)):
            x = _kv.normal(rng, n, cfg.kv_heads, D)
            if n:
                _kv.fill(cache, cfg, b, kind, x)
            into.append(_kv.fp4_round(x)[0] if cfg.cache_dtype == FP4 else x)
    rows = _kv.normal(rng, T + pad, cfg.n_heads + wide, D, std=std)
    q = _dev(rows)[:, : cfg.n_heads]
    out = torch.full((T + pad, cfg.n_heads + wide, D), 7.0, dtype=torch.bfloat16, device="cuda")[:, : cfg.n_heads]
    lse = torch.full((T + pad, cfg.n_heads), 7.0, device="cuda")
    st = _status()
    mq, mk = max(nq) + slack, max(kv) + (70 if slack else 0)
    need = csa.kv_workspace_bytes(cfg, B, T + pad, mq, mk)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if workspace and need else None
    scale = 1 / math.sqrt(D) if scale is None else scale
    call = csa.kv_cross_attend if cross else csa.kv_attend
    cu, lens = _cu(nq), torch.tensor(kv, dtype=torch.int32, device="cuda")

    def go():
        call(cfg, q, cu, cache, lens, mq, mk, out, lse=lse, scale=scale, workspace=ws, status=st)

    if capture:
        run = csa.capture(go)
        out.fill_(7.0)
        lse.fill_(7.0)
        run()
        run()
    else:
        go()
    assert int(st.item()) == 0
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    t0 = 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(nq):
        want = _kv.attend(rows[t0:t0 + n, : cfg.n_heads], ks[b], vs[b], scale, not cross, cfg.window)
        tol, ltol = _kv.tolerances(cfg, kv[b], *want)
        got, gl = o[t0:t0 + n], l[t0:t0 + n]
        empty = ~np.isfinite(want[1])
        assert (gl[empty] == -np.inf).all() and (got[empty] == 0).all()
        far = np.abs(got - want[0]) / tol
        assert far.max(initial=0) <= 1, "sequence %d: %.3g of the tolerance" % (b, far.max())
        lfar = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, want[1])) / ltol
        assert lfar.max(initial=0) <= 1, "sequence %d: lse %.3g of the tolerance" % (b, lfar.max())
        t0 += n
    return out


HEADS = [(64, 1, 1), (128, 8, 1), (64, 7, 1), (128, 28, 4), (64, 16, 16), (128, 64, 2), (64, 24, 2)]


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", HEADS)
def test_single_tokens(dtype, dim, hq, hkv):
    _attend_case(csa.KVCfg(hq, hkv, dim, dtype), [1] * 9, [1, 2, 63, 64, 65, 0, 130, 257, 500], seed=dim + hq)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", HEADS)
@pytest.mark.parametrize("cross", [False, True])
def test_ragged_rows(dtype, dim, hq, hkv, cross):
    # more rows than keys (rows that see nothing), none, one, tiles that end inside a page
    _attend_case(csa.KVCfg(hq, hkv, dim, dtype), [5, 0, 1, 33, 20, 65, 2], [5, 40, 90, 33, 7, 200, 0], cross=cross,
                 seed=dim + hq, pad=3, slack=9)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", [(128, 8, 8), (64, 8, 2), (128, 12, 1)])
@pytest.mark.parametrize("window", [1, 17, 64, 100, 2 ** 31 - 1])
def test_windows(dtype, dim, hq, hkv, window):
    cfg = csa.KVCfg(hq, hkv, dim, dtype, window=window)
    _attend_case(cfg, [1, 3, 70, 150], [300, 65, 70, 400], seed=window % 1000)
    _attend_case(cfg, [1, 2], [300, 65], seed=window % 1000 + 1)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", [(128, 8, 2), (64, 14, 2)])
@pytest.mark.parametrize("nq", [1, 5, 40])
@pytest.mark.parametrize("workspace", [False, True])
def test_long_keys_divided_or_not(dtype, dim, hq, hkv, nq, workspace):
    _attend_case(csa.KVCfg(hq, hkv, dim, dtype), [nq, nq], [6007, 1500], seed=nq, workspace=workspace)


@pytest.mark.parametrize("dim,hq,hkv,window", [(128, 256, 2, 0), (64, 128, 1, 0), (128, 128, 1, 30), (128, 128, 1, 40)])
@pytest.mark.parametrize("cross", [False, True])
def test_pages_decoded_ahead_or_in_passing(dim, hq, hkv, window, cross):
    # the products' operands and their order are the same: every bit is
    rng = np.random.default_rng(dim + window)
    cfg = csa.KVCfg(hq, hkv, dim, FP4, window=0 if cross else window)
    nq, kv = [150, 0, 1, 40, 65], [333, 90, 77, 20, 0]
    B, T, mq, mk = len(nq), sum(nq), 150, 400
    cache = _cache(cfg, B, mk)
    _noise(cache)
    for b, n in enumerate(kv):
        for kind in "kv":
            if n:
                _kv.fill(cache, cfg, b, kind, _kv.normal(rng, n, hkv, dim))
    cache.block_table[0, 4] = 10 ** 6  # one page is not there
    q = _dev(_kv.normal(rng, T, hq, dim))
    cu, lens = _cu(nq), torch.tensor(kv, dtype=torch.int32, device="cuda")
    call, pages = csa.kv_cross_attend if cross else csa.kv_attend, 2 * B * 7 * hkv * 64 * dim * 2
    ahead = cross or window != 30  # 51 tokens a sequence; 30 x 128 rows that read a key are fewer than 4096
    assert csa.kv_workspace_bytes(cfg, B, T, mq, mk) >= (pages if ahead else 0)
    got = []
    for n in (0, pages):
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
        out, lse, st = torch.full_like(q, 7.0), torch.full((T, hq), 7.0, device="cuda"), _status()
        call(cfg, q, cu, cache, lens, mq, mk, out, lse=lse, workspace=ws, status=st)
        assert int(st.item()) == 16
        got.append((out, lse))
    assert not ahead or bool((ws != 255).any())
    assert torch.isfinite(got[0][0].float()).all()
    if ahead:
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_one_prompt_among_many_single_tokens(dtype):
    # tiles are counted by what the sequences have, over more than one warp's 128 sequences
    rng = np.random.default_rng(8)
    nq = [1] * 70 + [90] + [1, 0, 2] * 40 + [200] + [1] * 9
    kv = [int(n) for n in rng.integers(0, 150, len(nq))]
    kv[70], kv[191] = 90, 333
    _attend_case(csa.KVCfg(14, 2, 64, dtype), nq, kv, seed=8, pad=5)


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_last_wave_of_row_tiles_divided(dtype):
    # 208 and 224 row tiles: the last 56 and 72 with their keys in parts
    cfg = csa.KVCfg(256, 16, 64, dtype)
    _attend_case(cfg, [208], [2700], seed=5)
    _attend_case(cfg, [97, 111], [1500, 2700], seed=6, capture=True)


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_pages_of_all_last_lengths(dtype):
    # the last page of a tile alone, full, and ending at every kind of place, for one row, few and many
    kv = [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 256]
    for nq in (1, 9, 150):
        _attend_case(csa.KVCfg(2, 1, 64, dtype), [nq] * len(kv), kv, cross=True, seed=nq)
        _attend_case(csa.KVCfg(2, 1, 128, dtype), [nq] * len(kv), kv, seed=nq)


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_many_small_sequences_and_one_long(dtype):
    kv = [3] * 40 + [9000] + [700] * 5
    _attend_case(csa.KVCfg(8, 4, 64, dtype), [1] * 46, kv, seed=3)
    _attend_case(csa.KVCfg(4, 4, 128, dtype), [2] * 46, kv, cross=True, seed=4)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("cross", [False, True])
def test_prompts(dtype, cross):
    _attend_case(csa.KVCfg(8, 2, 128, dtype), [300, 129, 64], [700, 129, 100], cross=cross, seed=5)
    _attend_case(csa.KVCfg(6, 3, 64, dtype), [260, 17], [261, 300], cross=cross, seed=6)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("nq", [1, 3, 90])
def test_rows_apart_and_extreme_scales(dtype, nq):
    cfg = csa.KVCfg(8, 2, 64, dtype)
    _attend_case(cfg, [nq, nq], [300, 100], seed=1, wide=3)
    _attend_case(cfg, [nq, nq], [300, 100], seed=2, std=30.0)              # peaked: one key takes all
    _attend_case(cfg, [nq, nq], [300, 100], seed=3, scale=-0.3)
    _attend_case(cfg, [nq, nq], [300, 100], seed=4, scale=0.0)             # all keys alike
    _attend_case(cfg, [nq, nq], [300, 100], seed=5, std=2.0 ** 60, scale=2.0 ** -63)   # beyond f16's range
    _attend_case(cfg, [nq, nq], [300, 100], seed=6, std=2.0 ** -40, scale=2.0 ** 37)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("nq,kv", [(1, 3000), (5, 900), (80, 500)])
def test_same_results_each_time_and_in_a_graph(dtype, nq, kv):
    cfg = csa.KVCfg(16, 2, 128, dtype)
    first = _attend_case(cfg, [nq] * 3, [kv, kv // 2, kv - 7], seed=9)
    again = _attend_case(cfg, [nq] * 3, [kv, kv // 2, kv - 7], seed=9)
    graph = _attend_case(cfg, [nq] * 3, [kv, kv // 2, kv - 7], seed=9, capture=True)
    assert torch.equal(first, again) and torch.equal(first, graph)


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("nq", [1, 60])
def test_a_bad_query_stays_alone(dtype, nq):
    cfg = csa.KVCfg(8, 2, 64, dtype)
    cache = _cache(cfg, 1, 256)
    rng = np.random.default_rng(8)
    for kind in "kv":
        _kv.fill(cache, cfg, 0, kind, _kv.normal(rng, 200, 2, 64))
    q = _dev(_kv.normal(rng, nq, 8, 64))
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    good, got = torch.empty_like(q), torch.empty_like(q)
    csa.kv_attend(cfg, q, _cu([nq]), cache, lens, nq, 200, good)
    q[nq - 1, 3, 5] = float("nan")
    q[0, 6, 0] = float("inf")
    csa.kv_attend(cfg, q, _cu([nq]), cache, lens, nq, 200, got)
    keep = torch.ones(nq, 8, dtype=torch.bool, device="cuda")
    keep[nq - 1, 3] = keep[0, 6] = False
    assert torch.equal(good[keep], got[keep])


@pytest.mark.parametrize("nq", [1, 70])
def test_reports_lengths_and_pages_out_of_bounds(nq):
    cfg = csa.KVCfg(4, 2, 64, FP4)
    rng = np.random.default_rng(4)
    T = 2 * nq

    def run(kv, cu, table=None, max_q=nq, max_kv=256):
        cache = csa.KVCache(cfg, 2, 256)
        for b in (0, 1):
            for kind in "kv":
                _kv.fill(cache, cfg, b, kind, _kv.normal(rng, 200, 2, 64))
        if table is not None:
            cache.block_table[0, 1] = table
        q = torch.ones(T, 4, 64, dtype=torch.bfloat16, device="cuda")
        out, st = torch.full_like(q, 7.0), _status()
        csa.kv_attend(cfg, q, torch.tensor(cu, dtype=torch.int32, device="cuda"), cache,
                      torch.tensor(kv, dtype=torch.int32, device="cuda"), max_q, max_kv, out, status=st)
        return int(st.item()), out

    for kv, cu in (([257, 200], [0, nq, T]), ([-1, 200], [0, nq, T]), ([200, 200], [-1, nq, T])):
        code, out = run(kv, cu)
        assert code == 17 and (out[:nq] == 7).all() and not (out[nq:] == 7).any()
    code, out = run([200, 200], [0, nq, T + 1])
    assert code == 17 and (out[nq:] == 7).all()
    code, out = run([200, 200], [0, nq + 1, nq])
    assert code == 17 and (out == 7).all()
    for page in (-1, 9, 1 << 30):
        code, out = run([200, 200], [0, nq, T], table=page)
        assert code == 16 and torch.isfinite(out.float()).all() and not (out == 7).any()


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_a_pool_past_32_bits(dtype):
    """Pages whose byte offsets pass 2^32 are read and written where they are."""
    cfg = csa.KVCfg(16, 8, 128, dtype, rope_dims=0)
    page = 8 * 64 * (64 if dtype == FP4 else 256)
    n = (1 << 32) // page + 40
    shape = (n, 8, 64, 64) if dtype == FP4 else (n, 8, 16, 64, 8)
    kind = torch.uint8 if dtype == FP4 else torch.bfloat16
    k_data, v_data = (torch.empty(shape, dtype=kind, device="cuda") for _ in "kv")
    sc = [torch.empty((n, 8, 64, 8), dtype=torch.uint8, device="cuda") for _ in "kv"] if dtype == FP4 else [None, None]
    table = torch.tensor([[n - 1, 0, n - 7, n - 3]], dtype=torch.int32, device="cuda")
    cache = csa.KVCache.over(cfg, k_data, v_data, table, *sc)
    rng = np.random.default_rng(2)
    x = _kv.normal(rng, 200, 32, 128)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    csa.kv_append(cfg, _dev(x[:, :8]), _dev(x[:, 8:16]), _cu([200]), zero, cache)
    stored = [_kv.fp4_round(x[:, 8 * i:8 * i + 8])[0] if dtype == FP4 else x[:, 8 * i:8 * i + 8] for i in (0, 1)]
    for nq in (1, 40):
        q = x[:nq, 16:]
        out = torch.empty(nq, 16, 128, dtype=torch.bfloat16, device="cuda")
        lens = torch.tensor([200], dtype=torch.int32, device="cuda")
        csa.kv_attend(cfg, _dev(q), _cu([nq]), cache, lens, nq, 200, out)
        want = _kv.attend(q, *stored, 1 / math.sqrt(128), True)
        assert (np.abs(out.double().cpu().numpy() - want[0]) <= _kv.tolerances(cfg, 200, *want)[0]).all()


# --------------------------------------------------- used one after another --

@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("window", [0, 50])
def test_prompt_then_steps(dtype, window):
    """A prompt appended and attended, then a token at a time: each step's rows equal those of the whole sequence
    computed at once from what the cache holds."""
    rng = np.random.default_rng(11)
    cfg = csa.KVCfg(8, 2, 64, dtype, window=window, rope_dims=64)
    prompt, steps, B = [37, 100], 4, 2
    total = [n + steps for n in prompt]
    cache = _cache(cfg, B, 128)
    table = csa.rope_table(128, 64)
    q, k, v = ([_kv.normal(rng, n, h, 64) for n in total] for h in (8, 2, 2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = [[] for _ in range(B)]
    at = [0] * B
    for step in range(steps + 1):
        n = prompt if step == 0 else [1] * B
        cut = [slice(a, a + m) for a, m in zip(at, n)]
        qd, kd, vd = (_dev(np.concatenate([x[b][cut[b]] for b in range(B)])) for x in (q, k, v))
        pos0 = torch.tensor(at, dtype=torch.int64, device="cuda")
        csa.kv_append(cfg, kd, vd, _cu(n), pos0, cache, rope=table, q=qd, q_out=qd)
        at = [a + m for a, m in zip(at, n)]
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        out = torch.empty_like(qd)
        csa.kv_attend(cfg, qd, _cu(n), cache, lens, max(n), 128, out)
        o = out.double().cpu().numpy()
        got[0].append(o[: n[0]])
        got[1].append(o[n[0]:])
    host = table.cpu().numpy()
    for b in range(B):
        qr = _kv.bf16(_kv.rotate(q[b], host, np.arange(total[b]), 64, False))
        ks, vs = (_kv.read(cache, cfg, b, kind, total[b])[0] for kind in "kv")
        want = _kv.attend(qr, ks, vs, 1 / 8, True, window)
        tol = _kv.tolerances(cfg, total[b], *want)[0]
        assert (np.abs(np.concatenate(got[b]) - want[0]) <= tol).all()


def test_decoder_over_its_encoder_in_graphs_on_two_streams():
    """An encoder's states appended once (no rotation), then decoder steps over them captured in two graphs with
    workspaces of their own and replayed on two streams at once."""
    rng = np.random.default_rng(12)
    cfg = csa.KVCfg(12, 4, 64, FP4, rope_dims=0)
    enc, B = [1500, 700, 0], 3
    cache = _cache(cfg, B, 1500)
    x = [_kv.normal(rng, n, 8, 64) for n in enc]
    rows = _dev(np.concatenate(x))
    csa.kv_append(cfg, rows[:, :4], rows[:, 4:], _cu(enc), torch.zeros(B, dtype=torch.int64, device="cuda"), cache)
    lens = torch.tensor(enc, dtype=torch.int32, device="cuda")
    cu = _cu([1] * B)
    runs = []
    for i in range(2):
        q = _kv.normal(rng, B, 12, 64)
        qd = _dev(q)
        out = torch.empty_like(qd)
        ws = torch.empty(csa.kv_workspace_bytes(cfg, B, B, 1, 1500), dtype=torch.uint8, device="cuda")
        g = csa.capture(lambda: csa.kv_cross_attend(cfg, qd, cu, cache, lens, 1, 1500, out, workspace=ws))
        runs.append((q, out, g, torch.cuda.Stream(), qd, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, _, g, s, _, _ in runs:
            with torch.cuda.stream(s):
                g()
    torch.cuda.synchronize()
    for q, out, *_ in runs:
        for b in range(B):
            ks, vs = (_kv.read(cache, cfg, b, kind, enc[b])[0] for kind in "kv")
            want = _kv.attend(q[b:b + 1], ks, vs, 1 / 8, False)
            tol = _kv.tolerances(cfg, enc[b], *want)[0]
            assert (np.abs(out[b:b + 1].double().cpu().numpy() - want[0]) <= tol).all()


def test_sequences_that_share_pages():
    """Samples of one prompt: their block tables name the same pages."""
    rng = np.random.default_rng(13)
    cfg = csa.KVCfg(8, 8, 64, FP4, rope_dims=0)
    cache = _cache(cfg, 3, 200)
    x = _kv.normal(rng, 130, 16, 64)
    for kind, part in (("k", x[:, :8]), ("v", x[:, 8:])):
        _kv.fill(cache, cfg, 0, kind, part)
    cache.block_table[1].copy_(cache.block_table[0])
    cache.block_table[2].copy_(cache.block_table[0])
    q = _kv.normal(rng, 3, 8, 64)
    out = torch.empty(3, 8, 64, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([130, 64, 1], dtype=torch.int32, device="cuda")
    csa.kv_attend(cfg, _dev(q), _cu([1, 1, 1]), cache, lens, 1, 130, out)
    for b, n in enumerate((130, 64, 1)):
        want = _kv.attend(q[b:b + 1], _kv.fp4_round(x[:n, :8])[0], _kv.fp4_round(x[:n, 8:])[0], 1 / 8, True)
        assert (np.abs(out[b:b + 1].double().cpu().numpy() - want[0]) <= _kv.tolerances(cfg, n, *want)[0]).all()


# ------------------------------------------- beside the library's other calls --

def _pages_at_random(cache, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (cache.k_data, cache.v_data):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (cache.k_scales, cache.v_scales):
        t.copy_(torch.randint(32, 64, t.shape, generator=g, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("how", ["append few", "append many", "rows", "cluster", "parts", "tiles", "tiles divided",
                                 "decoded ahead"])
def test_outputs_handed_to_the_sparse_attention(how):
    """csa2_attend reads its queries before it waits for the kernel ahead of it: handed what one of these calls has just
    been told to write, it has to see that, not what stood there."""
    B, hkv, keys = {"append few": (40, 2, 0), "append many": (120, 2, 0), "rows": (20, 32, 300), "cluster": (1, 32, 4000),
                    "parts": (3, 32, 9000), "tiles": (4, 2, 700), "tiles divided": (2, 2, 5000),
                    "decoded ahead": (2, 2, 3000)}[how]
    Tq = {"append few": 10, "append many": 10, "tiles": 64, "decoded ahead": 64}.get(how, 1)
    cfg = csa.KVCfg(256, hkv, 128, FP4, rope_dims=128)
    x = torch.empty(B * Tq, 256, 128, dtype=torch.bfloat16, device="cuda")
    cache = _cache(cfg, B, max(keys, Tq))
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(B * Tq, h, 128, generator=g, device="cuda", dtype=torch.bfloat16) for h in (256, hkv, hkv))
    cu = _cu([Tq] * B)
    if keys == 0:
        pos0, table = torch.zeros(B, dtype=torch.int64, device="cuda"), csa.rope_table(64, 128)

        def call():
            csa.kv_append(cfg, k, v, cu, pos0, cache, rope=table, q=q, q_out=x)
    else:
        _pages_at_random(cache, 6)
        lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
        ws = torch.empty(csa.kv_workspace_bytes(cfg, B, B * Tq, Tq, keys), dtype=torch.uint8, device="cuda")

        def call():
            csa.kv_attend(cfg, q, cu, cache, lens, Tq, keys, x, workspace=ws)

    sparse = csa.Cfg(ratio=1, topk=512, window=128)
    main = csa.PagedCache(B, 64, 512, csa.CACHE_FP4)
    n_ent = torch.zeros(B, dtype=torch.int32, device="cuda")
    topk = torch.full((B, Tq, 512), -1, dtype=torch.int32, device="cuda")
    swa = torch.randn(B, 128, 512, generator=g, device="cuda", dtype=torch.bfloat16)
    swa_len = torch.full((B,), 128, dtype=torch.int32, device="cuda")
    swa_pos0 = torch.zeros(B, dtype=torch.int64, device="cuda")
    q_pos = torch.full((B, Tq), 127, dtype=torch.int64, device="cuda")
    got, want = (torch.empty(B, Tq, 64, 512, device="cuda") for _ in "gw")

    def attend(out):
        csa.attend(sparse, x.view(B, Tq, 64, 512), main, n_ent, topk, swa, swa_len, swa_pos0, q_pos, out, scale=0.2)

    def handed_on():
        x.zero_()
        call()
        attend(got)

    run = csa.capture(handed_on)  # the launches right behind one another
    for _ in range(10):
        run()
        torch.cuda.synchronize()
        attend(want)
        torch.cuda.synchronize()
        assert x.any() and torch.equal(got, want)


_THREADS = """
import threading
import torch
import compressed_sparse_attention_07_gb300 as csa
cfg = csa.KVCfg(64, 8, 128, rope_dims=0)
jobs = []
for i in range(8):
    g = torch.Generator(device="cuda").manual_seed(i)
    cache = csa.KVCache(cfg, 2, 2048)
    q, k, v = (torch.randn(3000, h, 128, generator=g, device="cuda", dtype=torch.bfloat16) for h in (64, 8, 8))
    cu = torch.tensor([0, 1600, 3000], dtype=torch.int32, device="cuda")
    few = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1600, 1400], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q), torch.zeros_like(q[:3])]
    jobs.append((cache, q, k, v, cu, few, lens, torch.zeros(2, dtype=torch.int64, device="cuda"), outs, torch.cuda.Stream()))
torch.cuda.synchronize()
start = threading.Barrier(len(jobs))

def run(job):
    cache, q, k, v, cu, few, lens, pos0, outs, s = job
    start.wait()
    csa.kv_append(cfg, k, v, cu, pos0, cache, stream=s)
    csa.kv_attend(cfg, q, cu, cache, lens, 1600, 2048, outs[0], stream=s)
    csa.kv_attend(cfg, q[:3], few, cache, lens, 2, 2048, outs[1], stream=s)

ts = [threading.Thread(target=run, args=(j,)) for j in jobs]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
for cache, q, k, v, cu, few, lens, pos0, outs, s in jobs:
    again = [torch.zeros_like(o) for o in outs]
    csa.kv_attend(cfg, q, cu, cache, lens, 1600, 2048, again[0])
    csa.kv_attend(cfg, q[:3], few, cache, lens, 2, 2048, again[1])
    assert outs[0].any() and outs[1].any() and all(torch.equal(a, o) for a, o in zip(again, outs))
print("same")
"""


def test_first_calls_from_several_threads_at_once():
    """A process whose first calls of every kernel come from eight threads at the same time."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def _hard_groups(rng, n):
    """n groups of 16 bf16 values where encoding decides closely: values half way between two codes of every scale and
    their bf16 neighbours, largest values half way between two scales and theirs, ordinary ones of every size, also far
    past the largest scale and below the smallest."""
    def near(x):  # x (exact in bf16) or a neighbour
        bits = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16)
        step = torch.from_numpy(rng.integers(-1, 2, bits.shape).astype(np.int16))
        return torch.where(bits > 0, bits + step, bits).view(torch.bfloat16).double().numpy()

    code = np.arange(127)
    e, m = code >> 3, code & 7
    scales = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    kind = np.arange(n) % 4
    s = scales[1 + rng.integers(0, 126, n)]
    x = near(s[:, None] * mids[rng.integers(0, 7, (n, 16))])                     # 0: half way between codes of scale s
    x[:, 0] = 6 * s
    up = rng.integers(0, 126, n)                                                 # 1: half way between scales
    border = near(3 * (scales[up] + scales[up + 1]))
    some = _kv.bf16(rng.uniform(0, 1, (n, 16)) * border[:, None])
    some[:, 5] = border
    x = np.where((kind == 1)[:, None], np.minimum(some, border[:, None]), x)
    wide = _kv.bf16(np.abs(rng.standard_normal((n, 16))) * 2.0 ** rng.uniform(-18, 18, n)[:, None])
    x = np.where((kind == 2)[:, None], wide, x)                                  # 2: of every size
    top = _kv.bf16(rng.uniform(0.01, 3, (n, 16)) * 2.0 ** rng.choice([-126.0, -60, 12, 60, 125], n)[:, None])
    x = np.where((kind == 3)[:, None], top, x)                                   # 3: far out of the scales' range
    return x * rng.choice([-1.0, 1.0], x.shape)


@pytest.mark.parametrize("tokens", [40, 1300])
@pytest.mark.parametrize("dim", [64, 128])
def test_append_encodes_as_the_oracle_at_every_border(tokens, dim):
    rng = np.random.default_rng(tokens + dim)
    cfg = csa.KVCfg(8, 8, dim, FP4, rope_dims=0)
    cache = _cache(cfg, 1, tokens)
    k, v = (_hard_groups(rng, tokens * 8 * dim // 16).reshape(tokens, 8, dim) for _ in "kv")
    out, st = torch.empty(2, tokens, 8, dim, dtype=torch.bfloat16, device="cuda"), _status()
    csa.kv_append(cfg, _dev(k), _dev(v), _cu([tokens]), torch.zeros(1, dtype=torch.int64, device="cuda"), cache,
                  k_out=out[0], v_out=out[1], status=st)
    assert int(st.item()) == 0
    for kind, x, plain in (("k", k, out[0]), ("v", v, out[1])):
        val, codes, sc = _kv.fp4_round(x)
        _, gcodes, gsc = _kv.read(cache, cfg, 0, kind, tokens)
        assert len(np.unique(sc)) == 127  # every scale
        assert np.array_equal(gsc, sc) and np.array_equal(gcodes, codes)
        assert np.array_equal(plain.double().cpu().numpy(), val)


@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_workspace_of_the_divided_tiles_alone(dtype):
    """208 row tiles, of which one wave is not divided: a workspace that holds the partial outputs of the others' rows
    gives what a larger one does, bit for bit, a smaller one other parts, and nothing is written behind any."""
    rng = np.random.default_rng(15)
    cfg, n, keys = csa.KVCfg(256, 16, 64, dtype), 208, 2700
    cache = _cache(cfg, 1, keys)
    stored = []
    for kind in "kv":
        x = _kv.normal(rng, keys, 16, 64)
        _kv.fill(cache, cfg, 0, kind, x)
        stored.append(torch.from_numpy(_kv.fp4_round(x)[0] if dtype == FP4 else x).cuda())
    q = _dev(_kv.normal(rng, n, 256, 64))
    want = _kv.attend_sums(q, *stored, 1 / 8, True)
    lens = torch.tensor([keys], dtype=torch.int32, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    need, row = csa.kv_workspace_bytes(cfg, 1, n, n, keys), 65 * 4
    parts, rest = need // (n * 256 * row), n % sms
    assert parts >= 2 and need == parts * n * 256 * row and 0 < rest < n
    results = []
    for size in (need, parts * rest * 256 * row, parts * rest * 256 * row - 256, 2 * 256 * row, 0):
        ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse, st = torch.empty_like(q), torch.empty(n, 256, device="cuda"), _status()
        csa.kv_attend(cfg, q, _cu([n]), cache, lens, n, keys, out, lse=lse, workspace=ws[:size] if size else None, status=st)
        assert int(st.item()) == 0 and (ws[size:] == 0xFF).all()
        results.append((out, lse))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert not torch.equal(results[0][1], results[4][1])  # divided or not, the sums go another way
    for out, lse in results:
        each, rms = _kv.far(cfg, keys, out, *want)
        assert each < 1 and rms < 1
        # two fp32 sums of the same weights
        assert (lse - results[0][1]).abs().max() <= 2 * (2 * keys + 64) * 2.0 ** -24


# ------------------------------------------------------- the largest of each --

@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 1024, 1024), (64, 1024, 1), (128, 1000, 8), (128, 1024, 64)])
def test_the_most_heads(dtype, dim, hq, hkv):
    _attend_case(csa.KVCfg(hq, hkv, dim, dtype), [1, 0, 2], [130, 5, 64], seed=hq + hkv)
    _append_case(dtype, dim, hq, hkv, 64, INTER, [3, 0, 1, 2, 4], [0, 5, 63, 60, 128])


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("longest", [1, 40])
def test_the_most_sequences(dtype, longest):
    """65535 sequences of 0 to 3 keys with a token each (and one of 40): appended, then attended."""
    B, dim = 65535, 64
    cfg = csa.KVCfg(1, 1, dim, dtype, rope_dims=0)
    g = torch.Generator(device="cuda").manual_seed(longest)
    cache = csa.KVCache(cfg, B, 64)
    cache.block_table.copy_(torch.randperm(B, generator=g, device="cuda", dtype=torch.int32)[:, None])
    n = torch.randint(0, 4, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[B - 5] = longest if longest > 1 else 1
    cu = torch.cat((n.new_zeros(1), n.cumsum(0).int()))
    T = int(cu[-1])
    k, v, q = (torch.randn(m, 1, dim, generator=g, device="cuda", dtype=torch.bfloat16) for m in (T, T, B - 1 + longest))
    sk, sv, st = torch.empty_like(k), torch.empty_like(v), _status()
    csa.kv_append(cfg, k, v, cu, torch.zeros(B, dtype=torch.int64, device="cuda"), cache, k_out=sk, v_out=sv, status=st)
    rows = torch.ones_like(n)
    rows[B - 5] = longest
    cq = torch.cat((n.new_zeros(1), rows.cumsum(0).int()))
    out, lse = torch.full_like(q, 7.0), torch.full((len(q), 1), 7.0, device="cuda")
    csa.kv_attend(cfg, q, cq, cache, n, longest, 64, out, lse=lse, status=st)
    assert int(st.item()) == 0
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), rows.long())
    pos = n[seq] - rows[seq] + (torch.arange(len(q), device="cuda") - cq[seq])
    at = torch.arange(longest if longest > 3 else 3, device="cuda")
    see = at <= pos[:, None]
    idx = (cu[seq][:, None] + at).clamp(max=T - 1).long()
    x = torch.einsum("td,tjd->tj", q[:, 0].double(), sk[idx, 0].double()) / 8
    p = torch.softmax(x.masked_fill(~see, -math.inf), 1).nan_to_num(0)
    want = torch.einsum("tj,tjd->td", p, sv[idx, 0].double())
    mag = torch.einsum("tj,tjd->td", p, sv[idx, 0].double().abs())
    empty = ~see.any(1)
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    # weights within 2^-8 of themselves, the output within 2^-8, logits (below 2^5) within a few steps of 2^-24
    assert ((out[:, 0].double() - want).abs() <= 2.0 ** -8 * (want.abs() + 1.01 * mag) + 2.0 ** -14 * mag + 1e-30).all()
    wl = torch.logsumexp(x.masked_fill(~see, -math.inf), 1)
    assert ((lse[:, 0] - wl)[~empty].abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("nq", [1, 20])
def test_rows_further_apart_than_32_bits_and_ahead_of_the_first_sequence(dtype, nq):
    """Rows of q, k, v, their outputs and out 2^30 + 8 elements apart, and rows ahead of cu[0] that are left alone."""
    cfg, rng = csa.KVCfg(4, 2, 64, dtype, rope_dims=0), np.random.default_rng(nq)
    T, step = nq + 3, (1 << 30) + 8 if nq == 1 else (1 << 28) + 8
    room = [torch.empty((T - 1) * step + 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, out = (r.as_strided((T, 4, 64), (step, 64, 1)) for r in room)
    k, v = (room[0].as_strided((T, 2, 64), (step, 64, 1), 256 + 128 * i) for i in (0, 1))
    hq, hk, hv = (_kv.normal(rng, T, h, 64) for h in (4, 2, 2))
    for t, x in ((q, hq), (k, hk), (v, hv)):
        t.copy_(_dev(x))
    out.fill_(7.0)
    cache = _cache(cfg, 1, 200)
    ks, vs = ([_kv.fp4_round(x)[0] if dtype == FP4 else x for x in (_kv.normal(rng, 100, 2, 64), y[2:T - 1])]
              for y in (hk, hv))
    for kind, x in (("k", ks), ("v", vs)):
        _kv.fill(cache, cfg, 0, kind, x[0])
    cu = torch.tensor([2, T - 1], dtype=torch.int32, device="cuda")
    st = _status()
    csa.kv_append(cfg, k, v, cu, torch.tensor([100], device="cuda"), cache, status=st)
    csa.kv_attend(cfg, q, cu, cache, torch.tensor([100 + nq], dtype=torch.int32, device="cuda"), nq, 200, out, status=st)
    assert int(st.item()) == 0 and (out[:2] == 7).all() and (out[T - 1:] == 7).all()
    want = _kv.attend(hq[2:T - 1], np.concatenate(ks), np.concatenate(vs), 1 / 8, True)
    assert (np.abs(out[2:T - 1].double().cpu().numpy() - want[0]) <= _kv.tolerances(cfg, 100 + nq, *want)[0]).all()


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("hq,hkv,nq", [(4, 2, 1), (4, 2, 5), (4, 2, 150), (128, 1, 45)])
@pytest.mark.parametrize("window", [1, 100, 128])
def test_pages_behind_the_window_may_be_gone(dtype, hq, hkv, nq, window):
    """Pages that no row's window reaches are not asked for: their places in the block table may name none."""
    rng = np.random.default_rng(nq + window)
    cfg = csa.KVCfg(hq, hkv, 64, dtype, window=window)
    kv, B = [1000, 64 + nq, 333], 3
    cache = _cache(cfg, B, 1000)
    for b, n in enumerate(kv):
        for kind in "kv":
            _kv.fill(cache, cfg, b, kind, _kv.normal(rng, n, hkv, 64))
    q, cu, lens = _dev(_kv.normal(rng, B * nq, hq, 64)), _cu([nq] * B), torch.tensor(kv, dtype=torch.int32, device="cuda")
    ws = torch.empty(csa.kv_workspace_bytes(cfg, B, B * nq, nq, 1000), dtype=torch.uint8, device="cuda")
    results = []
    for gone in (False, True):
        if gone:
            for b, n in enumerate(kv):
                cache.block_table[b, :max(0, n - nq + 1 - window) // 64] = -1
                cache.block_table[b, -(-n // 64):] = 10 ** 9
        out, st = torch.empty_like(q), _status()
        csa.kv_attend(cfg, q, cu, cache, lens, nq, 1000, out, workspace=ws, status=st)
        assert int(st.item()) == 0
        results.append(out)
    assert torch.equal(*results) and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 1024, 16), (128, 56, 8), (64, 640, 5)])
def test_row_tiles_that_see_nothing_at_all(dtype, dim, hq, hkv):
    """Prompts with fewer keys than rows, and without any: no product runs in the row tiles that see none, and their
    rows are 0 whatever the queries are."""
    cfg = csa.KVCfg(hq, hkv, dim, dtype)
    kv, nq = [20, 0, 3, 0], [100, 90, 47, 100]
    cache = _cache(cfg, 4, 64, seed=hq)
    rng = np.random.default_rng(dim)
    for b, n in enumerate(kv):
        for kind in "kv":
            if n:
                _kv.fill(cache, cfg, b, kind, _kv.normal(rng, n, hkv, dim))
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(sum(nq), hq, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    at = np.cumsum([0] + nq)
    for call in (csa.kv_attend, csa.kv_cross_attend):
        for _ in range(5):
            out, lse, st = torch.full_like(q, 7.0), torch.full((sum(nq), hq), 7.0, device="cuda"), _status()
            call(cfg, q, _cu(nq), cache, lens, 100, 20, out, lse=lse, status=st)
            assert int(st.item()) == 0
            for b, (n, keys) in enumerate(zip(nq, kv)):
                none = n if keys == 0 else n - keys if call is csa.kv_attend else 0
                assert (lse[at[b]:at[b] + none] == -math.inf).all() and (out[at[b]:at[b] + none] == 0).all()
                assert torch.isfinite(lse[at[b] + none:at[b + 1]]).all() and torch.isfinite(out[at[b]:at[b + 1]].float()).all()
