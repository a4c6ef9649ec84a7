"""The operators of a generation step on the GPU against their plain restatement in 64 bits: projections with 4-bit
weights, appends with positions of several axes, beam selection, reordering of cached beams, and a run of all of them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import compressed_sparse_attention_07_gb300 as csa
import oracle
from tests import _kv, _step

pytestmark = pytest.mark.gpu

FP4, BF16 = csa.CACHE_FP4, csa.CACHE_BF16
HALF, INTER = csa.ROPE_HALF, csa.ROPE_INTERLEAVED


def _dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(dtype)


def _cu(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- projections --

def _packed(rng, n, k, alpha=1.0, lo=0x20, hi=0x50):
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, (n, k // 16), dtype=np.uint8)
    return csa.Fp4Weights.pack(_dev(codes, torch.uint8), _dev(scales, torch.uint8), alpha), _step.weights(codes, scales)


# rows: one, few, a full one and one more than a kernel or a tile has; sizes that end inside blocks, tiles and steps
LINEAR = [(1, 128, 16), (1, 16, 1), (2, 48, 17), (3, 1280, 130), (5, 4096, 200), (7, 144, 5000), (8, 272, 129), (9, 1280, 64),
          (12, 128, 2450), (16, 4096, 33), (16, 16, 257), (17, 128, 128), (17, 16, 1), (31, 400, 300), (32, 4096, 17),
          (33, 1040, 640), (64, 128, 129), (65, 272, 500), (100, 4096, 128), (128, 144, 1100), (129, 64, 96), (200, 1296, 257),
          (256, 128, 128), (257, 144, 130), (300, 2064, 700), (513, 32, 20000), (1, 70000, 20), (8, 9000 // 16 * 16, 40),
          (16, 20000, 36), (20, 33008, 130),
          # several tiles a CTA, for each number of rows that a tile takes
          (11, 70000, 300), (20, 128, 41000), (24, 400, 39001), (50, 272, 58000), (64, 528, 40000), (100, 144, 45000),
          (128, 656, 39000), (150, 272, 40001), (1500, 400, 4000)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,k,n", LINEAR)
def test_linear(T, k, n, f32):
    rng = np.random.default_rng(T + k + n)
    alpha = 0.37 / np.sqrt(k)
    w, plain = _packed(rng, n, k, alpha)
    bias = _kv.normal(rng, n) if (T + n) % 2 else None
    # slices of wider rows: what stands beside and behind them is not read, or written
    wide = torch.full((T + 2, k + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:T, 8:8 + k] = _dev(_kv.normal(rng, T, k))
    x = wide[:T, 8:8 + k]
    room = torch.full((T + 1, n + 3), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    st = _status()
    csa.fp4_linear(x, w, room[:T, :n], bias=None if bias is None else _dev(bias), status=st)
    assert int(st.item()) == 0
    y, tol = _step.linear(x.double().cpu().numpy(), plain, np.float32(alpha).astype(np.float64), bias)
    got = room[:T, :n].double().cpu().numpy()
    if not f32:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y)
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) / tol).max())
    assert (room[T:] == 7).all() and (room[:, n:] == 7).all()


@pytest.mark.parametrize("k", [400, 100000])
def test_a_single_row_has_no_stride(k):
    rng = np.random.default_rng(k)
    w, plain = _packed(rng, 40, k)
    x = _dev(_kv.normal(rng, 1, k))
    out = [torch.empty(1, 40, device="cuda") for _ in range(2)]
    csa.fp4_linear(x, w, out[0])
    assert csa.load().csa2_fp4_linear(w._ref, 1, x.data_ptr(), 1 << 60, None, out[1].data_ptr(), 1, 1 << 60, None,
                                      torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,k,n", [(20, 784, 20470), (50, 1552, 20480), (100, 2320, 20400), (1270, 2320, 4000)])
def test_linear_where_some_tiles_are_left_for_a_last_wave(T, k, n, f32):
    """160 tiles: each CTA has one, and clusters divide what is left."""
    test_linear(T, k, n, f32)


@pytest.mark.parametrize("T,k,n", [(1, 4096, 300), (8, 1280, 4096), (8, 4096, 39000), (11, 2048, 700), (16, 4096, 39000),
                                   (24, 1280, 3000), (40, 4096, 2560), (100, 4096, 640), (256, 1280, 1024), (700, 512, 2000)])
def test_linear_of_whole_numbers_is_exact(T, k, n):
    """Whole multiples of 1/2 whose sums fp32 holds: every weight and every row once, in its place."""
    rng = np.random.default_rng(k + n)
    w, plain = _packed(rng, n, k, 1.0, 0x38, 0x39)  # scales of 1
    x = rng.integers(-3, 4, (T, k)).astype(np.float64)
    out = torch.empty(T, n, device="cuda")
    csa.fp4_linear(_dev(x), w, out)
    want = torch.from_numpy(x).cuda() @ torch.from_numpy(plain).cuda().T
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("few", [True, False])
def test_every_code_and_scale(few):
    """Rows of x that pick out one channel: the weights themselves, each code with each scale."""
    k, n = 16 * 254, 16
    codes = (np.arange(k) + np.arange(n)[:, None]) % 16
    scales = np.tile(np.concatenate([np.arange(127), 128 + np.arange(127)]), (n, 1)).astype(np.uint8)
    packed = csa.Fp4Weights.pack(_dev(codes[:, 0::2] | codes[:, 1::2] << 4, torch.uint8), _dev(scales, torch.uint8))
    want = np.repeat(_step.e4m3(scales), 16, 1) * _step.E2M1[codes]
    eye = torch.eye(k, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(k, n, device="cuda")
    step = 16 if few else 1000
    for t in range(0, k, step):
        csa.fp4_linear(eye[t:t + step], packed, out[t:t + step])
    assert np.array_equal(out.double().cpu().numpy(), want.T)


def test_weights_encoded_as_the_oracle():
    rng = np.random.default_rng(5)
    n, k = 150, 272
    w = _kv.normal(rng, n, k, std=0.02)
    w[3, :16], w[4, 32:48] = 0.0, 1e-9
    w[5, 16:32] = np.resize([6, 5, -5, 3.5, 2.5, -1.75, 1.25, 0.75, 0.25, -0.25, 0.24, 4.9, -6, 0, 1, 2], 16) * 2.0 ** -9
    w[6, 0], w[7, 5] = 3e38, -3e38
    w = _kv.bf16(w)
    gain = 2.0 ** 9
    wide = torch.zeros(n, k + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :k] = _dev(w)
    st = _status()
    got = csa.Fp4Weights.encode(wide[:, :k], gain, status=st)
    assert int(st.item()) == 19 and got.alpha == 2.0 ** -9  # 3e38 x 512 is past fp32
    scaled = np.clip((w * gain).astype(np.float64), -3.4028234663852886e38, 3.4028234663852886e38)
    codes, scales = oracle.fp4_encode(scaled)
    same = csa.Fp4Weights.pack(_dev(codes, torch.uint8), _dev(scales, torch.uint8))
    assert torch.equal(got.data, same.data)
    # without a gain: a power of two that keeps the largest within the codec's range
    w = _kv.normal(rng, 16, 64, std=0.03)
    a = csa.Fp4Weights.encode(_dev(w))
    most = np.abs(w).max() / a.alpha
    assert 448 * 3 < most <= 448 * 6 and np.log2(a.alpha) % 1 == 0


def test_weights_near_nothing_are_encoded():
    """The largest below 2^-115: no gain that fp32 has would bring it to the codec's largest."""
    w = torch.full((16, 16), 2.0 ** -130, dtype=torch.bfloat16, device="cuda")
    got = csa.Fp4Weights.encode(w)
    assert got.alpha == 2.0 ** -126
    # 2^-130 x 2^126 = 1/16: scale e4m3(1/96) = 5/512 (steps of 2^-9 there), 6.4 of it: code 6
    out = torch.empty(1, 16, device="cuda")
    csa.fp4_linear(torch.full((1, 16), 2.0 ** 100, dtype=torch.bfloat16, device="cuda"), got, out)
    assert torch.equal(out, torch.full_like(out, 16 * 6 * 5 / 512 * 2.0 ** -26))


def test_packing_reports_scales_that_are_no_number():
    codes, scales = np.full((2, 32), 0x22, np.uint8), np.full((2, 4), 0x38, np.uint8)
    scales[1, 2], scales[0, 3] = 0x7F, 0xFF
    st = _status()
    w = csa.Fp4Weights.pack(_dev(codes, torch.uint8), _dev(scales, torch.uint8), status=st)
    assert int(st.item()) == 19
    out = torch.empty(1, 2, device="cuda")
    csa.fp4_linear(torch.ones(1, 64, dtype=torch.bfloat16, device="cuda"), w, out)
    assert out.tolist() == [[48.0, 48.0]]


@pytest.mark.parametrize("T", [1, 5, 16, 20, 70, 300])
def test_a_row_that_is_not_finite_stays_alone(T):
    rng = np.random.default_rng(T)
    w, plain = _packed(rng, 300, 400)
    x = _kv.normal(rng, T, 400)
    good, bad = _dev(x), _dev(x)
    rows = sorted({0, T // 2})
    bad[rows[0], 17], bad[rows[-1], 399] = float("inf"), float("nan")
    a, b = torch.empty(T, 300, device="cuda"), torch.empty(T, 300, device="cuda")
    csa.fp4_linear(good, w, a)
    csa.fp4_linear(bad, w, b)
    keep = [t for t in range(T) if t not in rows]
    assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(b[rows[-1]]).any()
    assert not torch.isfinite(b[rows[0]][torch.from_numpy(plain[:, 17] != 0).cuda()]).any()


@pytest.mark.parametrize("T", [2, 16, 24])
@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -100, 1.0, 2.0 ** 90, 2.0 ** 126])
def test_rows_of_any_size(T, size):
    """Rows far apart in size, and channels far below their row's largest."""
    rng = np.random.default_rng(7)
    w, plain = _packed(rng, 40, 256, 2.0 ** -20)
    x = _kv.normal(rng, T, 256)
    x[:, 0] = 1.5
    x[:, 1::2] *= 2.0 ** -20
    x = _kv.bf16(np.clip(x, -1.9, 1.9) * size * 2.0 ** -np.arange(T)[:, None])
    out = torch.empty(T, 40, device="cuda")
    csa.fp4_linear(_dev(x), w, out)
    y, tol = _step.linear(x, plain, 2.0 ** -20)
    tol = tol + 2.0 ** -149 * 256 * 500  # products below fp32's normal range lose bits
    got = out.double().cpu().numpy()
    # sums are fp32, before alpha: some order of adding passes its largest, 2^128, only where the magnitudes add up to it
    past = np.abs(x) @ np.abs(plain).T >= 2.0 ** 127.99
    assert ((np.abs(got - y) <= tol) | (past & ~np.isfinite(got))).all()


@pytest.mark.parametrize("T,k,n", [(1, 1280, 4096), (8, 4096, 10240), (16, 4096, 5000), (40, 4096, 2048), (300, 1024, 3000)])
def test_linear_is_the_same_each_time_in_graphs_and_on_two_streams(T, k, n):
    rng = np.random.default_rng(n)
    w, _ = _packed(rng, n, k)
    x = [_dev(_kv.normal(rng, T, k)) for _ in range(2)]
    first = [torch.empty(T, n, device="cuda") for _ in x]
    for a, o in zip(x, first):
        csa.fp4_linear(a, w, o)
    again = [torch.empty(T, n, device="cuda") for _ in x]
    graphs = [csa.capture(lambda a=a, o=o: csa.fp4_linear(a, w, o)) for a, o in zip(x, again)]
    for o in again:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g()
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


# -------------------------------------------------------------------- axes --

@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("dim,hq,hkv,rope,style,axes,woven,many", [
    (64, 4, 2, 64, INTER, 3, False, False), (128, 28, 4, 128, HALF, 3, True, False), (128, 8, 8, 96, HALF, 2, False, False),
    (64, 2, 1, 16, INTER, 4, True, False), (128, 5, 5, 64, INTER, 1, False, False), (64, 3, 1, 64, HALF, 4, True, True),
    (128, 64, 8, 128, HALF, 3, False, True), (128, 200, 2, 64, INTER, 2, True, True), (64, 0, 2, 32, HALF, 3, False, True)])
def test_append_of_several_axes(dtype, dim, hq, hkv, rope, style, axes, woven, many):
    lengths, starts = ([901, 0, 1, 400, 64], [0, 5, 63, 60, 128]) if many else ([3, 0, 1, 70, 64], [0, 5, 63, 60, 128])
    rng = np.random.default_rng(dim + hq + rope + axes)
    cfg = csa.KVCfg(hq or hkv, hkv, dim, dtype, rope_dims=rope, rope_style=style)
    cache = csa.KVCache(cfg, 5, max(a + b for a, b in zip(lengths, starts)), spare_pages=1)
    T, pairs, rows = sum(lengths), rope // 2, 700
    x = _kv.normal(rng, T, hq + 2 * hkv, dim)
    wide = _dev(x)
    where = rng.integers(0, rows, (T, axes))
    of = [i % axes for i in range(pairs)] if woven else sorted(rng.integers(0, axes, pairs).tolist())
    table = csa.rope_table(rows, rope)
    q_out = torch.empty(T, hq, dim, dtype=torch.bfloat16, device="cuda") if hq else None
    k_out, v_out = (torch.empty(T, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    st = _status()
    csa.kv_append_axes(cfg, wide[:, hq:hq + hkv], wide[:, hq + hkv:], _cu(lengths), torch.tensor(starts, device="cuda"), cache,
                       _dev(where, torch.int32), of, table, q=wide[:, :hq] if hq else None, q_out=q_out, k_out=k_out,
                       v_out=v_out, status=st)
    assert int(st.item()) == 0
    # the restatement takes one row of angles a token: these rows, put together for each
    angles = table.cpu().numpy()[where[:, of], np.arange(pairs)]
    turn = lambda rows_: _kv.rotate(rows_, angles, np.arange(T), rope, style == HALF)
    if hq:
        assert torch.equal(q_out.cpu(), torch.from_numpy(turn(x[:, :hq])).to(torch.bfloat16))
    want = {"k": turn(x[:, hq:hq + hkv]), "v": x[:, hq + hkv:]}
    t0 = 0
    for b, (n, s) in enumerate(zip(lengths, starts)):
        for kind, plain in (("k", k_out), ("v", v_out)):
            part = want[kind][t0:t0 + n]
            val = _kv.fp4_round(part)[0] if dtype == FP4 else _kv.bf16(part)
            assert np.array_equal(_kv.read(cache, cfg, b, kind, s + n)[0][s:], val)
            assert np.array_equal(plain[t0:t0 + n].double().cpu().numpy(), val)
        t0 += n


@pytest.mark.parametrize("many", [False, True])
def test_axes_all_alike_are_the_plain_append(many):
    rng = np.random.default_rng(2)
    n = 3000 if many else 9
    cfg = csa.KVCfg(16, 4, 128, FP4, rope_dims=128, rope_style=HALF)
    table = csa.rope_table(n + 20, 128)
    q, k, v = (_dev(_kv.normal(rng, n, h, 128)) for h in (16, 4, 4))
    pos0 = torch.tensor([11], device="cuda")
    a, b = csa.KVCache(cfg, 1, n + 20), csa.KVCache(cfg, 1, n + 20)
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    csa.kv_append(cfg, k, v, _cu([n]), pos0, a, rope=table, q=q, q_out=qa)
    where = (11 + torch.arange(n, device="cuda", dtype=torch.int32))[:, None].repeat(1, 3)
    csa.kv_append_axes(cfg, k, v, _cu([n]), pos0, b, where, [0, 1, 2, 1] * 16, table, q=q, q_out=qb)
    assert torch.equal(qa, qb)
    for x, y in ((a.k_data, b.k_data), (a.v_data, b.v_data), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("many", [False, True])
def test_axes_outside_the_table_are_reported(many):
    """A row with a position outside is skipped, the others stand; a running position past the table is none."""
    rng = np.random.default_rng(4)
    n = 3000 if many else 6
    cfg = csa.KVCfg(8, 2, 64, BF16, rope_dims=64)
    table = csa.rope_table(5, 64)
    k, v = (_dev(_kv.normal(rng, n, 2, 64)) for _ in "kv")
    where = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    where[2, 0], where[4, 1] = 5, -1
    cache = csa.KVCache(cfg, 1, n + 90)
    k_out = torch.full((n, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    st = _status()
    csa.kv_append_axes(cfg, k, v, _cu([n]), torch.tensor([80], device="cuda"), cache, where, [0, 1] * 16, table, k_out=k_out,
                       status=st)
    assert int(st.item()) == 17
    good = [i for i in range(n) if i not in (2, 4)]
    assert torch.equal(k_out[good], k[good]) and (k_out[[2, 4]] == 7).all()  # (angles of position 0 turn nothing)


# ------------------------------------------------------------------- beams --

def _select(logits, cum, take, done=None, end=0, status=None):
    groups = cum.shape[0]
    out = [torch.full((groups, take), 5, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    lse = torch.full((logits.shape[0],), 5.0, device="cuda")
    ws = torch.full((max(256, csa.beam_workspace_bytes(groups, cum.shape[1], logits.shape[1], take)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    csa.beam_select(logits, cum, *out, ws, done=done, end_token=end, lse=lse, status=status)
    return (*out, lse)


def _check_beams(logits, cum, take, done=None, end=0, code=0):
    st = _status()
    got = _select(logits, cum, take, done, end, st)
    scores, parents, tokens, lse, off = _step.beam_select(logits.double().cpu().numpy(), cum.double().cpu().numpy(), take,
                                                          None if done is None else done.cpu().numpy(), end)
    g = [t.double().cpu().numpy() for t in got]
    assert int(st.item()) == code
    assert np.array_equal(g[1], parents) and np.array_equal(g[2], tokens)
    fin = np.isfinite(lse)
    assert np.array_equal(fin, np.isfinite(g[3]))
    assert (np.abs(g[3][fin] - lse[fin]) <= off[fin] + 2.0 ** -24 * np.abs(lse[fin])).all()
    there = np.isfinite(scores)
    assert np.array_equal(there, np.isfinite(g[0])) and (g[0][~there] == -np.inf).all()
    # a score's fp64 sum takes the error of its beam's lse; one rounding
    assert (np.abs(g[0][there] - scores[there]) <= off[parents[there]] + 2.0 ** -24 * np.abs(scores[there])).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,take", [
    (1, 1, 1, 1), (1, 1, 7, 16), (2, 3, 2, 16), (1, 4, 1000, 4), (3, 5, 1023, 10), (2, 8, 2049, 16), (1, 2, 16391, 64),
    (5, 1, 4097, 17), (2, 64, 300, 64), (1, 64, 5003, 33), (7, 4, 51865, 8), (1, 3, 128001, 6), (40, 6, 20011, 12),
    (300, 4, 1500, 8)])
def test_beams(groups, beams, vocab, take, dtype):
    rng = np.random.default_rng(groups + beams + vocab)
    n = groups * beams
    # rows of a wider array, an odd distance apart, with more than candidates beside them
    wide = torch.full((n, vocab + 3), float("nan"), dtype=dtype, device="cuda")
    wide[:, :vocab] = _dev(rng.standard_normal((n, vocab)) * 3, dtype)
    wide[:, :vocab][torch.from_numpy(rng.random((n, vocab)) < 0.05).cuda()] = -float("inf")
    cum = _dev(rng.standard_normal((groups, beams)) - 10, torch.float32)
    _check_beams(wide[:, :vocab], cum, take)
    done = _dev(rng.random((groups, beams)) < 0.4, torch.uint8)
    _check_beams(wide[:, :vocab], cum, take, done, vocab // 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,take,beams", [(50000, 16, 3), (700, 64, 2), (2048, 1, 1), (9001, 40, 4), (130000, 33, 8)])
def test_beams_of_ties_and_order(vocab, take, beams, dtype):
    """All logits alike, few values, ascending and descending rows: of equal scores the lower beam, then token."""
    cum = torch.zeros(1, beams, device="cuda")
    flat = torch.full((beams, vocab), 1.5, dtype=dtype, device="cuda")
    _check_beams(flat, cum, take)
    few = _dev(np.random.default_rng(vocab).integers(-2, 3, (beams, vocab)), dtype)
    few[-1] = few[0]
    few[0, vocab // 2:] = few[-1, vocab // 2:] = -0.0
    _check_beams(few, cum, take)
    up = torch.linspace(-20, 20, vocab, device="cuda").to(dtype).repeat(beams, 1)
    _check_beams(up, cum - 0.125 * torch.arange(beams, device="cuda"), take)
    _check_beams(up.flip(1).contiguous(), cum - 0.125 * torch.arange(beams, device="cuda"), take)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [3, 900, 5000, 40001])
def test_beams_that_cannot_go_on(vocab, dtype):
    """Masked rows, beams without a score, single candidates, values that are no number."""
    rng = np.random.default_rng(vocab)
    x = _dev(rng.standard_normal((12, vocab)) * 2, dtype)
    inf = float("inf")
    x[0] = -inf
    x[1] = -inf
    x[1, vocab - 1] = -3.0
    x[2] = torch.finfo(dtype).min
    x[3, : vocab // 2] = torch.finfo(dtype).min
    cum = torch.full((3, 4), -1.0, device="cuda")
    cum[1, 1:] = -inf      # a first step: one beam alone
    cum[2] = -inf          # nothing at all
    _check_beams(x, cum, 8)
    x[4, vocab // 3], x[5, 0], x[6, vocab - 1] = float("nan"), inf, float("nan")
    _check_beams(x, cum, 8, code=19)
    x[4:7] = torch.nan_to_num(x[4:7], 0, 0, -1)
    cum[0, 2], cum[0, 3] = float("nan"), inf
    _check_beams(x, cum, 8, code=19)


@pytest.mark.parametrize("groups,beams,vocab", [(1, 1, 17), (5, 4, 32000), (70, 8, 999), (2, 64, 3001)])
def test_scores_written_over_the_sums_they_come_from(groups, beams, vocab):
    rng = np.random.default_rng(vocab)
    x = _dev(rng.standard_normal((groups * beams, vocab)) * 3)
    cum = _dev(rng.standard_normal((groups, beams)), torch.float32)
    want = _select(x, cum, beams)
    parents, tokens = (torch.empty(groups, beams, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(csa.beam_workspace_bytes(groups, beams, vocab, beams), dtype=torch.uint8, device="cuda")
    csa.beam_select(x, cum, cum, parents, tokens, ws)
    assert torch.equal(cum, want[0]) and torch.equal(parents, want[1]) and torch.equal(tokens, want[2])


def test_beams_beyond_32_bits_of_logits():
    rows, vocab = 40, 60_000_000
    if torch.cuda.mem_get_info()[0] < 12e9:
        pytest.skip("not enough memory")
    x = torch.full((rows, vocab), -4.0, dtype=torch.bfloat16, device="cuda")
    x[rows - 1, vocab - 7], x[3, 59_000_001] = 9.0, 8.0
    cum = torch.zeros(1, rows, device="cuda")
    scores, parents, tokens, lse = _select(x, cum, 3)
    others = np.log(vocab - 1.0) - 4.0
    z = [np.logaddexp(others, a) for a in (9.0, 8.0, -4.0)]
    assert parents.tolist() == [[rows - 1, 3, 0]] and tokens.tolist() == [[vocab - 7, 59_000_001, 0]]
    assert np.allclose(scores.cpu().numpy(), [[9 - z[0], 8 - z[1], -4 - z[2]]], rtol=0, atol=1e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,take", [(30, 64), (5000, 17), (9000, 33), (40001, 64)])
def test_beams_with_fewer_candidates_than_are_taken(vocab, take, dtype):
    rng = np.random.default_rng(vocab)
    x = torch.full((6, vocab), -float("inf"), dtype=dtype, device="cuda")
    x[0, vocab // 2], x[1, 0], x[4, vocab - 1] = 1.0, -2.0, torch.finfo(dtype).min
    x[5, :9] = _dev(rng.standard_normal(9), dtype)
    cum = _dev(rng.standard_normal((2, 3)), torch.float32)
    _check_beams(x, cum, take)
    _check_beams(x, cum, take, _dev(np.array([[0, 1, 0], [1, 1, 0]]), torch.uint8), 3)
    # a row whose logits are all alike beside them
    x[2] = 0.5
    _check_beams(x, cum, take)


FIRST = """
import sys, torch
import compressed_sparse_attention_07_gb300 as csa
rows = int(sys.argv[1])
torch.manual_seed(rows)
w = csa.Fp4Weights.encode(torch.randn(20480, 1280, device="cuda").bfloat16())
x = torch.randn(rows, 1280, device="cuda").bfloat16()
out, again = (torch.full((rows, 20480), 5.0, device="cuda") for _ in range(2))
cum = torch.zeros(rows // 4, 4, device="cuda")
s, p, t = (torch.zeros(rows // 4, 40, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32))
ws = torch.empty(csa.beam_workspace_bytes(rows // 4, 4, 20480, 40), dtype=torch.uint8, device="cuda")

def step():
    csa.fp4_linear(x, w, out)
    csa.beam_select(out, cum, s, p, t, ws)

g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    step()
g.replay()
csa.fp4_linear(x, w, again)
torch.cuda.synchronize()
assert torch.equal(out, again)
best, at = again.view(rows // 4, -1).double().sub(torch.logsumexp(again.double(), 1).view(rows // 4, 4, 1).expand(-1, -1, 20480).reshape(rows // 4, -1)).topk(40)
# half a step of a score below 128 (2^-18) and the exponentials' 2^-20
assert best.min() > -128 and (s.double() - best).abs().max() < 2.0 ** -18 + 2.0 ** -20
print("fine")
"""


@pytest.mark.parametrize("rows", [8, 20, 64, 516])
def test_the_first_calls_of_a_process_inside_a_capture(rows):
    run = subprocess.run([sys.executable, "-c", FIRST, str(rows)], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and run.stdout.strip() == "fine", run.stderr[-2000:]


def test_beams_in_graphs_on_two_streams():
    rng = np.random.default_rng(8)
    sets = []
    for seed in range(2):
        x = _dev(rng.standard_normal((64, 30011)) * 3)
        cum = _dev(rng.standard_normal((8, 8)), torch.float32)
        out = [torch.zeros((8, 16), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
        ws = torch.empty(csa.beam_workspace_bytes(8, 8, 30011, 16), dtype=torch.uint8, device="cuda")
        sets.append((x, cum, out, ws))
    graphs = [csa.capture(lambda s=s: csa.beam_select(s[0], s[1], *s[2], s[3])) for s in sets]
    want = [_select(s[0], s[1], 16)[:3] for s in sets]
    for s in sets:
        for t in s[2]:
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g()
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        for a, b in zip(s[2], w):
            assert torch.equal(a, b)


# ----------------------------------------------------------------- reorder --

def _caches(cfg, layers, table, pages, rng):
    made = []
    for _ in range(layers):
        c = csa.KVCache(cfg, table.shape[0], 64 * table.shape[1], page_order=torch.arange(pages), spare_pages=pages - table.numel())
        for t in (c.k_data, c.v_data, c.k_scales, c.v_scales):
            if t is not None:
                t.view(torch.uint8).random_(0, 256)
        made.append(csa.KVCache.over(cfg, c.k_data, c.v_data, table, c.k_scales, c.v_scales))
    return made


@pytest.mark.parametrize("dtype", [FP4, BF16])
@pytest.mark.parametrize("groups,beams,layers,hkv,dim,lengths", [
    (1, 1, 1, 1, 64, [70]), (1, 4, 3, 2, 64, [0]), (2, 3, 2, 4, 128, [1, 63]), (3, 5, 1, 1, 64, [64, 128, 191]),
    (2, 8, 17, 2, 64, [100, 300]), (4, 33, 2, 1, 128, [65, 130, 200, 255]), (1, 64, 1, 3, 64, [319]), (9, 2, 128, 1, 64, [50] * 9),
    (1, 6, 2, 8, 128, [5000])])
def test_reorder(groups, beams, layers, hkv, dim, lengths, dtype):
    rng = np.random.default_rng(beams + layers + dim)
    cfg = csa.KVCfg(hkv, hkv, dim, dtype, rope_dims=0)
    max_pages = max(lengths) // 64 + 2
    n = groups * beams
    pages = n * max_pages + 3
    host = rng.permutation(pages)[: n * max_pages].reshape(n, max_pages).astype(np.int32)
    for trial in range(4):
        table = _dev(host, torch.int32)
        caches = _caches(cfg, layers, table, pages, rng)
        before = [[t.clone() for t in (c.k_data, c.v_data, c.k_scales, c.v_scales) if t is not None] for c in caches]
        local = [np.arange(beams), rng.integers(0, beams, beams), np.full(beams, beams - 1), rng.permutation(beams)][trial]
        parents = np.concatenate([g * beams + (local if g % 2 == 0 else rng.integers(0, beams, beams)) for g in range(groups)])
        if trial == 1:
            parents[rng.integers(0, n)] = -1
        st = _status()
        csa.kv_reorder(cfg, caches, beams, _dev(parents, torch.int32), _dev(np.repeat(lengths, beams), torch.int32), status=st)
        assert int(st.item()) == 0
        new, copies = _step.reorder(host, parents, lengths, beams)
        assert np.array_equal(table.cpu().numpy(), new)
        for c, old in zip(caches, before):
            now = [t for t in (c.k_data, c.v_data, c.k_scales, c.v_scales) if t is not None]
            for t, o in zip(now, old):
                for a, b, m in copies:
                    if dtype == FP4:
                        o[b, :, :m] = o[a, :, :m]
                    else:
                        o[b, :, :, :m] = o[a, :, :, :m]
                assert torch.equal(t.view(torch.uint8), o.view(torch.uint8))


def test_reorder_reports_what_is_wrong():
    rng = np.random.default_rng(3)
    cfg = csa.KVCfg(2, 2, 64, FP4, rope_dims=0)
    host = np.arange(24, dtype=np.int32).reshape(8, 3)
    good = np.array([0, 0, 1, 3, 4, 5, 4, 5])

    def run(parents=good, length=np.full(8, 100), table=host):
        t = _dev(table, torch.int32)
        caches = _caches(cfg, 2, t, 24, rng)
        was = [c.k_data.clone() for c in caches]
        st = _status()
        csa.kv_reorder(cfg, caches, 4, _dev(parents, torch.int32), _dev(length, torch.int32), status=st)
        return int(st.item()), t.cpu().numpy(), all(torch.equal(c.k_data, w) for c, w in zip(caches, was))

    want = _step.reorder(host, good, [100, 100], 4)[0]
    assert run()[0] == 0
    for bad in (4, -2, 8, 2 ** 31 - 1):  # of another group, or none
        p = good.copy()
        p[1] = bad
        code, t, _ = run(p)
        assert code == 17 and np.array_equal(t[:4], host[:4]) and np.array_equal(t[4:], want[4:])
    for at, n in ((5, 99), (4, 193), (6, -1)):
        length = np.full(8, 100)
        length[at] = n
        if n == 193:
            length[4:] = 193
        code, t, _ = run(length=length)
        assert code == 17 and np.array_equal(t[4:], host[4:]) and np.array_equal(t[:4], want[:4])
    bad = host.copy()
    bad[:, 1] = 24  # last pages that are not there
    code, t, same = run(table=bad)
    assert code == 16 and same


# ----------------------------------------------- a run of them, as in use --

@pytest.mark.parametrize("batch", [3, 24])
def test_projections_feed_the_sparse_path(batch):
    """The model's own decode step with its queries projected just ahead: low-rank ones to the indexer's and to the
    attention's, which the calls read as soon as they may.  Compared with the same calls on queries that lie there."""
    rng = np.random.default_rng(batch)
    cfg = csa.Cfg(ratio=2, topk=64, window=32)
    ctx, lora = 600, 1280
    main = csa.PagedCache(batch, ctx // 2, 512, FP4)
    idx = csa.PagedCache(batch, ctx // 2, 128, FP4)
    x = _dev(_kv.normal(rng, batch, ctx, 512))
    n_ent = torch.zeros(batch, dtype=torch.int32, device="cuda")
    merge = _dev(np.full((2, 512), 0.7), torch.float32)
    csa.compress(cfg, x, torch.zeros(batch, dtype=torch.int64, device="cuda"), merge, _dev(_kv.normal(rng, 512, 128, std=0.04)),
                 main, idx, n_ent)
    wq = csa.Fp4Weights.encode(_dev(_kv.normal(rng, 64 * 512, lora, std=0.02)))
    wi = csa.Fp4Weights.encode(_dev(_kv.normal(rng, 32 * 128, lora, std=0.02)))
    swa = _dev(_kv.normal(rng, batch, 32, 512))
    swa_len = torch.full((batch,), 32, dtype=torch.int32, device="cuda")
    pos = torch.full((batch, 1), ctx - 1, dtype=torch.int64, device="cuda")
    swa_pos0 = torch.full((batch,), ctx - 32, dtype=torch.int64, device="cuda")
    ws = torch.empty(csa.index_workspace_bytes(cfg, batch, 1, ctx // 2), dtype=torch.uint8, device="cuda")

    def step(low, q, q_idx, topk, out, project):
        if project:
            csa.fp4_linear(low, wq, q.view(batch, -1))
            csa.fp4_linear(low, wi, q_idx.view(batch, -1))
        csa.index_topk(cfg, q_idx, pos, idx, n_ent, ctx // 2, topk, ws)
        csa.attend(cfg, q, main, n_ent, topk, swa, swa_len, swa_pos0, pos, out)

    def room():
        return (torch.zeros(batch, 1, 64, 512, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(batch, 1, 32, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(batch, 1, 64, dtype=torch.int32, device="cuda"), torch.zeros(batch, 1, 64, 512, device="cuda"))

    a, b = room(), room()
    low = _dev(_kv.normal(rng, batch, lora))
    graph = csa.capture(lambda: step(low, *a, True))
    for _ in range(4):
        low.copy_(_dev(_kv.normal(rng, batch, lora)))
        graph()
        torch.cuda.synchronize()
        b[0].copy_(a[0]), b[1].copy_(a[1])
        torch.cuda.synchronize()
        step(low, *b, False)
        torch.cuda.synchronize()
        assert torch.isfinite(a[3]).all() and (a[3] != 0).any()
        assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])



@pytest.mark.parametrize("dtype", [FP4, BF16])
def test_a_captioner_writes_with_beams(dtype):
    """Prompts with image tokens, then steps of: projection -> append -> attention -> logits -> beams -> reorder, over
    two layers, the steps from a captured graph.  What each beam has cached is followed token by token."""
    rng = np.random.default_rng(11)
    G, K, hidden, hq, hkv, dim, vocab, layers, steps = 2, 3, 256, 4, 2, 64, 1003, 2, 70
    N, axes, of = G * K, 3, [0] * 8 + [1] * 12 + [2] * 12
    prompt = [70, 33]
    cfg = csa.KVCfg(hq, hkv, dim, dtype, rope_dims=64, rope_style=HALF)
    width = (hq + 2 * hkv) * dim
    qkv_w = [csa.Fp4Weights.encode(_dev(_kv.normal(rng, width, hidden, std=1 / 16))) for _ in range(layers)]
    out_w = [csa.Fp4Weights.encode(_dev(_kv.normal(rng, hidden, hq * dim, std=1 / 16))) for _ in range(layers)]
    head = csa.Fp4Weights.encode(_dev(_kv.normal(rng, vocab, hidden, std=1 / 4)))
    embed = _dev(_kv.normal(rng, vocab, hidden))
    first = csa.KVCache(cfg, N, 70 + steps + 2)
    caches = [first] + [csa.KVCache.over(cfg, *(torch.zeros_like(t) for t in (first.k_data, first.v_data)), first.block_table,
                                         *(None if t is None else torch.zeros_like(t) for t in (first.k_scales, first.v_scales)))
                        for _ in range(layers - 1)]
    rope = csa.rope_table(200, 64)
    stored = [[None] * N for _ in range(layers)]  # k and v rows of each beam

    def forward(x, cu, pos0, where, kv_len, max_q, max_kv, ws, keep):
        for l in range(layers):
            qkv = torch.empty(x.shape[0], hq + 2 * hkv, dim, dtype=torch.bfloat16, device="cuda")
            csa.fp4_linear(x, qkv_w[l], qkv.view(x.shape[0], width))
            q, k, v = qkv.split((hq, hkv, hkv), 1)
            kk, vv = (torch.empty(x.shape[0], hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
            csa.kv_append_axes(cfg, k, v, cu, pos0, caches[l], where, of, rope, q=q, q_out=q, k_out=kk, v_out=vv)
            o = torch.empty(x.shape[0], hq, dim, dtype=torch.bfloat16, device="cuda")
            csa.kv_attend(cfg, q, cu, caches[l], kv_len, max_q, max_kv, o, workspace=ws)
            keep.append((q, kk, vv, o))
            y = torch.empty_like(x)
            csa.fp4_linear(o.view(x.shape[0], hq * dim), out_w[l], y)
            x = x + y
        logits = torch.empty(x.shape[0], vocab, device="cuda")
        csa.fp4_linear(x, head, logits)
        return logits

    # the prompts, in each group's first beam
    lengths = [prompt[i // K] if i % K == 0 else 0 for i in range(N)]
    T = sum(lengths)
    kv_len = _dev(np.array(lengths), torch.int32)
    keep = []
    x = _dev(_kv.normal(rng, T, hidden))
    where = _dev(np.concatenate([np.minimum(np.arange(n)[:, None], [n, 5, 9]) for n in prompt]), torch.int32)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    logits = forward(x, _cu(lengths), torch.zeros(N, dtype=torch.int64, device="cuda"), where, kv_len, max(lengths), first.capacity, ws, keep)
    for l, (q, k, v, o) in enumerate(keep):
        t0 = 0
        for i, n in enumerate(lengths):
            stored[l][i] = [k[t0:t0 + n].double().cpu().numpy(), v[t0:t0 + n].double().cpu().numpy()] if n else None
            t0 += n
    last = _dev(np.cumsum(prompt) - 1, torch.int64)
    state = torch.zeros(N, vocab, device="cuda")
    state[::K] = logits[last]
    cum = torch.full((G, K), -float("inf"), device="cuda")
    cum[:, 0] = 0.0
    length = _dev(np.repeat(prompt, K), torch.int32)
    parents, tokens = (torch.empty(G, K, dtype=torch.int32, device="cuda") for _ in "pt")
    bws = torch.empty(csa.beam_workspace_bytes(G, K, vocab, K), dtype=torch.uint8, device="cuda")
    st, one = _status(), _cu([1] * N)
    where1 = torch.empty(N, axes, dtype=torch.int32, device="cuda")
    graph, kept = None, []

    def step():
        csa.beam_select(state, cum, cum, parents, tokens, bws, status=st)  # (each group's cum is read before it is written)
        csa.kv_reorder(cfg, caches, K, parents.view(-1), length, status=st)
        pos0 = length.long()
        where1.copy_(length[:, None].expand(N, axes))
        length.add_(1)
        del kept[:]
        state.copy_(forward(embed[tokens.view(-1).long()], one, pos0, where1, length, 1, first.capacity, ws, kept))

    for i in range(steps):
        was = (state.double().cpu().numpy(), cum.double().cpu().numpy(), first.block_table.cpu().numpy().copy(), length.cpu().numpy().copy())
        if i < 2:
            step()
        else:
            if graph is None:
                # (a capture runs nothing: the step is the first replay's)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        s, p, t, _, _ = _step.beam_select(was[0], was[1], K)
        assert np.array_equal(parents.cpu().numpy(), p) and np.array_equal(tokens.cpu().numpy(), t)
        assert np.allclose(cum.cpu().numpy(), s, atol=1e-4)
        assert np.array_equal(first.block_table.cpu().numpy(), _step.reorder(was[2], p.ravel(), was[3][::K], K)[0])
        for l, (q, k, v, o) in enumerate(kept):
            rows = [t_.double().cpu().numpy() for t_ in (k, v)]
            stored[l] = [[np.concatenate([a, r[j:j + 1]]) for a, r in zip(stored[l][par], rows)] for j, par in enumerate(p.ravel())]
            if i % 23 in (0, 1) or i == steps - 1:
                for j in range(N):
                    n = len(stored[l][j][0])
                    for kind, want in zip("kv", stored[l][j]):
                        assert np.array_equal(_kv.read(caches[l], cfg, j, kind, n)[0], want), (i, l, j)
                    out, lse, *rest = _kv.attend(q[j:j + 1].double().cpu().numpy(), *stored[l][j], dim ** -0.5, True)
                    tol, _ = _kv.tolerances(cfg, n, out, lse, *rest)
                    assert (np.abs(o[j:j + 1].double().cpu().numpy() - out) <= tol).all()


def _peaked_bound(x):
    """Of rows whose largest stands alone, a bound on |log-sum-exp - largest - exact| in fp32: what is beside the largest is
    off by 2^-22 and by its distance times 2^-22 (arguments of exponentials), and 2^-24 by rounding; the 64-bit sum of 1 and
    what is beside it is itself rounded at 2^-53, and so is its logarithm."""
    x = np.asarray(x, np.float64)
    d = np.where(np.isfinite(x), x, -1e4) - x.max(1, keepdims=True)
    e = np.exp(d) * (d < 0)
    return (e * (2.0 ** -22 + 2.0 ** -22 * np.abs(d))).sum(1) + 2.0 ** -24 * np.log1p(e.sum(1)) + 2.0 ** -52


@pytest.mark.parametrize("stride", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beams_with_the_same_largest_logit_keep_their_own_sums(dtype, stride):
    """Two words, the second far below: the sums are 1 and a little, and the beam with less beside it comes first.  A beam
    that is done beside them (its sum counts as 1 of a largest of 0) lends its sum to none."""
    wide = torch.zeros(6, stride, dtype=dtype, device="cuda")
    wide[:, 1] = torch.tensor([-14, -16.1, -15, -16.1, -14, -30], dtype=dtype)
    x = wide[:, :2]
    xs = x.double().cpu().numpy()
    for cum in (torch.zeros(1, 6, device="cuda"), torch.zeros(3, 2, device="cuda")):
        for done in (None, torch.zeros_like(cum, dtype=torch.uint8)):
            if done is not None:
                done.view(-1)[4] = 1
            scores, parents, tokens, lse = _select(x, cum, 4, done, 1)
            s, p, t, want, _ = _step.beam_select(xs, cum.double().cpu().numpy(), 4, None if done is None else done.cpu().numpy(), 1)
            assert np.array_equal(parents.cpu().numpy(), p) and np.array_equal(tokens.cpu().numpy(), t)
            off = _peaked_bound(xs)
            assert (np.abs(lse.double().cpu().numpy() - want) <= off).all()
            there = p >= 0
            got = scores.double().cpu().numpy()
            assert (np.abs(got[there] - s[there]) <= off[p[there]] + 2.0 ** -24 * np.abs(s[there])).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beams,vocab,pad", [(2, 9, 0), (5, 51865, 0), (8, 128001, 0), (64, 1003, 0), (16, 4099, 2), (8, 70000, 1)])
def test_beams_of_the_same_logits_have_the_same_sums(beams, vocab, pad, dtype):
    """Wherever their rows begin: ties go to the lower beam.  A row that differs in one
    word is not the same."""
    rng = np.random.default_rng(beams + vocab)
    wide = torch.full((2 * beams, vocab + pad), float("nan"), dtype=dtype, device="cuda")
    x = wide[:, :vocab]
    x[:] = _dev(rng.standard_normal(vocab) * 3, dtype)
    x[:, vocab // 2] = -0.0
    x[1::2, vocab // 2] = 0.0
    x[beams + 1, vocab // 4] = 5.5  # (in the second group; of 128001 words a change of 2e-5, and an error of 2^-18 at most)
    cum = torch.full((2, beams), -3.5, device="cuda")
    _check_beams(x, cum, min(64, 2 * beams))
    lse = _select(x, cum, 4)[3].view(2, beams)
    assert (lse[0] == lse[0, 0]).all() and (lse[1, [i for i in range(beams) if i != 1]] == lse[1, 0]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,beams,likely", [(32000, 16, 28), (32001, 16, 28), (8, 4, 17), (2048, 8, 21), (128001, 8, 30), (5003, 64, 24)])
def test_beams_of_one_likely_word_each(vocab, beams, likely, dtype):
    """The same likely word everywhere: what is beside it, 1e-7 of it or so, decides between the beams, and is their score."""
    rng = np.random.default_rng(vocab + beams)
    x = _dev(rng.standard_normal((3 * beams, vocab)) * 2, dtype)
    x[:, vocab // 3] = likely
    x[beams:2 * beams, 1] = likely - 12  # beside another word in its vector's or another's
    x[2 * beams:, vocab - 1] = likely - 9
    cum = torch.zeros(3, beams, device="cuda")
    take = max(1, beams // 2)
    got = [t.double().cpu().numpy() for t in _select(x, cum, take)]
    xs = x.double().cpu().numpy()
    s, p, t, lse, _ = _step.beam_select(xs, cum.double().cpu().numpy(), take + 1)
    off = _peaked_bound(xs)
    gap = 2 * off.reshape(3, beams).max(1, keepdims=True)
    sure = (s[:, :-1] - s[:, 1:] > gap) & (np.concatenate([np.full((3, 1), np.inf), s[:, :-2] - s[:, 1:-1]], 1) > gap)
    assert sure[0].mean() > 0.9 and sure.mean() > 0.5
    assert np.array_equal(got[1][sure], p[:, :-1][sure]) and np.array_equal(got[2], t[:, :-1])
    assert (np.abs(got[0] - s[:, :-1])[sure] <= (off[p[:, :-1]] + 2.0 ** -24 * np.abs(s[:, :-1]))[sure]).all()
    assert (np.abs(got[3] - lse) <= off + 2.0 ** -24 * np.abs(lse)).all()


def test_weights_laid_out_on_another_stream():
    """What the current stream still does with memory that was freed does not reach the weights, and the largest weight is
    read after what the given stream has yet to write."""
    rng = np.random.default_rng(3)
    n, k = 512, 1024
    codes, scales = _dev(rng.integers(0, 256, (n, k // 2)), torch.uint8), _dev(rng.integers(0x20, 0x50, (n, k // 16)), torch.uint8)
    w = _dev(_kv.normal(rng, n, k, std=0.02))
    want, same = csa.Fp4Weights.pack(codes, scales), csa.Fp4Weights.encode(w)
    late = torch.full_like(w, 100.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for wanted, make in ((want, lambda: csa.Fp4Weights.pack(codes, scales, stream=s)),
                         (same, lambda: csa.Fp4Weights.encode(w, 1 / same.alpha, stream=s))):
        freed = torch.empty_like(want.data)
        torch.cuda._sleep(20_000_000)
        freed.fill_(255)
        del freed
        got = make()
        torch.cuda.synchronize()
        assert torch.equal(got.data, wanted.data)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(w)
    got = csa.Fp4Weights.encode(late, stream=s)
    torch.cuda.synchronize()
    assert got.alpha == same.alpha and torch.equal(got.data, same.data)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,k,n", [(1, 64, 40), (16, 64, 40), (20, 64, 40), (40, 2048, 700), (70, 64, 300), (300, 64, 300)])
@pytest.mark.parametrize("alpha", [2.0 ** 127, -1.5 * 2.0 ** 121, 2.0 ** -126])
def test_any_factor_that_fp32_has(alpha, T, k, n, f32):
    rng = np.random.default_rng(T + n)
    w, plain = _packed(rng, n, k, alpha, 0x38, 0x39)
    size = 2.0 ** -60 if abs(alpha) > 1 else 2.0 ** 60
    x = rng.integers(-3, 4, (T, k)) * size
    x[-1] = 0.0
    out = torch.empty(T, n, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    csa.fp4_linear(_dev(x), w, out)
    want = torch.from_numpy(x @ plain.T * alpha)  # (whole multiples, which fp32 holds)
    assert torch.equal(out.cpu().double(), want.to(out.dtype).double())


def _cut_off(adds, joins):
    """Of what additions to an accumulator that cuts off below 24 bits, and then of such sums in fp32, make of a sum of
    random terms, relative to it.  The j-th of `adds` finds (j / adds)^(1/2) of the sum and loses, towards zero, half a
    step of 2^-23 of that times 0.72 (the mean of 1 / m for a mantissa m in [1, 2) is log 2 = 0.69, weighted as 1 / m by
    Benford 0.72): all of them 2 / 3 adds 2^-24 0.72.  Joins round either way, by 2^-24 / 3^(1/2) of the sum so far."""
    return adds * 2 / 3 * 2.0 ** -24 * 0.72 + (joins / 6) ** 0.5 * 2.0 ** -24 + 2.0 ** -24


@pytest.mark.parametrize("T,k,n,adds", [(1, 4096, 700, 8), (16, 4096, 700, 8), (17, 4096, 700, 64), (40, 4096, 40000, 64),
                                        (64, 1280, 700, 64), (128, 4096, 700, 64), (16, 16384, 300, 64),
                                        (60, 16384, 300, 64), (300, 16384, 300, 64), (300, 1024, 700, 64),
                                        (300, 4096, 300, 256), (20, 70000, 40, 64), (130, 70000, 40, 64)])
def test_fp32_outputs_are_sums_of_short_sums(T, k, n, adds):
    """An accumulator takes 128 channels of few rows, 1024 of more, 4096 of more than 128: that many 16s."""
    rng = np.random.default_rng(T + k)
    w, plain = _packed(rng, n, k, 1.0 / np.sqrt(k))
    x = _dev(_kv.normal(rng, T, k))
    out = torch.empty(T, n, device="cuda")
    csa.fp4_linear(x, w, out)
    y = x.double() @ torch.from_numpy(plain).cuda().T * float(np.float32(1.0 / np.sqrt(k)))
    assert float((out.double() - y).norm() / y.norm()) <= _cut_off(adds, k / (16 * adds))


def test_bf16_outputs_of_very_long_rows():
    rng = np.random.default_rng(1)
    k = 1 << 18
    w, plain = _packed(rng, 36, k, 1.0 / np.sqrt(k))
    for T in (20, 200):
        x = _dev(_kv.normal(rng, T, k))
        out = torch.empty(T, 36, dtype=torch.bfloat16, device="cuda")
        csa.fp4_linear(x, w, out)
        y = x.double() @ torch.from_numpy(plain).cuda().T * float(np.float32(1.0 / np.sqrt(k)))
        # half a step of bf16, and five times what sums of 1024 channels lose
        assert ((out.double() - y).abs() <= 2.0 ** -8 * y.abs() + 5 * _cut_off(64, k / 1024) * y.norm() / y.numel() ** 0.5).all()


@pytest.mark.parametrize("T", [1, 8, 16, 17, 200])
@pytest.mark.parametrize("below", [24, 31, 34, 39, 41, 60])
def test_channels_far_below_their_rows_largest(T, below):
    """The largest meets a weight of 0, and the outputs come from channels 2^-below of it: exact down to 2^-31, else off by
    2^-39 of the largest each (what f16 keeps beside it); more than 16 rows are exact."""
    rng = np.random.default_rng(below)
    n, k = 48, 256
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    codes[:, 0] &= 0xF0
    w = csa.Fp4Weights.pack(_dev(codes, torch.uint8), torch.full((n, k // 16), 0x38, dtype=torch.uint8, device="cuda"))
    plain = _step.weights(codes, np.full((n, k // 16), 0x38, np.uint8))
    x = rng.integers(64, 128, (T, k)) / 64.0 * np.where(rng.random((T, k)) < 0.5, -1, 1) * 2.0 ** -below
    x[:, 0] = 1.75
    out = torch.empty(T, n, device="cuda")
    csa.fp4_linear(_dev(x), w, out)
    got, want = out.double().cpu().numpy(), x @ plain.T  # (whole multiples of 2^-7 below, less than 2^17 of them: fp32 holds every sum)
    if T > 16 or below <= 31:
        assert np.array_equal(got, want)
    else:
        assert (np.abs(got - want) <= 2.0 ** -39 * 1.75 * np.abs(plain).sum(1)).all()


@pytest.mark.parametrize("stride", [4000, 4001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_fp64_does_not_hold_beside_one_decides_nothing(dtype, stride):
    """One word with all the probability that fp64 tells from 1, what is beside it anywhere in the row: ties, of which the
    lower beam comes first."""
    wide = torch.full((6, stride), -1000.0, dtype=dtype, device="cuda")
    for i, (word, gap) in enumerate([(3, 44), (2000, 60), (3999, 50), (17, 48), (1234, 80), (3000, 41)]):
        wide[i, word] = 20.0
        wide[i, (word + 1777 * (i + 1)) % 4000] = 20.0 - gap
    _check_beams(wide[:, :4000], torch.zeros(1, 6, device="cuda"), 6)
    _check_beams(wide[:, :4000], torch.zeros(2, 3, device="cuda"), 3)
