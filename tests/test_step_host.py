"""The operators of a generation step without a GPU: sizes, refusals (each call below fails validation, so nothing is
launched) and the plain restatement that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import compressed_sparse_attention_07_gb300 as csa
import oracle
from tests import _step

FAKE = 0x10000  # never dereferenced


def _kv_cache(**kw):
    d = dict(k_data=FAKE, k_scales=FAKE, v_data=FAKE, v_scales=FAKE, block_table=FAKE, max_pages=4, num_pages=8)
    d.update(kw)
    return csa._KVCacheDesc(**d)


# ------------------------------------------------------------- projections --

def _linear(w=None, **kw):
    a = dict(T=4, x=FAKE, xs=256, bias=None, out=FAKE, dtype=0, os=128, status=None)
    a.update(kw)
    d = dict(data=FAKE, n=100, k=256, alpha=1.0, reserved=0)
    d.update(w or {})
    return csa.load().csa2_fp4_linear(C.byref(csa._Fp4Desc(**d)), a["T"], a["x"], a["xs"], a["bias"], a["out"], a["dtype"],
                                      a["os"], a["status"], None)


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=FAKE + 64), dict(n=0), dict(k=0), dict(k=24), dict(k=1 << 24),
                                 dict(n=1 << 24), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(reserved=1)])
def test_weights_refused(bad):
    assert _linear(bad) == 1


@pytest.mark.parametrize("bad", [dict(T=-1), dict(x=None), dict(x=FAKE + 8), dict(xs=248), dict(xs=260), dict(out=None),
                                 dict(out=FAKE + 1), dict(out=FAKE + 2, dtype=1), dict(os=99), dict(dtype=2), dict(bias=FAKE + 1),
                                 dict(status=FAKE + 2)])
def test_linear_arguments_refused(bad):
    assert _linear(**bad) == 1


def test_no_rows_are_nothing_to_do():
    assert _linear(T=0, x=None, out=None) == 0


def test_weight_bytes():
    f = csa.load().csa2_fp4_weight_bytes
    # blocks of 16 rows x 128 channels, eight of them together: 9/16 of a byte a weight
    assert f(128, 128) == 128 * 128 * 9 // 16
    assert f(1, 16) == f(128, 128)
    assert f(129, 144) == 4 * f(128, 128)
    for n, k in ((0, 16), (1, 0), (1, 8), (1 << 24, 16), (16, 1 << 24), (-1, 16)):
        assert f(n, k) == 0


@pytest.mark.parametrize("bad", [dict(n=0), dict(k=24), dict(w=None), dict(w=FAKE + 8), dict(stride=248), dict(stride=252),
                                 dict(gain=float("nan")), dict(packed=None), dict(packed=FAKE + 64), dict(status=FAKE + 1)])
def test_encode_arguments_refused(bad):
    a = dict(n=16, k=256, w=FAKE, stride=256, gain=1.0, packed=FAKE, status=None)
    a.update(bad)
    assert csa.load().csa2_fp4_encode(a["n"], a["k"], a["w"], a["stride"], a["gain"], a["packed"], a["status"], None) == 1


@pytest.mark.parametrize("bad", [dict(n=0), dict(k=24), dict(codes=None), dict(codes=FAKE + 2), dict(scales=None),
                                 dict(packed=None), dict(packed=FAKE + 32), dict(status=FAKE + 1)])
def test_pack_arguments_refused(bad):
    a = dict(n=16, k=256, codes=FAKE, scales=FAKE, packed=FAKE, status=None)
    a.update(bad)
    assert csa.load().csa2_fp4_pack(a["n"], a["k"], a["codes"], a["scales"], a["packed"], a["status"], None) == 1


# ------------------------------------------------------------------- beams --

def _beam(**kw):
    a = dict(groups=2, beams=4, vocab=100, take=8, logits=FAKE, dtype=0, stride=100, cum=FAKE, done=None, end=0, scores=FAKE,
             parents=FAKE, tokens=FAKE, lse=None, ws=FAKE, wn=1 << 20, status=None)
    a.update(kw)
    return csa.load().csa2_beam_select(
        a["groups"], a["beams"], a["vocab"], a["take"], a["logits"], a["dtype"], a["stride"], a["cum"], a["done"], a["end"],
        a["scores"], a["parents"], a["tokens"], a["lse"], a["ws"], a["wn"], a["status"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(groups=-1), 1), (dict(beams=0), 1), (dict(vocab=0), 1), (dict(take=0), 1), (dict(beams=65), 2), (dict(take=65), 2),
    (dict(groups=1 << 30, beams=64), 2), (dict(logits=None), 1), (dict(logits=FAKE + 8), 1), (dict(stride=99), 1),
    (dict(cum=None), 1), (dict(cum=FAKE + 2), 1), (dict(scores=None), 1), (dict(parents=None), 1), (dict(tokens=FAKE + 1), 1),
    (dict(lse=FAKE + 2), 1), (dict(dtype=3), 1), (dict(done=FAKE, end=100), 1), (dict(done=FAKE, end=-1), 1),
    (dict(ws=None), 4), (dict(wn=16), 4), (dict(ws=FAKE + 16), 1), (dict(status=FAKE + 1), 1)])
def test_beam_arguments_refused(bad, code):
    assert _beam(**bad) == code


def test_no_groups_are_nothing_to_do():
    assert _beam(groups=0, logits=None) == 0


def test_beam_workspace_grows_with_what_it_holds():
    f = csa.beam_workspace_bytes
    assert f(1, 65, 100, 1) == 0 and f(1, 1, 100, 65) == 0 and f(1, 1, 0, 1) == 0
    assert 0 < f(1, 1, 1, 1) <= f(1, 4, 1, 1) <= f(1, 4, 1, 64) <= f(64, 4, 1, 64)
    # a part of a row has at least 1024 logits but the last
    assert f(1, 1, 1 << 20, 1) <= 256 + 1024 * 16 + 1024 * 8


# ----------------------------------------------------------------- reorder --

def _reorder(cfg=None, caches=None, **kw):
    cfg = csa.KVCfg() if cfg is None else cfg
    caches = [_kv_cache(), _kv_cache()] if caches is None else caches
    a = dict(layers=len(caches), groups=2, beams=4, parents=FAKE, kv_len=FAKE, status=None)
    a.update(kw)
    array = (csa._KVCacheDesc * max(1, len(caches)))(*caches)
    return csa.load().csa2_kv_reorder(C.byref(cfg), a["layers"], array, a["groups"], a["beams"], a["parents"], a["kv_len"],
                                      a["status"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(layers=-1), 1), (dict(groups=-1), 1), (dict(beams=0), 1), (dict(beams=65), 1), (dict(layers=129), 2),
    (dict(groups=1 << 23, beams=4), 2), (dict(parents=None), 1), (dict(kv_len=None), 1), (dict(parents=FAKE + 2), 1),
    (dict(kv_len=FAKE + 1), 1), (dict(status=FAKE + 2), 1)])
def test_reorder_arguments_refused(bad, code):
    assert _reorder(**bad) == code


@pytest.mark.parametrize("bad", [dict(block_table=FAKE + 64), dict(max_pages=5), dict(num_pages=9), dict(k_data=None),
                                 dict(v_scales=None)])
def test_layers_of_unlike_caches_refused(bad):
    assert _reorder(caches=[_kv_cache(), _kv_cache(**bad)]) == 1


def test_nothing_to_reorder():
    assert _reorder(caches=[], layers=0) == 0
    assert _reorder(groups=0, parents=None) == 0


def test_reordering_keeps_every_last_page_its_own():
    """The rule itself, many steps of random parents: no two beams ever write to one page, every beam reads what its
    parents wrote, and no page is needed that the table does not hold."""
    rng = np.random.default_rng(0)
    beams, max_pages = 5, 6
    table = np.arange(beams * max_pages).reshape(beams, max_pages)
    table[:, 0] = 0  # a shared full page of the prompt, and part of the next in the first beam alone
    store = np.full((beams * max_pages, 64), -1)
    length, said = 70, [[] for _ in range(beams)]
    store[0] = np.arange(64)
    store[table[0, 1], :6] = np.arange(64, 70)
    said[0] = list(range(70))
    parents = np.zeros(beams, int)
    for step in range(300):
        table, copies = _step.reorder(table, parents, [length], beams)
        for a, b, n in copies:
            store[b, :n] = store[a, :n]
        said = [list(said[p]) if p >= 0 else None for p in parents]
        live = [i for i in range(beams) if said[i] is not None]
        page, slot = divmod(length, 64)
        assert len({table[i, page] for i in range(beams)}) == beams
        for i in live:
            got = [store[table[i, j // 64], j % 64] for j in range(length)]
            assert got == said[i]
            word = 1000 + step * beams + i
            store[table[i, page], slot] = word
            said[i].append(word)
        length += 1
        if length == 64 * max_pages:
            break
        parents = rng.choice(live, beams)
        if rng.random() < 0.2 and len(live) > 1:
            parents[rng.integers(beams)] = -1
            if (parents < 0).all():
                parents[0] = live[0]


# -------------------------------------------------------------------- axes --

def _axes(cfg=None, **kw):
    cfg = csa.KVCfg() if cfg is None else cfg
    a = dict(B=1, T=4, axes=FAKE, n_axes=3, axis_of=bytes([0, 1, 2, 0] * 8), rope=FAKE, rows=64)
    a.update(kw)
    return csa.load().csa2_kv_append_axes(
        C.byref(cfg), a["B"], a["T"], None, 0, FAKE, 1024, FAKE, 1024, FAKE, FAKE, a["axes"], a["n_axes"], a["axis_of"],
        a["rope"], a["rows"], C.byref(_kv_cache()), None, 0, None, None, FAKE + 1, None)


@pytest.mark.parametrize("bad", [dict(axes=None), dict(axes=FAKE + 2), dict(n_axes=0), dict(n_axes=5), dict(axis_of=None),
                                 dict(axis_of=bytes([0] * 31 + [3])), dict(rope=None), dict(rows=-1), dict()])
def test_axes_refused(bad):
    assert _axes(**bad) == 1  # (with a status that is not aligned: good arguments are refused for that alone)


def test_axes_without_rotation_refused():
    c = csa.KVCfg(rope_dims=0)
    assert _axes(c, rope=None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    with pytest.raises(ValueError):
        csa.beam_select(torch.zeros(4, 10), torch.zeros(1, 4), torch.zeros(1, 2), torch.zeros(1, 2, dtype=torch.int32),
                        torch.zeros(1, 2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8))
    w = csa.Fp4Weights(torch.zeros(9216, dtype=torch.uint8), 16, 64, 1.0)
    x, out = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 16)
    for args in ((x, w, out), (x.float(), w, out), (x[:, :32], w, out), (x, w, out.half()), (x, w, out[:1])):
        with pytest.raises((TypeError, ValueError)):
            csa.fp4_linear(*args)
    with pytest.raises(ValueError):
        csa.Fp4Weights.pack(torch.zeros(4, 12, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))


# ------------------------------------------------------------- restatement --

def test_plain_weights_are_the_oracles():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (7, 32), dtype=np.uint8)
    scales = rng.integers(0, 127, (7, 4), dtype=np.uint8)
    assert np.array_equal(_step.weights(codes, scales), oracle.fp4_decode(codes, scales))
    every = np.arange(127, dtype=np.uint8)
    assert np.array_equal(_step.e4m3(every), torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy())


def test_plain_selection_by_hand():
    logits = np.log(np.array([[0.5, 0.25, 0.25], [0.25, 0.5, 0.25]]))
    s, p, t, lse, _ = _step.beam_select(logits, np.array([[0.0, 0.0]]), 4)
    assert np.allclose(lse, 0) and p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 1, 1, 2]]
    s, p, t, lse, _ = _step.beam_select(logits, np.array([[0.0, -0.1]]), 3, np.array([[0, 1]]), end=2)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[2, 0, 1]] and lse[1] == 0 and s[0, 0] == -0.1


def test_sizes_that_32_bits_of_places_do_not_hold_are_refused():
    assert csa.beam_workspace_bytes(1, 1, 1 << 30, 1) > 0
    for vocab in ((1 << 30) + 1, (1 << 31) - 1):
        assert csa.beam_workspace_bytes(1, 1, vocab, 1) == 0
        assert _beam(groups=1, beams=1, vocab=vocab, take=1, stride=vocab) == 2
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        assert _linear(dict(n=1, k=16), T=T) == 2


@pytest.mark.parametrize("gain", [0.0, float("inf"), float("nan"), 1e39, 1e-39])
def test_gains_without_a_reciprocal_refused(gain):
    with pytest.raises(ValueError):
        csa.Fp4Weights.encode(torch.ones(1, 16, dtype=torch.bfloat16), gain)


def test_no_layers_to_reorder_refused():
    with pytest.raises(ValueError):
        csa.kv_reorder(csa.KVCfg(4, 2, 64, csa.CACHE_FP4, 0, 0, csa.ROPE_HALF), [], 1, None, None)


def test_a_workspace_serves_smaller_calls():
    f, rng = csa.beam_workspace_bytes, np.random.default_rng(3)
    for _ in range(3000):
        a = [int(2 ** (rng.random() * m)) for m in (8, 6, 18, 6)]
        b = [int(rng.integers(1, v + 1)) if rng.random() < 0.7 else v for v in a]
        assert 0 < f(*b) <= f(*a), (b, a)


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("how", ["pack", "encode"])
def test_weights_are_laid_out_on_the_callers_stream(how, given, monkeypatch):
    """Memory, the largest weight and the kernel all on one stream: the given one, or the current."""
    import contextlib

    class Stream:
        cuda_stream = 7

    current, seen, mine = ["current"], [], Stream()
    want = mine if given else "current"

    @contextlib.contextmanager
    def on(stream):
        current.append(current[-1] if stream is None else stream)
        yield
        current.pop()

    class Lib:
        csa2_fp4_weight_bytes = csa.load().csa2_fp4_weight_bytes
        csa2_fp4_pack = csa2_fp4_encode = None

    def note(name, fn):
        def run(*args, **kw):
            seen.append((name, current[-1]))
            return fn(*args, **kw)
        return run

    def call(index, fn, stream, *args):
        seen.append(("kernel", current[-1] if stream is None else stream))
        return 0

    monkeypatch.setattr(csa, "load", lambda: Lib)
    monkeypatch.setattr(csa, "_on", call)
    monkeypatch.setattr(csa, "_plain", lambda t, *rest: None if t is None else t.data_ptr())
    monkeypatch.setattr(csa, "_rows_of", lambda t, width, name, index: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", note("memory", torch.empty))
    monkeypatch.setattr(torch.Tensor, "amax", note("largest", torch.Tensor.amax))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    s = mine if given else None
    if how == "pack":
        csa.Fp4Weights.pack(torch.zeros(16, 8, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.uint8), stream=s)
    else:
        csa.Fp4Weights.encode(torch.ones(16, 16, dtype=torch.bfloat16), stream=s)
    names = {name for name, _ in seen}
    assert names == ({"memory", "kernel"} if how == "pack" else {"memory", "kernel", "largest"})
    assert all(where is want for _, where in seen), seen


def test_packing_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        csa.Fp4Weights.pack(torch.zeros(16, 8, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.uint8))


@pytest.mark.parametrize("data,error", [(torch.zeros(9215, dtype=torch.uint8), ValueError), (torch.zeros(9216), TypeError),
                                        (torch.zeros(2, 9216, dtype=torch.uint8).t(), ValueError)])
def test_weights_over_memory_that_does_not_hold_them_refused(data, error):
    with pytest.raises(error):
        csa.Fp4Weights(data, 16, 64, 1.0)
    with pytest.raises(ValueError):
        csa.Fp4Weights(torch.zeros(9216, dtype=torch.uint8), 16, 72, 1.0)


@pytest.mark.parametrize("of", [[0, 1, 2], (0, 1, 2), b"\0\1\2", bytearray(b"\0\1\2"), np.array([0, 1, 2]),
                                np.array([0, 1, 2], np.int32), np.array([0, 1, 2], np.uint8), torch.tensor([0, 1, 2])])
def test_axes_of_pairs_may_be_any_sequence(of, monkeypatch):
    got = []
    monkeypatch.setattr(csa, "_kv_append", lambda *args: got.append(args[-1]))
    csa.kv_append_axes(None, None, None, None, None, None, None, of, None)
    assert got == [b"\0\1\2"]


@pytest.mark.parametrize("of", [3, [0, 256], [0, -1], [0.5]])
def test_axes_of_pairs_that_are_no_small_integers_refused(of):
    with pytest.raises((TypeError, ValueError)):
        csa.kv_append_axes(None, None, None, None, None, None, None, of, None)


LOG = """
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
static int __float_as_int(float x) { int i; std::memcpy(&i, &x, 4); return i; }
static float __int_as_float(int i) { float x; std::memcpy(&x, &i, 4); return x; }
%s
int main() {
  double most = 0, near = 0;
  for (int i = 0; i < 4000000; ++i) {
    const double at = 0.5 * std::pow(2.0, 32.0 * i / 4000000);
    const float h = (float)at, l = (float)(i %% 2 ? at - (double)h : h * std::ldexp(1.0, -26) * (i %% 5 - 2));
    const double d = std::fabs(log_of(h, l).exact() - (double)std::log((long double)h + l));
    if (d > most) most = d;
  }
  for (int i = 0; i < 200; ++i) {  // beside 1: relative to the little
    const float l = std::ldexp(1.0f + i %% 7 * 0.1f, -25 - i / 4);
    const double want = std::log1p((double)l), d = std::fabs(log_of(1.0f, l).exact() - want) / want;
    if (d > near) near = d;
  }
  std::printf("%%g %%g\\n", most, near);
}
"""


def test_logarithms_of_sums(tmp_path):
    """The join's logarithm, from its source, over what it says it takes, from 1/2 on, and of 1 and a little.  Its series
    from z^3 on is 0.0029 at most, doubled, with six roundings of 2^-24, and the last sums two of 2^-25 of 0.006: 2.4e-9,
    below 2^-28; beside 1 it is l / h, one division and its own square's half."""
    import os
    import subprocess

    text = open(os.path.join(os.path.dirname(csa.__file__), "csrc", "beam.cu")).read()
    code = text[text.index("struct Log {"):text.index("// fp64 -> unsigned in the same order")]
    (tmp_path / "log.cpp").write_text(LOG % code)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ffp-contract=off", str(tmp_path / "log.cpp"), "-o", str(tmp_path / "log")], check=True)
    most, near = (float(v) for v in subprocess.run([str(tmp_path / "log")], capture_output=True, text=True, check=True).stdout.split())
    assert most <= 2.0 ** -28 and near <= 2.0 ** -23, (most, near)
