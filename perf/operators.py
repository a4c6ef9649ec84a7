"""Cases of the paged key / value operators: `kv_append` (new keys and values rotated, encoded and written to
their pages, queries rotated beside them), `kv_attend` (causal attention over such a cache, one new token or
many per sequence) and `kv_cross_attend` (the same without a causal mask, over an encoder's states).

`run` computes each in a plain form, or through the package where `own` is set; `exact` gives the same from the
definitions in 64 bits.

Layout of a cache (64 tokens a page, token j of sequence b in page block_table[b][j // 64]):
  fp4   codes  [pages][kv heads][64][dim / 2]     two E2M1 codes a byte, even channel low
        scales [pages][kv heads][64][dim / 16]    one E4M3 scale per 16 channels
  bf16  values [pages][kv heads][dim / 8][64][8]
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between neighbouring E2M1 magnitudes


# ------------------------------------------------------------------ cases --

def _case(name, op, **kw):
    c = dict(name=name, op=op, cache="fp4", batch=1, heads=64, kv_heads=8, dim=128, q_min=1, q_max=1, ctx_min=0,
             ctx_max=0, window=0, rope_dims=64, rope_half=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a small batch: the smallest call, all latency
        _case("append_step_b8_fp4", "append", batch=8, ctx_min=32768, ctx_max=32768),
        # prompts of many lengths written in one call
        _case("append_prompts_b8_fp4", "append", batch=8, q_min=37, q_max=2021, rope_dims=128, rope_half=True),
        # a prompt chunk of a smaller model into a cache that is not quantised
        _case("append_chunk_4096_bf16", "append", cache="bf16", heads=32, kv_heads=4, dim=64, q_min=4096, q_max=4096,
              ctx_min=16384, ctx_max=16384),
        # one user's chat: a token at a time on a few thousand
        _case("decode_b1_ctx4095_fp4", "attend", ctx_min=4095, ctx_max=4095),
        # a serving batch of long contexts: the cache's bytes decide
        _case("decode_b32_ctx32768_fp4", "attend", batch=32, ctx_min=32767, ctx_max=32767),
        # a serving batch of every length, seven query heads to a key head, not quantised
        _case("decode_b48_ragged_bf16", "attend", cache="bf16", batch=48, heads=28, kv_heads=4, dim=64, ctx_max=16383),
        # a drafted block of five positions verified at once
        _case("draft5_b8_ctx32768_fp4", "attend", batch=8, q_min=5, q_max=5, ctx_min=32763, ctx_max=32763),
        # a prompt's chunk on what came before it: the largest
        _case("chunk_2048_on_16384_fp4", "attend", q_min=2048, q_max=2048, ctx_min=16384, ctx_max=16384),
        # whole prompts of many lengths under a sliding window
        _case("prompts_b4_window128_bf16", "attend", cache="bf16", batch=4, heads=16, kv_heads=4, q_min=501, q_max=4096,
              window=128),
        # a decoder's step over its encoder's states, every head its own keys
        _case("cross_step_b16_enc1500_bf16", "cross", cache="bf16", batch=16, heads=16, kv_heads=16, dim=64,
              ctx_min=1211, ctx_max=1500),
        # a decoder's prompts over encoder states of other lengths
        _case("cross_prompts_b8_enc1500_fp4", "cross", batch=8, heads=28, kv_heads=4, q_min=65, q_max=448, ctx_min=700,
              ctx_max=1501),
        # many short texts, some without any encoder state
        _case("cross_short_b64_fp4", "cross", batch=64, heads=16, kv_heads=2, dim=64, q_max=33, ctx_max=77),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "attend", "attend", "cross"))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 4, 7, 8, 16))
    heads, dim = kv_heads * min(group, 64 // kv_heads), rng.choice((64, 128))
    c = dict(op=op, cache=rng.choice(("fp4", "fp4", "bf16")), batch=log(1, 48), heads=heads, kv_heads=kv_heads, dim=dim,
             window=0, rope_dims=rng.choice((dim // 2, dim)), rope_half=rng.random() < 0.5)
    if op == "append":
        c["q_max"] = log(1, 8192 // c["batch"])
        c["ctx_max"] = log(1, 32768)
    elif rng.random() < 0.5:  # single tokens and short drafts
        c["q_max"] = rng.choice((1, 1, 2, 4, 5, 7))
        c["ctx_max"] = log(1, min(32768, 500000 // c["batch"]))
    else:
        c["q_max"] = log(8, max(8, 4096 // c["batch"]))
        c["ctx_max"] = log(1, min(16384, (1 << 23) // (c["q_max"] * c["batch"])))
    c["q_min"] = rng.choice((c["q_max"], 1 + c["q_max"] // 2, 1))
    c["ctx_min"] = rng.choice((c["ctx_max"], c["ctx_max"] // 2, 0))
    if op == "attend" and rng.random() < 0.25:
        c["window"] = rng.choice((1, 100, 128, 1024))
    return c


def _spread(lo, hi, n, step):
    """n lengths spread over lo..hi, both ends among them: a case's own, whatever the seed."""
    x = [(i * step) % n for i in range(n)] if math.gcd(step, n) == 1 else list(range(n))
    return [hi - (hi - lo) * v // max(1, n - 1) for v in x]


def _lengths(c):
    """New tokens (or decoder rows) and what was in the cache before them, for each sequence."""
    return _spread(c["q_min"], c["q_max"], c["batch"], 5), _spread(c["ctx_min"], c["ctx_max"], c["batch"], 7)


def _kv_lengths(c):
    nq, ctx = _lengths(c)
    return ctx if c["op"] == "cross" else [a + b for a, b in zip(nq, ctx)]


def _seen(c):
    """Pairs of a query and a key that it sees, over all sequences."""
    n = 0
    for q, kv in zip(_lengths(c)[0], _kv_lengths(c)):
        if c["op"] == "cross":
            n += q * kv
        elif c["window"]:
            n += sum(min(c["window"], kv - q + i + 1) for i in range(q))
        else:
            n += q * (kv - q) + q * (q + 1) // 2
    return n


def _row_bytes(c):
    return c["dim"] // 2 + c["dim"] // 16 if c["cache"] == "fp4" else 2 * c["dim"]


def work(c):
    nq, ctx = _lengths(c)
    tokens, kv = sum(nq), _kv_lengths(c)
    if c["op"] == "append":
        rows = tokens * (c["heads"] + 2 * c["kv_heads"])
        stored = 2 * tokens * c["kv_heads"]
        # rows read, queries and stored values written, the pages, the table of angles
        return {"bytes": rows * c["dim"] * 4 + stored * _row_bytes(c) + tokens * c["rope_dims"] * 4,
                "flops": 3 * rows * c["dim"]}
    keys = sum(min(n, c["window"] + q - 1) if c["window"] else n for n, q in zip(kv, nq))
    return {"bytes": 2 * keys * c["kv_heads"] * _row_bytes(c) + tokens * c["heads"] * (4 * c["dim"] + 4),
            "flops": 4 * _seen(c) * c["heads"] * c["dim"]}


# ----------------------------------------------------------------- inputs --

def _encode(x):
    """FP4 codes and scales of rows: scale = E4M3 nearest to amax / 6, code = E2M1 nearest to x / scale (ties to the
    even code, no negative zero)."""
    n = x.shape[-1]
    g = x.reshape(*x.shape[:-1], n // 16, 16)
    amax = g.abs().amax(-1)
    scale = torch.clamp(amax / torch.full_like(amax, 6.0), max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = g.abs()
    m = torch.zeros_like(g, dtype=torch.uint8)
    for k, mid in enumerate(MIDS):
        t = s * mid
        m += (a >= t) if k & 1 else (a > t)
    m = torch.where(s > 0, m, torch.zeros_like(m))
    m = torch.where((g < 0) & (m > 0), m | 8, m).reshape(x.shape)
    return m[..., 0::2] | (m[..., 1::2] << 4), scale.view(torch.uint8)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, ctx = _lengths(c)
    kv = _kv_lengths(c)
    tokens, hkv, dim = sum(nq), c["kv_heads"], c["dim"]
    max_pages = max(1, -(-max(kv) // PAGE))
    per = [-(-n // PAGE) for n in kv]
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    first = torch.tensor([0] + list(np.cumsum(per)), device="cuda")
    at = torch.arange(max_pages, device="cuda")
    lens = torch.tensor(per, device="cuda")
    table = order[torch.clamp(first[:-1, None] + at, max=pages - 1)]
    table = torch.where(at < lens[:, None], table, torch.zeros_like(table)).contiguous()
    s = {"case": c, "table": table, "max_q": max(nq), "max_kv": max(kv),
         "cu": torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"),
         "pos0": torch.tensor(ctx, dtype=torch.int64, device="cuda")}

    def rows(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    for name in ("k", "v"):
        if c["op"] == "append":  # pages as the tokens before left them
            if c["cache"] == "fp4":
                s[name + "_data"] = torch.randint(0, 256, (pages, hkv, PAGE, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
                s[name + "_scales"] = torch.randint(32, 64, (pages, hkv, PAGE, dim // 16), generator=g, device="cuda", dtype=torch.uint8)
            else:
                s[name + "_data"] = rows(pages, hkv, dim // 8, PAGE, 8)
        elif c["cache"] == "fp4":
            s[name + "_data"], s[name + "_scales"] = _encode(rows(pages, hkv, PAGE, dim).float())
        else:
            s[name + "_data"] = rows(pages, hkv, dim // 8, PAGE, 8)
    if c["op"] == "append":
        # one projection's rows hold a token's queries, keys and values side by side
        qkv = rows(tokens, c["heads"] + 2 * hkv, dim)
        s["q"], s["k"], s["v"] = qkv.split((c["heads"], hkv, hkv), dim=1)
        n = max(kv)
        half = c["rope_dims"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()
        s["q_out"] = torch.empty(tokens, c["heads"], dim, dtype=torch.bfloat16, device="cuda")
        s["k_out"], s["v_out"] = (torch.empty(tokens, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    else:
        s["q"] = rows(tokens, c["heads"], dim)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(tokens, c["heads"], dtype=torch.float32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(dim)
    return s


# ------------------------------------------------------------ plain forms --

def _decode(data, scales, dim):
    """Rows of 32-bit values of the pages of a cache."""
    if scales is None:  # [..., dim / 8, 64, 8] -> [..., 64, dim]
        return data.transpose(-3, -2).reshape(*data.shape[:-3], PAGE, dim).float()
    codes = torch.stack((data & 15, data >> 4), -1).reshape(*data.shape[:-1], dim)
    e, m = ((codes >> 1) & 3).float(), (codes & 1).float()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    val = torch.where(codes >= 8, -mag, mag)
    return val * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _rotate(x, cos, sin, dims, half):
    x = x.float()
    r, rest = x[..., :dims], x[..., dims:]
    a, b = (r[..., : dims // 2], r[..., dims // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    u, w = a * cos - b * sin, a * sin + b * cos
    return torch.cat((torch.cat((u, w), -1) if half else torch.stack((u, w), -1).flatten(-2), rest), -1)


def _token_places(s):
    """Sequence and position of each new token."""
    cu, n = s["cu"], s["q"].shape[0]
    i = torch.arange(n, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], i, right=True)
    return b, s["pos0"][b] + (i - cu[b])


def _append_plain(s):
    c = s["case"]
    b, pos = _token_places(s)
    cos, sin = (t.unsqueeze(1) for t in s["rope"][pos].unbind(-1))
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rope_dims"], c["rope_half"]))
    page, slot = s["table"][b, pos // PAGE].long(), pos % PAGE
    out = {"q": s["q_out"]}
    for name in ("k", "v"):
        x = _rotate(s["k"], cos, sin, c["rope_dims"], c["rope_half"]) if name == "k" else s["v"].float()
        data = s[name + "_data"]
        if c["cache"] == "fp4":
            codes, scales = _encode(x)
            data[page, :, slot] = codes
            s[name + "_scales"][page, :, slot] = scales
            s[name + "_out"].copy_(_decode(codes, scales, c["dim"]))
            out[name + "_scales"] = s[name + "_scales"]
        else:
            x = x.to(torch.bfloat16)
            data[page, :, :, slot] = x.reshape(*x.shape[:-1], c["dim"] // 8, 8)
            s[name + "_out"].copy_(x)
        out[name], out[name + "_data"] = s[name + "_out"], data
    return out


def _attend_plain(s):
    c, cu = s["case"], s["cu"]
    b, hkv, dim, group = c["batch"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    nq, mq = cu[1:] - cu[:-1], s["max_q"]
    i = torch.arange(mq, device=cu.device)
    there = i < nq[:, None]                                            # [b][mq]
    token = torch.where(there, cu[:-1, None] + i, torch.zeros_like(i)).long()
    q = s["q"][token].float().reshape(b, mq, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(b, hkv, mq * group, dim)
    table = s["table"].long()
    k, v = (_decode(s[n + "_data"][table], s[n + "_scales"][table] if c["cache"] == "fp4" else None, dim)
            .transpose(1, 2).reshape(b, hkv, -1, dim) for n in ("k", "v"))
    j = torch.arange(k.shape[2], device=cu.device)
    see = (j < s["kv_len"][:, None])[:, None].expand(b, mq, -1)        # [b][mq][keys]
    if c["op"] == "attend":
        pos = (s["kv_len"] - nq)[:, None, None] + i[:, None]
        see = see & (j <= pos)
        if c["window"]:
            see = see & (j > pos - c["window"])
    see = see[:, None, :, None].expand(b, 1, mq, group, -1).reshape(b, 1, mq * group, -1)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = x.masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    some = m > -math.inf
    m = torch.where(some, m, torch.zeros_like(m))
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(some, l, torch.ones_like(l))
    lse = torch.where(some, m + l.log(), torch.full_like(m, -math.inf))
    o, lse = (t.reshape(b, hkv, mq, group, -1).permute(0, 2, 1, 3, 4).reshape(b, mq, c["heads"], -1) for t in (o, lse))
    at = _rows_of(s)
    s["out"].copy_(o.reshape(b * mq, c["heads"], dim)[at])
    s["lse"].copy_(lse.reshape(b * mq, c["heads"])[at])
    return {"out": s["out"], "lse": s["lse"]}


def _rows_of(s):
    """Where each query token stands in an array of max_q rows for each sequence."""
    cu = s["cu"]
    n = torch.arange(s["q"].shape[0], device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], n, right=True)
    return b * s["max_q"] + (n - cu[b])


# -------------------------------------------------------------- own calls --

def _own_handle(s):
    """The configuration, the cache over the state's pages and the workspace, kept with the state as a program would."""
    import compressed_sparse_attention_07_gb300 as csa

    c = s["case"]
    cfg = csa.KVCfg(n_heads=c["heads"], kv_heads=c["kv_heads"], head_dim=c["dim"],
                    cache_dtype=csa.CACHE_FP4 if c["cache"] == "fp4" else csa.CACHE_BF16, window=c["window"],
                    rope_dims=c["rope_dims"], rope_style=csa.ROPE_HALF if c["rope_half"] else csa.ROPE_INTERLEAVED)
    cache = csa.KVCache.over(cfg, s["k_data"], s["v_data"], s["table"], s.get("k_scales"), s.get("v_scales"))
    ws = None
    if c["op"] != "append":
        n = csa.kv_workspace_bytes(cfg, c["batch"], s["q"].shape[0], s["max_q"], s["max_kv"])
        ws = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    s["handle"] = csa, cfg, cache, ws
    return s["handle"]


def _run_own(s):
    csa, cfg, cache, ws = s.get("handle") or _own_handle(s)
    c = s["case"]
    if c["op"] == "append":
        csa.kv_append(cfg, s["k"], s["v"], s["cu"], s["pos0"], cache, rope=s["rope"], q=s["q"], q_out=s["q_out"],
                      k_out=s["k_out"], v_out=s["v_out"])
        names = ("k_scales", "k_data", "v_scales", "v_data") if c["cache"] == "fp4" else ("k_data", "v_data")
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], **{n: s[n] for n in names}}
    attend = csa.kv_cross_attend if c["op"] == "cross" else csa.kv_attend
    attend(cfg, s["q"], s["cu"], cache, s["kv_len"], s["max_q"], s["max_kv"], s["out"], lse=s["lse"], scale=s["scale"],
           workspace=ws)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return _append_plain(state) if state["case"]["op"] == "append" else _attend_plain(state)


# ------------------------------------------------------------------ exact --

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        return _append_exact(c, s)
    if 4 * _seen(c) * c["heads"] * c["dim"] > 1e13:
        return None
    nq, kv = _lengths(c)[0], _kv_lengths(c)
    group, dim = c["heads"] // c["kv_heads"], c["dim"]
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    out = torch.zeros(sum(nq), c["heads"], dim, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(nq), c["heads"]), -math.inf, dtype=torch.float64, device="cuda")

    def states(name, b, h):
        ids = s["table"][b, : -(-kv[b] // PAGE)].long()
        d = s[name + "_data"][ids, h]
        if c["cache"] != "fp4":
            return d.double().permute(0, 2, 1, 3).reshape(-1, dim)[: kv[b]]
        d = d.reshape(-1, dim // 2)[: kv[b]].long()
        f = s[name + "_scales"][ids, h].view(torch.float8_e4m3fn).double().reshape(-1, dim // 16, 1)[: kv[b]]
        x = torch.empty(kv[b], dim, dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = e2m1[d % 16], e2m1[d // 16]
        return (x.reshape(-1, dim // 16, 16) * f).reshape(-1, dim)

    t0 = 0
    for b in range(c["batch"]):
        t1 = t0 + nq[b]
        if kv[b]:
            for h in range(c["kv_heads"]):
                k, v = states("k", b, h), states("v", b, h)
                at = torch.arange(kv[b] - nq[b], kv[b], device="cuda")[:, None] - torch.arange(kv[b], device="cuda")
                hide = torch.zeros_like(at, dtype=torch.bool) if c["op"] == "cross" else at < 0
                if c["window"]:
                    hide |= at >= c["window"]
                for i in range(h * group, (h + 1) * group):
                    x = (s["q"][t0:t1, i].double() @ k.T) * s["scale"]
                    x[hide] = -math.inf
                    z = torch.logsumexp(x, 1, keepdim=True)
                    out[t0:t1, i], lse[t0:t1, i] = torch.exp(x - z) @ v, z[:, 0]
        t0 = t1
    return {"out": out, "lse": lse}


def _append_exact(c, s):
    """The rotated queries, and the keys and values of a bf16 cache, before their rounding. What FP4 keeps of a row is a
    choice of codes: no 64-bit value stands for it."""
    nq, ctx = _lengths(c)
    pos = np.concatenate([np.arange(n) + p for n, p in zip(nq, ctx)])
    half = c["rope_dims"] // 2
    table = s["rope"].double()[torch.from_numpy(pos).cuda()]
    turn = torch.complex(table[..., 0], table[..., 1]).unsqueeze(1)

    def rotated(x):
        x = x.double().clone()
        r = x[..., : 2 * half]
        pair = torch.complex(r[..., :half], r[..., half:]) if c["rope_half"] else torch.view_as_complex(r.reshape(*r.shape[:-1], half, 2))
        z = pair * turn
        x[..., : 2 * half] = torch.cat((z.real, z.imag), -1) if c["rope_half"] else torch.view_as_real(z).reshape(r.shape)
        return x

    out = {"q": rotated(s["q"]), "k": None, "v": None, "k_data": None, "v_data": None}
    if c["cache"] == "fp4":
        return {**out, "k_scales": None, "v_scales": None}
    return {**out, "k": rotated(s["k"]), "v": s["v"].double()}
