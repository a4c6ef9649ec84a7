"""Cases of the operators around the paged key / value layers in one generation step: `fp4_linear` (projections with
4-bit weights in the caches' codec), `kv_append_axes` (new tokens whose rotary positions have several axes, as those of
images and video), `beam_select` (the best continuations over beams and vocabulary) and `kv_reorder` (the beams' cached
states put in the order of what was selected).

`run` computes each in a plain form, or through the package where `own` is set; `exact` gives the same from the
definitions in 64 bits.

Layout of a cache (64 tokens a page, token j of sequence b in page block_table[b][j // 64]):
  fp4   codes  [pages][kv heads][64][dim / 2]     two E2M1 codes a byte, even channel low
        scales [pages][kv heads][64][dim / 16]    one E4M3 scale per 16 channels
  bf16  values [pages][kv heads][dim / 8][64][8]
Weights: codes [n][k / 2] and scales [n][k / 16] alike, value = alpha * code * scale.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between neighbouring E2M1 magnitudes


# ------------------------------------------------------------------ cases --

def _linear(name, t, k, n, **kw):
    return dict(dict(name=name, op="linear", t=t, k=k, n=n, bias=False, out="bf16"), **kw)


def _append(name, **kw):
    return dict(dict(name=name, op="append", cache="fp4", batch=8, heads=64, kv_heads=8, dim=128, q_min=1, q_max=1,
                     ctx_min=0, ctx_max=0, rope_dims=128, rope_half=True, axes=3, woven=False), **kw)


def _beam(name, groups, beams, vocab, take, **kw):
    return dict(dict(name=name, op="beam", groups=groups, beams=beams, vocab=vocab, take=take, logits="bf16", done=0), **kw)


def _reorder(name, groups, beams, layers, **kw):
    return dict(dict(name=name, op="reorder", groups=groups, beams=beams, layers=layers, cache="fp4", kv_heads=8, dim=128,
                     len_min=100, len_max=600, alive=max(1, beams * 5 // 8)), **kw)


def listed():
    return [
        # one token's indexer queries from the low-rank ones: the smallest product
        _linear("linear_1_1280_to_4096", 1, 1280, 4096),
        # a small batch's attention queries, 64 heads of 512 from the low-rank ones
        _linear("linear_8_1280_to_32768", 8, 1280, 32768),
        # queries, keys and values of eight sequences' drafted blocks of five
        _linear("linear_40_4096_to_10240_bias", 40, 4096, 10240, bias=True),
        # logits of a serving step over a vocabulary of odd size
        _linear("logits_16_4096_to_128001", 16, 4096, 128001, out="fp32"),
        # a prompt's chunk through the same projection: the most operations
        _linear("linear_chunk_4096_to_10240", 4096, 4096, 10240),
        # one decode step of a batch that has seen images
        _append("append_axes_step_b8_fp4", ctx_min=32768, ctx_max=32768),
        # prompts with images of many lengths written in one call
        _append("append_axes_prompts_b8_fp4", q_min=37, q_max=2021),
        # one user's four beams
        _beam("beam_1x4_of_32000", 1, 4, 32000, 4),
        # a batch of transcriptions, some beams ended, scores not rounded to bf16
        _beam("beam_16x5_of_51865_fp32", 16, 5, 51865, 10, logits="fp32", done=1),
        # a serving batch over a large vocabulary, twice the beams kept for those that end
        _beam("beam_64x8_of_128001", 64, 8, 128001, 16, done=1),
        # one user's four beams go on
        _reorder("reorder_1x4_fp4", 1, 4, 12),
        # a serving batch's beams over all layers
        _reorder("reorder_16x8_bf16", 16, 8, 16, cache="bf16", kv_heads=4),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("linear", "linear", "append", "beam", "beam", "reorder"))
    if op == "linear":
        c = dict(op=op, k=16 * log(8, 1024), n=log(64, 131072), bias=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "fp32")))
        while c["k"] * c["n"] > 1 << 29:
            c["n"] = 1 + c["n"] // 2
        most = min(4096, (1 << 37) // (c["k"] * c["n"]))
        c["t"] = log(1, max(1, most)) if rng.random() < 0.6 else rng.choice((1, 2, 4, 8, 16))
        return c
    if op == "append":
        kv_heads = rng.choice((1, 2, 4, 5, 8))
        group = rng.choice((1, 2, 4, 7, 8, 16))
        heads, dim = kv_heads * min(group, 64 // kv_heads), rng.choice((64, 128))
        c = dict(op=op, cache=rng.choice(("fp4", "fp4", "bf16")), batch=log(1, 48), heads=heads, kv_heads=kv_heads, dim=dim,
                 rope_dims=rng.choice((dim // 2, dim)), rope_half=rng.random() < 0.5, axes=rng.choice((2, 3, 3, 4)),
                 woven=rng.random() < 0.5)
        c["q_max"] = log(1, 8192 // c["batch"])
        c["ctx_max"] = log(1, 32768)
        c["q_min"] = rng.choice((c["q_max"], 1 + c["q_max"] // 2, 1))
        c["ctx_min"] = rng.choice((c["ctx_max"], c["ctx_max"] // 2, 0))
        return c
    beams = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
    if op == "beam":
        vocab = log(100, 160000)
        c = dict(op=op, beams=beams, vocab=vocab, take=rng.choice((beams, 2 * beams)), logits=rng.choice(("bf16", "fp32")),
                 done=rng.choice((0, 0, beams // 3)))
        c["groups"] = log(1, max(1, min(256, 60000000 // (vocab * beams))))
        return c
    c = dict(op=op, beams=beams, layers=log(1, 32), cache=rng.choice(("fp4", "fp4", "bf16")), kv_heads=rng.choice((1, 2, 4, 8)),
             dim=rng.choice((64, 128)), len_max=log(1, 1200))
    c["len_min"] = rng.choice((c["len_max"], 1 + c["len_max"] // 2, 1))
    c["alive"] = rng.randint(1, beams)
    page = 2 * c["kv_heads"] * PAGE * _row_bytes(c) * c["layers"] * beams * (2 + c["len_max"] // PAGE)
    c["groups"] = log(1, max(1, min(128, (1 << 31) // page)))
    return c


def _spread(lo, hi, n, step):
    """n lengths spread over lo..hi, both ends among them: a case's own, whatever the seed."""
    x = [(i * step) % n for i in range(n)] if math.gcd(step, n) == 1 else list(range(n))
    return [hi - (hi - lo) * v // max(1, n - 1) for v in x]


def _lengths(c):
    """(append) New tokens and what was in the cache before them, for each sequence."""
    return _spread(c["q_min"], c["q_max"], c["batch"], 5), _spread(c["ctx_min"], c["ctx_max"], c["batch"], 7)


def _row_bytes(c):
    return c["dim"] // 2 + c["dim"] // 16 if c["cache"] == "fp4" else 2 * c["dim"]


def work(c):
    if c["op"] == "linear":
        out = 2 if c["out"] == "bf16" else 4
        return {"bytes": c["t"] * c["k"] * 2 + c["n"] * c["k"] * 9 // 16 + c["t"] * c["n"] * out + (2 * c["n"] if c["bias"] else 0),
                "flops": 2 * c["t"] * c["k"] * c["n"]}
    if c["op"] == "append":
        tokens = sum(_lengths(c)[0])
        rows = tokens * (c["heads"] + 2 * c["kv_heads"])
        stored = 2 * tokens * c["kv_heads"]
        # rows read, queries and stored values written, the pages, the angles and where they are
        return {"bytes": rows * c["dim"] * 4 + stored * _row_bytes(c) + tokens * 4 * (c["rope_dims"] + c["axes"]),
                "flops": 3 * rows * c["dim"]}
    if c["op"] == "beam":
        live = c["groups"] * (c["beams"] - c["done"])
        return {"bytes": live * c["vocab"] * (2 if c["logits"] == "bf16" else 4) + c["groups"] * (c["beams"] * 9 + c["take"] * 12),
                "flops": 4 * live * c["vocab"]}
    lens = _spread(c["len_min"], c["len_max"], c["groups"], 5)
    slots = sum(n % PAGE for n in lens) * (c["beams"] - c["alive"])
    entries = sum(n // PAGE for n in lens) * c["beams"]
    return {"bytes": 2 * slots * c["layers"] * 2 * c["kv_heads"] * _row_bytes(c) + 8 * entries + 8 * c["groups"] * c["beams"],
            "flops": 0}


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
    return {"linear": _prepare_linear, "append": _prepare_append, "beam": _prepare_beam, "reorder": _prepare_reorder}[c["op"]](c, g)


def _prepare_linear(c, g):
    t, k, n = c["t"], c["k"], c["n"]
    s = {"case": c, "alpha": 1.0 / (64 * math.sqrt(k))}
    s["codes"] = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(n, k // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // k)
    for i in range(0, n, step):  # weights of deviation 1 / sqrt(k), 64 sqrt(k) times as large where they are encoded
        w = torch.randn(min(step, n - i), k, generator=g, device="cuda") * 64
        s["codes"][i:i + step], s["scales"][i:i + step] = _encode(w)
    s["x"] = torch.randn(t, k, generator=g, device="cuda", dtype=torch.bfloat16)
    s["bias"] = torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16) if c["bias"] else None
    s["out"] = torch.empty(t, n, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")
    return s


def _axis_of(c):
    """Axis of each rotated pair: runs of pairs one after another, the first the shortest, or axes in turn."""
    pairs = c["rope_dims"] // 2
    if c["woven"]:
        return [i % c["axes"] for i in range(pairs)]
    first = pairs // (c["axes"] + 1)
    rest = pairs - first
    return [0 if i < first else 1 + (i - first) * (c["axes"] - 1) // rest for i in range(pairs)]


def _prepare_append(c, g):
    nq, ctx = _lengths(c)
    kv = [a + b for a, b in zip(nq, ctx)]
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
    s = {"case": c, "table": table, "cu": torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device="cuda"),
         "pos0": torch.tensor(ctx, dtype=torch.int64, device="cuda")}

    def rows(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    for name in ("k", "v"):  # pages as the tokens before left them
        if c["cache"] == "fp4":
            s[name + "_data"] = torch.randint(0, 256, (pages, hkv, PAGE, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
            s[name + "_scales"] = torch.randint(32, 64, (pages, hkv, PAGE, dim // 16), generator=g, device="cuda", dtype=torch.uint8)
        else:
            s[name + "_data"] = rows(pages, hkv, dim // 8, PAGE, 8)
    # one projection's rows hold a token's queries, keys and values side by side
    qkv = rows(tokens, c["heads"] + 2 * hkv, dim)
    s["q"], s["k"], s["v"] = qkv.split((c["heads"], hkv, hkv), dim=1)
    # text runs along all axes at once; every third stretch of 64 tokens is an image, whose tokens stand 8 to a row at one time
    n = max(kv)
    i = torch.arange(tokens, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:], i, right=True)
    p = (s["pos0"][b] + (i - s["cu"][b])).to(torch.int32)
    image = (p // 64) % 3 == 1
    at = p - p % 64
    images = (at, at + p % 64 // 8, at + p % 8, at + p % 4)
    s["axes"] = torch.stack([torch.where(image, images[a], p) for a in range(c["axes"])], 1).clamp_(max=n - 1).contiguous()
    half = c["rope_dims"] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * freq
    s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()
    s["axis_of"] = _axis_of(c)
    s["q_out"] = torch.empty(tokens, c["heads"], dim, dtype=torch.bfloat16, device="cuda")
    s["k_out"], s["v_out"] = (torch.empty(tokens, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    return s


def _prepare_beam(c, g):
    n, take = c["groups"] * c["beams"], c["take"]
    dtype = torch.bfloat16 if c["logits"] == "bf16" else torch.float32
    s = {"case": c, "logits": torch.empty(n, c["vocab"], dtype=dtype, device="cuda"), "end": c["vocab"] // 3}
    for i in range(0, n, 64):  # a few likely words, some that are not allowed
        x = torch.randn(min(64, n - i), c["vocab"], generator=g, device="cuda") * 3
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.01] = -math.inf
        s["logits"][i:i + 64] = x
    s["cum"] = -20 - torch.rand(c["groups"], c["beams"], generator=g, device="cuda") * 4
    s["done"] = None
    if c["done"]:
        who = torch.rand(c["groups"], c["beams"], generator=g, device="cuda").argsort(1)
        s["done"] = (who < c["done"]).to(torch.uint8)
    s["scores"] = torch.empty(c["groups"], take, dtype=torch.float32, device="cuda")
    s["parents"], s["tokens"] = (torch.empty(c["groups"], take, dtype=torch.int32, device="cuda") for _ in "pt")
    s["lse"] = torch.empty(n, dtype=torch.float32, device="cuda")
    return s


def _prepare_reorder(c, g):
    k, groups = c["beams"], c["groups"]
    lens = _spread(c["len_min"], c["len_max"], groups, 5)
    max_pages = max(lens) // PAGE + 1
    table, page = torch.empty(groups, k, max_pages, dtype=torch.int32), 0
    for i, n in enumerate(lens):
        shared = n // PAGE // 2  # pages of the prompt
        table[i, :, :shared] = torch.arange(page, page + shared, dtype=torch.int32)
        page += shared
        rest = k * (max_pages - shared)
        table[i, :, shared:] = torch.arange(page, page + rest, dtype=torch.int32).reshape(k, -1)
        page += rest
    order = torch.randperm(page, generator=g, device="cuda", dtype=torch.int32)
    s = {"case": c, "table": order[table.reshape(groups * k, max_pages).long().cuda()].contiguous(),
         "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda").repeat_interleave(k)}
    # `alive` beams go on, each once at least
    who = torch.rand(groups, k, generator=g, device="cuda").argsort(1)[:, : c["alive"]]
    more = torch.randint(0, c["alive"], (groups, k - c["alive"]), generator=g, device="cuda")
    local = torch.cat((who, who.gather(1, more)), 1)
    local = local.gather(1, torch.rand(groups, k, generator=g, device="cuda").argsort(1))
    s["parents"] = (local + k * torch.arange(groups, device="cuda")[:, None]).to(torch.int32).flatten().contiguous()
    s["layers"] = []
    for _ in range(c["layers"]):
        layer = {}
        for name in ("k", "v"):
            h, d = c["kv_heads"], c["dim"]
            if c["cache"] == "fp4":
                layer[name + "_data"] = torch.randint(0, 256, (page, h, PAGE, d // 2), generator=g, device="cuda", dtype=torch.uint8)
                layer[name + "_scales"] = torch.randint(32, 64, (page, h, PAGE, d // 16), generator=g, device="cuda", dtype=torch.uint8)
            else:
                layer[name + "_data"] = torch.randn(page, h, d // 8, PAGE, 8, generator=g, device="cuda", dtype=torch.bfloat16)
        s["layers"].append(layer)
    return s


# ------------------------------------------------------------ plain forms --

def _decode(codes, scales):
    """32-bit values of rows of codes."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e, m = ((c >> 1) & 3).float(), (c & 1).float()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    val = torch.where(c >= 8, -mag, mag)
    return val * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _linear_plain(s):
    y = torch.matmul(s["x"].float(), _decode(s["codes"], s["scales"]).t()) * s["alpha"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["out"].copy_(y)
    return s["out"]


def _rotate(x, cos, sin, dims, half):
    x = x.float()
    r, rest = x[..., :dims], x[..., dims:]
    a, b = (r[..., : dims // 2], r[..., dims // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    u, w = a * cos - b * sin, a * sin + b * cos
    return torch.cat((torch.cat((u, w), -1) if half else torch.stack((u, w), -1).flatten(-2), rest), -1)


def _append_plain(s):
    c, cu = s["case"], s["cu"]
    i = torch.arange(s["q"].shape[0], device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], i, right=True)
    pos = s["pos0"][b] + (i - cu[b])
    axis_of = torch.tensor(s["axis_of"], device=cu.device)
    turn = s["rope"][s["axes"].long()[:, axis_of], torch.arange(c["rope_dims"] // 2, device=cu.device)]
    cos, sin = (t.unsqueeze(1) for t in turn.unbind(-1))
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
            s[name + "_out"].copy_(_decode(codes, scales))
            out[name + "_scales"] = s[name + "_scales"]
        else:
            x = x.to(torch.bfloat16)
            data[page, :, :, slot] = x.reshape(*x.shape[:-1], c["dim"] // 8, 8)
            s[name + "_out"].copy_(x)
        out[name], out[name + "_data"] = s[name + "_out"], data
    return out


def _beam_plain(s):
    """In 64 bits from the exponentials on: continuations of different beams differ by less than 32 bits keep."""
    c = s["case"]
    groups, k, vocab, take = c["groups"], c["beams"], c["vocab"], c["take"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    lse = m[:, 0].double() + (x - m).double().exp().sum(1).log()
    # the best of each beam, the first of equal ones first
    best, token = torch.sort(x, dim=1, descending=True, stable=True)
    best, token = best[:, :take].double(), token[:, :take]
    if s["done"] is not None:
        done = s["done"].bool().flatten()
        lse = torch.where(done, torch.zeros_like(lse), lse)
        first = torch.arange(best.shape[1], device=x.device) == 0
        ended = torch.where(first, 0.0, -math.inf).double()
        best = torch.where(done[:, None], ended, best)
        token = torch.where(done[:, None], torch.full_like(token, s["end"]), token)
    score = (best + (s["cum"].double().flatten() - lse)[:, None]).reshape(groups, -1)
    width = best.shape[1]
    score, at = torch.sort(score, dim=1, descending=True, stable=True)
    score, at = score[:, :take], at[:, :take]
    n = score.shape[1]
    there = score > -math.inf
    parent = at // width + k * torch.arange(groups, device=x.device)[:, None]
    none = torch.full_like(at, -1)
    s["scores"].fill_(-math.inf)[:, :n] = score
    s["parents"].fill_(-1)[:, :n] = torch.where(there, parent, none)
    s["tokens"].fill_(-1)[:, :n] = torch.where(there, token.reshape(groups, -1).gather(1, at), none)
    s["lse"].copy_(lse)
    return {n: s[n] for n in ("scores", "parents", "tokens", "lse")}


def _reorder_plain(s):
    c = s["case"]
    groups, k, table = c["groups"], c["beams"], s["table"]
    dev = table.device
    seq = torch.arange(k, device=dev)
    parent = s["parents"].long().reshape(groups, k) - k * torch.arange(groups, device=dev)[:, None]
    child = parent[:, None, :] == seq[:, None]                              # [g][of beam][beam i]
    alive = child.any(2)
    stays = child.diagonal(dim1=1, dim2=2)                                  # a beam that goes on in its own place
    first = child.to(torch.uint8).argmax(2)
    keeper = torch.where(stays, seq, first)                                 # who keeps a beam's last page
    keeps = keeper.gather(1, parent) == seq
    n = k - c["alive"]
    extra = torch.sort(keeps.to(torch.uint8), dim=1, stable=True).indices[:, :n]            # the others, in order, and the beams that end
    dead = torch.sort(alive.to(torch.uint8), dim=1, stable=True).indices[:, :n]
    length = s["kv_len"].reshape(groups, k)[:, 0].long()
    full, rest = length // PAGE, length % PAGE
    rows = table.reshape(groups, k, -1)
    tail = rows.gather(2, full.clamp(max=rows.shape[2] - 1)[:, None, None].expand(groups, k, 1))[:, :, 0]
    src = tail.gather(1, parent.gather(1, extra)).long().flatten()
    dst = tail.gather(1, dead).long().flatten()
    keep = (torch.arange(PAGE, device=dev) < rest[:, None]).repeat_interleave(n, 0)
    for layer in s["layers"]:
        for data in layer.values():
            at = keep[:, None, :, None] if c["cache"] == "fp4" else keep[:, None, None, :, None]
            data[dst] = torch.where(at, data[src], data[dst])
    new_tail = tail.gather(1, parent).scatter(1, extra, tail.gather(1, dead))
    new_tail = torch.where(rest[:, None] > 0, new_tail, tail)
    col = torch.arange(rows.shape[2], device=dev)
    moved = rows.gather(1, parent[:, :, None].expand_as(rows))
    new = torch.where(col < full[:, None, None], moved, rows)
    new = torch.where(col == full[:, None, None], new_tail[:, :, None], new)
    table.copy_(new.reshape(table.shape))
    return {"table": table, "layers": s["layers"]}


# -------------------------------------------------------------- own calls --

def _own_handle(s):
    """Weights laid out, caches over the state's pages and workspaces, kept with the state as a program would."""
    import compressed_sparse_attention_07_gb300 as csa

    c = s["case"]
    if c["op"] == "linear":
        s["handle"] = csa, csa.Fp4Weights.pack(s["codes"], s["scales"], alpha=s["alpha"])
    elif c["op"] == "beam":
        n = csa.beam_workspace_bytes(c["groups"], c["beams"], c["vocab"], c["take"])
        s["handle"] = csa, torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    else:
        cfg = csa.KVCfg(n_heads=c.get("heads", c["kv_heads"]), kv_heads=c["kv_heads"], head_dim=c["dim"],
                        cache_dtype=csa.CACHE_FP4 if c["cache"] == "fp4" else csa.CACHE_BF16, rope_dims=c.get("rope_dims", 0),
                        rope_style=csa.ROPE_HALF if c.get("rope_half") else csa.ROPE_INTERLEAVED)
        layers = [s] if c["op"] == "append" else s["layers"]
        caches = [csa.KVCache.over(cfg, y["k_data"], y["v_data"], s["table"], y.get("k_scales"), y.get("v_scales")) for y in layers]
        s["handle"] = csa, cfg, caches
    return s["handle"]


def _run_own(s):
    csa, *kept = s.get("handle") or _own_handle(s)
    c = s["case"]
    if c["op"] == "linear":
        csa.fp4_linear(s["x"], kept[0], s["out"], bias=s["bias"])
        return s["out"]
    if c["op"] == "append":
        cfg, caches = kept
        csa.kv_append_axes(cfg, s["k"], s["v"], s["cu"], s["pos0"], caches[0], s["axes"], s["axis_of"], s["rope"], q=s["q"],
                           q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])
        names = ("k_scales", "k_data", "v_scales", "v_data") if c["cache"] == "fp4" else ("k_data", "v_data")
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], **{n: s[n] for n in names}}
    if c["op"] == "beam":
        csa.beam_select(s["logits"], s["cum"], s["scores"], s["parents"], s["tokens"], kept[0], done=s["done"],
                        end_token=s["end"], lse=s["lse"])
        return {n: s[n] for n in ("scores", "parents", "tokens", "lse")}
    cfg, caches = kept
    csa.kv_reorder(cfg, caches, c["beams"], s["parents"], s["kv_len"])
    return {"table": s["table"], "layers": s["layers"]}


def run(state):
    if own:
        return _run_own(state)
    return {"linear": _linear_plain, "append": _append_plain, "beam": _beam_plain, "reorder": _reorder_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --

def exact(c, seed):
    if c["op"] == "linear" and 2 * c["t"] * c["k"] * c["n"] > 5e12:
        return None
    s = prepare(c, seed)
    return {"linear": _linear_exact, "append": _append_exact, "beam": _beam_exact, "reorder": _reorder_exact}[c["op"]](c, s)


def _linear_exact(c, s):
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    x, k = s["x"].double(), c["k"]
    out = torch.empty(c["t"], c["n"], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // k)
    for i in range(0, c["n"], step):
        codes = s["codes"][i:i + step].long()
        w = torch.empty(codes.shape[0], k, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = e2m1[codes % 16], e2m1[codes // 16]
        f = s["scales"][i:i + step].view(torch.float8_e4m3fn).double().unsqueeze(-1)
        out[:, i:i + step] = x @ (w.reshape(-1, k // 16, 16) * f).reshape(-1, k).T
    out *= s["alpha"]
    return out if s["bias"] is None else out + s["bias"].double()


def _append_exact(c, s):
    """The rotated queries, and the keys and values of a bf16 cache, before their rounding. What FP4 keeps of a row is a
    choice of codes: no 64-bit value stands for it."""
    half, table = c["rope_dims"] // 2, s["rope"].double()
    turn = torch.empty(s["q"].shape[0], half, dtype=torch.complex128, device="cuda")
    for pair, axis in enumerate(s["axis_of"]):
        turn[:, pair] = torch.view_as_complex(table[:, pair].contiguous())[s["axes"][:, axis].long()]
    turn = turn.unsqueeze(1)

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


def _beam_exact(c, s):
    k, vocab, take = c["beams"], c["vocab"], c["take"]
    out = {"scores": torch.full((c["groups"], take), -math.inf, dtype=torch.float64, device="cuda"),
           "parents": torch.full((c["groups"], take), -1, device="cuda"), "tokens": torch.full((c["groups"], take), -1, device="cuda"),
           "lse": torch.zeros(c["groups"] * k, dtype=torch.float64, device="cuda")}
    done = None if s["done"] is None else s["done"].tolist()
    for g in range(c["groups"]):
        all_ = torch.full((k, vocab), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(k):
            if done and done[g][b]:
                all_[b, s["end"]] = s["cum"][g, b]
                continue
            x = s["logits"][g * k + b].double()
            out["lse"][g * k + b] = z = torch.logsumexp(x, 0)
            all_[b] = x - z + s["cum"][g, b].double()
        flat = all_.flatten()
        # everything that reaches the last place, then the order of score, beam and token
        least = torch.topk(flat, min(take, flat.numel())).values[-1]
        at = torch.nonzero((flat >= least) & (flat > -math.inf)).flatten().tolist()
        at = sorted(zip((-flat[at]).tolist(), at))[:take]
        for i, (score, j) in enumerate(at):
            out["scores"][g, i], out["parents"][g, i], out["tokens"][g, i] = -score, g * k + j // vocab, j % vocab
    return out


def _reorder_exact(c, s):
    """One beam after another, by the rule: who goes on in its place, or else the first child, keeps the last page; the
    other children take the last pages of beams without children, in order."""
    k, table, parents, lens = c["beams"], s["table"].tolist(), s["parents"].tolist(), s["kv_len"].tolist()
    new, copies = [list(r) for r in table], []
    for g in range(c["groups"]):
        mine = range(g * k, g * k + k)
        full, rest = divmod(lens[g * k], PAGE)
        kept = {}
        for i in mine:
            if parents[i] not in kept or parents[i] == i:
                kept[parents[i]] = i
        free = iter([i for i in mine if i not in kept])
        for i in mine:
            new[i][:full] = table[parents[i]][:full]
            if kept[parents[i]] != i:
                page = next(free)
                if rest:
                    new[i][full] = table[page][full]
                    copies.append((table[parents[i]][full], table[page][full], rest))
            elif rest:
                new[i][full] = table[parents[i]][full]
    for layer in s["layers"]:
        for data in layer.values():
            for a, b, n in copies:
                if c["cache"] == "fp4":
                    data[b, :, :n] = data[a, :, :n]
                else:
                    data[b, :, :, :n] = data[a, :, :, :n]
    return {"table": torch.tensor(new, dtype=torch.int32, device="cuda"), "layers": s["layers"]}
