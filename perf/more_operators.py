"""Cases, plain forms and exact values of the operators that append to the paged cache with the position rotation on
the way, and of attention over a cache with one scale for each page and head.

Three operators, each with its plain form (elementary torch operations in 32 bits) and the call a user makes of the
library (``own``):

* ``append``  queries and keys are rotated to their positions; keys and values are quantized into the pages of each
              sequence's last tokens.  The block-scaled kinds keep a scale per 32 elements; ``fp8_e4m3_page`` keeps one
              power of two for each page of 16 tokens, K or V, and head, and rescales a page that outgrows its own
* ``decode``  one new token per sequence attends over a cache of ``fp8_e4m3_page``
* ``extend``  the last n tokens of each sequence attend causally over such a cache
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"
LOW, HIGH = -32, 32  # exponents of a page's scale
# (query heads, kv heads, K width, V width, latent row)
HEADS = {"tiny": (8, 2, 128, 128, False), "qwen3_1p7b": (16, 8, 128, 128, False), "long_gqa": (16, 2, 256, 256, False),
         "serving": (32, 8, 128, 128, False), "mla": (128, 1, 576, 512, True),
         # narrow heads, every head its own keys, one key head for all, an odd number of query heads per key head
         "narrow": (32, 8, 64, 64, False), "own_keys": (6, 6, 64, 64, False), "one_key": (8, 1, 128, 128, False),
         "fives": (10, 2, 128, 128, False)}
KINDS = ("fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled", "fp8_e4m3_page")


def listed():
    return [
        # one chat's next token: the call's own latency
        dict(name="append_one_chat", op="append", heads="serving", kind="fp8_e4m3", batch=1, ctx_lo=1003, ctx_hi=1003, n_lo=1,
             n_hi=1, part=1.0, pairs=False, slices=False, shape=1),
        # a serving batch's next tokens, from slices of one projection
        dict(name="append_serving", op="append", heads="qwen3_1p7b", kind="q8_0", batch=64, ctx_lo=200, ctx_hi=8192, n_lo=1,
             n_hi=1, part=1.0, pairs=False, slices=True, shape=2),
        # a prefill batch of ragged prompts over the latent row: its last 64 elements are rotated, neighbours paired
        dict(name="append_latent_prompts", op="append", heads="mla", kind="fp8_e4m3", batch=4, ctx_lo=0, ctx_hi=0, n_lo=400,
             n_hi=2048, part=1.0, pairs=True, slices=False, shape=3),
        # next tokens into pages that other tokens share a scale with
        dict(name="append_page_serving", op="append", heads="serving", kind="fp8_e4m3_page", batch=64, ctx_lo=200,
             ctx_hi=8192, n_lo=1, n_hi=1, part=1.0, pairs=False, slices=True, shape=4),
        # ragged prompts that go on from a stored one, into pages with a scale each
        dict(name="append_page_prompts", op="append", heads="serving", kind="fp8_e4m3_page", batch=8, ctx_lo=5, ctx_hi=900,
             n_lo=500, n_hi=4096, part=0.5, pairs=False, slices=False, shape=5),
        # one chat over a short context: latency
        dict(name="decode_one_chat", op="decode", heads="tiny", batch=1, ctx_lo=505, ctx_hi=505, shape=6),
        # a serving batch of ragged contexts
        dict(name="decode_serving", op="decode", heads="serving", batch=64, ctx_lo=256, ctx_hi=16384, shape=7),
        # long documents, eight query heads to a key head
        dict(name="decode_long", op="decode", heads="long_gqa", batch=4, ctx_lo=131072, ctx_hi=131072, shape=8),
        # one chat's next turn of some words
        dict(name="extend_one_chat", op="extend", heads="tiny", batch=1, ctx_lo=480, ctx_hi=480, n_lo=25, n_hi=25, shape=9),
        # turns of several chats over ragged contexts
        dict(name="extend_serving", op="extend", heads="qwen3_1p7b", batch=8, ctx_lo=700, ctx_hi=8192, n_lo=100, n_hi=1024,
             shape=10),
        # narrow heads
        dict(name="extend_narrow", op="extend", heads="narrow", batch=4, ctx_lo=300, ctx_hi=2048, n_lo=600, n_hi=2048,
             shape=11),
        # a chunk of a long document
        dict(name="extend_long", op="extend", heads="serving", batch=1, ctx_lo=30000, ctx_hi=30000, n_lo=2048, n_hi=2048,
             shape=12),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "decode", "extend"))
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        c = dict(op=op, shape=rng.randrange(1 << 30), batch=_spread(rng, 1, 64))
        c["heads"] = rng.choice([h for h in HEADS if op == "append" or h != "mla"])
        c["ctx_hi"] = _spread(rng, 1, 65536 if op == "decode" else 16384)
        c["ctx_lo"] = max(1, int(c["ctx_hi"] * rng.uniform(0.1, 1.0)))
        if op != "decode":
            c["n_hi"] = _spread(rng, 1, 4096)
            c["n_lo"] = max(1, int(c["n_hi"] * rng.uniform(0.1, 1.0)))
        if op == "append":
            c["kind"] = rng.choice([k for k in KINDS if c["heads"] != "mla" or k != "fp8_e4m3_page"])
            c["part"] = rng.choice((1.0, 0.5))
            c["pairs"] = rng.random() < 0.5
            c["slices"] = rng.random() < 0.5
            if rng.random() < 0.3:  # fresh sequences
                c["ctx_lo"] = c["ctx_hi"] = 0
        if _room(c) <= 1.2e10 and _cost(c) <= most:
            return c


# ---------------------------------------------------------------------------------------------- shapes
def _ints(case, what, lo, hi, count):
    r = random.Random("%d %s" % (case["shape"], what))
    return [r.randint(lo, hi) for _ in range(count)]


def _lens(case):
    """Stored tokens before the call's and the call's own tokens of each sequence (a decode's own token is stored)."""
    ctx = _ints(case, "ctx", case["ctx_lo"], case["ctx_hi"], case["batch"])
    if case["op"] == "decode":
        return ctx, [0] * case["batch"]
    return ctx, _ints(case, "n", case["n_lo"], case["n_hi"], case["batch"])


def _pages(tokens):
    return -(-tokens // PAGE)


def _rot(case):
    """First rotated element of a row, and how many."""
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    return (dv, d - dv) if mla else (0, int(d * case["part"]))


def _cost(case):
    """About a plain pass's time: padded to the longest sequence."""
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    ctx, n = _lens(case)
    if case["op"] == "append":
        return float(sum(n)) * (hq + 2 * hkv) * d
    longest = max(c + m for c, m in zip(ctx, n))
    if case["op"] == "decode":
        return float(case["batch"]) * longest * hkv * d
    return float(case["batch"]) * max(n) * longest * hq * d


def _room(case):
    """About the plain pass's largest arrays, in numbers."""
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    ctx, n = _lens(case)
    longest = max(c + m for c, m in zip(ctx, n))
    most = float(case["batch"]) * longest * 2 * hkv * d
    return most if case["op"] != "extend" else max(most, float(case["batch"]) * max(n) * longest * hq)


def work(case):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    ctx, n = _lens(case)
    nkv = 1 if mla else 2
    if case["op"] == "append":
        t = sum(n)
        first, rot = _rot(case)
        code = nkv * hkv * d * (17 / 16 if case["kind"] in ("fp8_e4m3", "q8_0") else 1)
        b = t * (2 * hq + nkv * hkv) * d * 2 + t * code + len(set().union(*(range(c, c + m) for c, m in zip(ctx, n)))) * rot * 4
        b += sum(_pages(c + m) - c // PAGE for c, m in zip(ctx, n)) * (4 + (8 * nkv * hkv if "page" in case["kind"] else 0))
        return {"bytes": b, "flops": t * (hq + hkv) * rot * 3.0}
    kv = sum(c + m for c, m in zip(ctx, n)) * 2 * hkv * d
    pages = sum(_pages(c + m) for c, m in zip(ctx, n))
    if case["op"] == "decode":
        return {"bytes": kv + pages * (4 + 8 * hkv) + case["batch"] * hq * d * 4, "flops": 4.0 * hq * d * sum(ctx)}
    return {"bytes": kv + pages * (4 + 8 * hkv) + sum(n) * hq * d * 4,
            "flops": sum(4.0 * hq * d * (m * c + m * (m + 1) / 2) for c, m in zip(ctx, n))}


# ---------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _on(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).to(DEV)


def _power(e):
    """2^e of whole numbers, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _page_exponent(amax):
    """The least e with amax <= 448 * 2^e, within LOW and HIGH."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, LOW).clamp(LOW, HIGH)


def _fill(case, kind, num_pages, g):
    """A pool of num_pages as the library writes it, from K with per-channel spread and V ~ N(0, 1), the pages' sizes
    apart by a few factors of two: codes uint8 [pages][kv][heads][16][D] and the kind's scales."""
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    nkv = 1 if mla else 2
    codes = torch.empty(num_pages, nkv, hkv, PAGE, d, dtype=torch.uint8, device=DEV)
    scales = None
    if kind == "fp8_e4m3_page":
        scales = torch.empty(num_pages, nkv, hkv, dtype=torch.float32, device=DEV)
    elif not kind.endswith("unscaled"):
        scales = torch.empty(num_pages, nkv, hkv, PAGE, d // 32, dtype=torch.int16, device=DEV)
    spread = torch.exp(0.5 * torch.randn(nkv, hkv, 1, d, generator=g, device=DEV))
    if not mla:
        spread[1] = 1.0
    step = max(1, (1 << 27) // (nkv * hkv * PAGE * d))
    for p in range(0, num_pages, step):
        m = min(step, num_pages - p)
        x = torch.randn(m, nkv, hkv, PAGE, d, generator=g, device=DEV) * spread
        if kind == "fp8_e4m3_page":
            x *= torch.exp(0.3 * torch.randn(m, nkv, hkv, 1, 1, generator=g, device=DEV))
            s = _power(_page_exponent(x.abs().amax((-1, -2))))
            scales[p:p + m] = s
            codes[p:p + m] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        elif kind == "fp8_e4m3_unscaled":
            codes[p:p + m] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif kind == "fp8_e5m2_unscaled":
            codes[p:p + m] = x.to(torch.float8_e5m2).view(torch.uint8)
        else:
            x = x.view(m, nkv, hkv, PAGE, d // 32, 32)
            s = (x.abs().amax(-1, keepdim=True) / (448.0 if kind == "fp8_e4m3" else 127.0)).to(torch.float16)
            y = x / s.float()
            y = (y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if kind == "fp8_e4m3"
                 else torch.round(y).clamp(-127, 127).to(torch.int8).view(torch.uint8))
            codes[p:p + m] = y.view(m, nkv, hkv, PAGE, d)
            scales[p:p + m] = s.squeeze(-1).view(torch.int16)
    return codes, scales


def _tables(lens, num_pages, seed):
    """Block tables over pages in an order drawn at random."""
    order = np.random.RandomState(seed % (1 << 31)).permutation(num_pages)
    t = np.full((len(lens), max(1, max(_pages(x) for x in lens))), -1, np.int32)
    at = 0
    for b, x in enumerate(lens):
        t[b, :_pages(x)] = order[at:at + _pages(x)]
        at += _pages(x)
    return t


def _angles(positions, rot):
    """cos and sin of position * 10000^(-2i / rot), i < rot / 2, from 64 bits: fp32 [positions][rot]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def prepare(case, seed):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    g = _gen(seed)
    ctx, n = _lens(case)
    lens = [c + m for c, m in zip(ctx, n)]
    kind = case.get("kind", "fp8_e4m3_page")
    s = {"case": dict(case), "kind": kind, "pages": sum(_pages(x) for x in lens)}
    s["codes"], s["scales"] = _fill(case, kind, s["pages"], g)
    s["table"] = _on(_tables(lens, s["pages"], seed))
    s["lens"] = _on(lens, torch.int32)
    s["start"] = _on(np.concatenate([[0], np.cumsum(n)]), torch.int32)
    s["n_max"] = max(n)
    if case["op"] == "append":
        t = sum(n)
        nkv = 1 if mla else 2
        # rows as a projection leaves them: q, k and v of a token side by side, or apart
        rows = torch.randn(t, hq + nkv * hkv, d, generator=g, device=DEV)
        rows[:, hq:hq + hkv] *= torch.exp(0.5 * torch.randn(hkv, d, generator=g, device=DEV))
        rows = rows.to(torch.bfloat16)
        parts = [rows[:, :hq], rows[:, hq:hq + hkv]] + ([] if mla else [rows[:, hq + hkv:]])
        if not case["slices"]:
            parts = [x.contiguous() for x in parts]
        s["q"], s["k"], s["v"] = (parts + [None])[:3]
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["angles"] = _angles(max(lens), _rot(case)[1])
        # pages that a sequence's new tokens touch, at most
        s["touched"] = max(_pages(c + m) - c // PAGE for c, m in zip(ctx, n))
        return s
    rows = case["batch"] if case["op"] == "decode" else sum(n)
    s["q"] = torch.randn(rows, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _rotated(x, cos, sin, first, rot, pairs):
    """Rows [T, H, D] in 32 bits, the rot elements from `first` on rotated: element i with its partner half a rotation
    away, or with its neighbour."""
    x = x.to(torch.float32)
    r = x[..., first:first + rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    c, e = cos[:, None], sin[:, None]
    a, b = a * c - b * e, b * c + a * e
    r = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([x[..., :first], r, x[..., first + rot:]], -1)


def _places(s):
    """Of each new token its sequence, its place there, and its angles' cos and sin."""
    start, lens = s["start"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    at = lens[b] - start[b + 1] + t
    a = s["angles"][at]
    return b, at, a[:, :a.shape[1] // 2], a[:, a.shape[1] // 2:]


def _rounded(y, kind):
    """Codes of scaled values."""
    if kind == "q8_0":  # half away from zero
        y = torch.trunc(y.double() + torch.copysign(torch.full_like(y, 0.5), y).double())
        return y.clamp(-127, 127).to(torch.int8).view(torch.uint8)
    if kind == "fp8_e5m2_unscaled":
        return y.clamp(-57344, 57344).to(torch.float8_e5m2).view(torch.uint8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _shown(s):
    """The pool's arrays as the numbers they hold."""
    kind, codes = s["kind"], s["codes"]
    codes = codes.view(torch.int8 if kind == "q8_0" else torch.float8_e5m2 if "e5m2" in kind else torch.float8_e4m3fn)
    scales = s["scales"]
    if scales is not None and scales.dtype == torch.int16:
        scales = scales.view(torch.float16)
    return {"q": s["q_out"], "codes": codes, "scales": scales}


def _plain_append(s):
    case, kind, codes, scales = s["case"], s["kind"], s["codes"], s["scales"]
    first, rot = _rot(case)
    b, at, cos, sin = _places(s)
    s["q_out"] = _rotated(s["q"], cos, sin, first, rot, case["pairs"]).to(torch.bfloat16)
    rows = [_rotated(s["k"], cos, sin, first, rot, case["pairs"])]
    if s["v"] is not None:
        rows.append(s["v"].to(torch.float32))
    x = torch.stack(rows, 1)                                                # [T, kv, heads, D]
    if kind == "fp8_e4m3_page":
        return _plain_append_pages(s, x)
    page, off = s["table"].long()[b, at // PAGE], at % PAGE
    if scales is not None:
        x = x.unflatten(-1, (-1, 32))
        top = torch.tensor(448.0 if kind == "fp8_e4m3" else 127.0, device=DEV)
        sc = (x.abs().amax(-1) / top).clamp(max=65504).to(torch.float16)
        scales[page, :, :, off] = sc.view(torch.int16)
        sc = sc.float().unsqueeze(-1)
        x = torch.where(sc > 0, x / torch.where(sc > 0, sc, torch.ones_like(sc)), torch.zeros_like(x)).flatten(-2)
    codes[page, :, :, off] = _rounded(x, kind)
    return _shown(s)


def _plain_append_pages(s, x):
    codes, scales = s["codes"], s["scales"]
    start, lens = s["start"].long(), s["lens"].long()
    old = lens - (start[1:] - start[:-1])                                  # tokens stored before
    count = torch.where(lens > old, (lens + PAGE - 1) // PAGE - old // PAGE, 0)
    j = torch.arange(s["touched"], device=DEV)
    j = torch.minimum(j[None, :], (count - 1).clamp(min=0)[:, None])       # (a page listed twice is written twice alike)
    at = (old // PAGE)[:, None] + j                                        # [B, J]: number within the sequence
    pos = at[:, :, None] * PAGE + torch.arange(PAGE, device=DEV)           # [B, J, 16]
    new = (pos >= old[:, None, None]) & (pos < lens[:, None, None])
    kept = pos < old[:, None, None]
    row = (start[:-1] - old)[:, None, None] + pos
    v = x[row.clamp(0, x.shape[0] - 1)].permute(0, 1, 3, 4, 2, 5)           # [B, J, kv, heads, 16, D]
    new, kept = new[:, :, None, None, :, None], kept[:, :, None, None, :, None]
    page = s["table"].long().gather(1, at)
    had = torch.frexp(scales[page])[1] - 1
    e = _page_exponent(torch.where(new, v.abs(), 0).amax((-1, -2)))
    e = torch.where(kept.any(4)[..., 0], torch.maximum(e, had), e)
    was = codes[page]
    again = was.view(torch.float8_e4m3fn).float() * _power(had - e)[..., None, None]
    fresh = _rounded(v / _power(e)[..., None, None], "fp8_e4m3")
    codes[page] = torch.where(new, fresh, torch.where(kept, _rounded(again, "fp8_e4m3"), was))
    scales[page] = _power(e)
    return _shown(s)


def _cached(s):
    """Keys and values [B, heads, S, D] of the sequences' pages, and which columns hold a token's page."""
    hq, hkv, d, dv, mla = HEADS[s["case"]["heads"]]
    table = s["table"].long()
    page = table.clamp(min=0)
    x = s["codes"][page].view(torch.float8_e4m3fn).float() * s["scales"][page][..., None, None]
    x = x.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)                           # [kv, B, heads, S, D]
    return x[0], x[1], (table >= 0).repeat_interleave(PAGE, 1)


def _softmax_times(scores, seen, v):
    """softmax over the seen columns times v; rows that see nothing give zeros."""
    scores = scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s):
    k, v, there = _cached(s)
    b, hkv, cols, d = k.shape
    q = s["q"].to(torch.float32).view(b, hkv, -1, d) * s["scale"]
    seen = there & (torch.arange(cols, device=DEV) < s["lens"].long()[:, None])
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)), seen[:, None, None], v)
    return o.reshape(b, -1, d).to(torch.bfloat16)


def _plain_extend(s):
    k, v, there = _cached(s)
    b, hkv, cols, d = k.shape
    start, lens, m = s["start"].long(), s["lens"].long(), s["n_max"]
    n = start[1:] - start[:-1]
    i = torch.arange(m, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)              # [B, m]
    q = s["q"][row].to(torch.float32).view(b, m, hkv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3) * s["scale"]
    pos = (lens - n)[:, None] + i
    col = torch.arange(cols, device=DEV)
    seen = (col <= pos[:, :, None]) & (col < lens[:, None, None]) & there[:, None]      # [B, m, S]
    seen = seen[:, None, None].expand(b, 1, q.shape[2] // m, m, cols).flatten(2, 3)
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)), seen, v)
    o = o.view(b, hkv, -1, m, d).permute(0, 3, 1, 2, 4).reshape(b, m, -1, d)
    t = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return o[of, t - start[of]].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------- the library's calls
def _own(s):
    from block_quantized_bit_gb300 import kvq
    case = s["case"]
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    if "layout" not in s:
        s["layout"] = kvq.Layout(s["pages"], PAGE, hkv, d, dv, mla)
    L, kind = s["layout"], s["kind"]
    if case["op"] == "append":
        if "ws" not in s:
            s["ws"] = kvq.alloc_append_workspace(DEV)
        kvq.kvq_append(s["codes"], s["scales"], s["k"], s["v"], s["table"], s["lens"], s["start"], s["ws"], L, kind, q=s["q"],
                       q_out=s["q_out"], cos_sin=s["angles"], rot_offset=_rot(case)[0], interleaved=case["pairs"])
        return _shown(s)
    if case["op"] == "decode":
        if "ws" not in s:
            s["ws"] = kvq.alloc_workspace(L, s["lens"].numel(), hq, s["table"].shape[1], DEV, kind=kind)
        kvq.kvq_decode(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["out"], s["ws"], L, kind, s["scale"])
    else:
        if "ws" not in s:
            s["ws"] = kvq.alloc_extend_workspace(DEV, L, s["q"].shape[0], hq, s["table"].shape[1], kind=kind,
                                                 batch=s["lens"].numel())
        kvq.kvq_extend(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["start"], s["out"], s["ws"], L, kind,
                       s["scale"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_append(state) if op == "append" else _plain_decode(state) if op == "decode" else _plain_extend(state)


# ---------------------------------------------------------------------------------------------- 64 bits
def _near(y, kind):
    """The code values nearest to 64-bit numbers within the codes' range."""
    if kind == "q8_0":
        return torch.sign(y) * torch.floor(y.abs() + 0.5)
    return y.to(torch.float8_e5m2 if "e5m2" in kind else torch.float8_e4m3fn).double()


def _exact_append(s):
    """The rotation as a product of complex numbers, and the codes nearest to its results, page after page."""
    case, kind = s["case"], s["kind"]
    first, rot = _rot(case)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    at = torch.cat([torch.arange(x - (hi - lo), x, device=DEV) for x, lo, hi in zip(lens, start, start[1:])])
    f = s["angles"].double()[at]
    z = torch.complex(f[:, :rot // 2], f[:, rot // 2:])[:, None]
    i = torch.arange(rot // 2, device=DEV)
    re, im = (2 * i + first, 2 * i + 1 + first) if case["pairs"] else (i + first, i + rot // 2 + first)

    def turned(x):
        x = x.double()
        y = torch.complex(x[..., re], x[..., im]) * z
        x[..., re], x[..., im] = y.real, y.imag
        return x

    x = torch.stack([turned(s["k"])] + ([] if s["v"] is None else [s["v"].double()]), 1)
    shown = _shown(s)
    codes, scales = shown["codes"].double(), None if s["scales"] is None else shown["scales"].double()
    top = {"q8_0": 127.0, "fp8_e5m2_unscaled": 57344.0}.get(kind, 448.0)
    for b in range(len(lens)):
        old = lens[b] - (start[b + 1] - start[b])
        for p in range(old // PAGE, _pages(lens[b]) if lens[b] > old else 0):
            lo, hi, page = max(old, p * PAGE), min(lens[b], (p + 1) * PAGE), int(s["table"][b, p])
            y = x[start[b] + lo - old:start[b] + hi - old].permute(1, 2, 0, 3)      # [kv, heads, tokens, D]
            rows, kept = slice(lo - p * PAGE, hi - p * PAGE), slice(0, lo - p * PAGE)
            if kind == "fp8_e4m3_page":
                m, e = torch.frexp(y.abs().amax((-1, -2)))              # the largest is m 2^e; 448 = 0.875 * 2^9
                e = torch.where(m > 0.875, e - 8, e - 9).masked_fill(m == 0, LOW).clamp(LOW, HIGH)
                scale = ((e.long() + 1023) << 52).view(torch.float64)
                if lo > p * PAGE:
                    scale = torch.maximum(scale, scales[page])
                    codes[page, :, :, kept] = _near(codes[page, :, :, kept] * (scales[page] / scale)[..., None, None], kind)
                scales[page] = scale
                y = y / scales[page][..., None, None]
            elif scales is not None:
                y = y.unflatten(-1, (-1, 32))
                sc = (y.abs().amax(-1) / top).clamp(max=65504).to(torch.float16).double()
                scales[page, :, :, rows] = sc
                y = torch.where(sc.unsqueeze(-1) > 0, y / sc.clamp(min=2.0 ** -24).unsqueeze(-1), 0).flatten(-2)
            codes[page, :, :, rows] = _near(y.clamp(-top, top), kind)
    return {"q": turned(s["q"]), "codes": None if kind == "q8_0" else codes, "scales": scales}


def exact(case, seed):
    """From the definitions in 64 bits, one sequence after the other."""
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    lens, start = s["lens"].tolist(), s["start"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, length in enumerate(lens):
        lo, hi = (b, b + 1) if case["op"] == "decode" else (start[b], start[b + 1])
        if lo == hi or length == 0:
            continue
        page = s["table"][b, :_pages(length)].long()
        c = s["codes"][page].view(torch.float8_e4m3fn).to(torch.float64) * s["scales"][page].double()[..., None, None]
        c = c.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :length]
        step = max(1, (1 << 28) // (length * (hq // hkv)))
        for h in range(hkv):
            for r in range(lo, hi, step):
                q = s["q"][r:min(r + step, hi), h * (hq // hkv):(h + 1) * (hq // hkv)].double()
                a = torch.einsum("ngd,td->ngt", q, c[0, h]) * s["scale"]
                last = length - (hi - r) + torch.arange(q.shape[0], device=DEV)
                see = torch.arange(length, device=DEV)[None, :] <= last[:, None]
                w = torch.softmax(a.masked_fill(~see[:, None, :], float("-inf")), -1)
                out[r:r + q.shape[0], h * (hq // hkv):(h + 1) * (hq // hkv)] = torch.einsum("ngt,td->ngd", w, c[1, h])
    return out
