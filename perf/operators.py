"""Cases, plain forms and exact values of the operators that act on a prompt, on drafted tokens and on
the pages of the 8-bit cache.

Five operators, each with its plain form (elementary torch operations in 32 bits) and the call a user
makes of the library (``own``):

* ``tree``    attention of drafted tokens, arranged as a tree, over the paged 8-bit cache
* ``prompt``  causal attention over whole prompts, packed one behind the other, grouped heads, bf16
* ``copy``    copies of whole pages
* ``fork``    sequences that take over other sequences' pages (beams, samples), and the copies of the
              partly filled last pages that this asks for
* ``accept``  the page work of one speculative step: pages for the drafted tokens, the accepted tokens'
              rows moved together, the surplus pages released
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"
KINDS = ("fp8_e4m3", "q8_0", "fp8_e4m3_unscaled", "fp8_e5m2_unscaled")
# (query heads, kv heads, K width, V width, latent row) of the repository's own workloads
HEADS = {"tiny": (8, 2, 128, 128, False), "qwen3_1p7b": (16, 8, 128, 128, False), "long_gqa": (16, 2, 256, 256, False),
         "serving": (32, 8, 128, 128, False), "mla": (128, 1, 576, 512, True)}


def listed():
    return [
        # one chat, one small tree behind a short context: the call's own latency
        dict(name="tree_one_chat", op="tree", heads="tiny", kind="fp8_e4m3", batch=1, ctx_lo=505, ctx_hi=505, n_lo=8,
             n_hi=8, shape=1),
        # a serving batch, ragged contexts and ragged trees
        dict(name="tree_serving", op="tree", heads="serving", kind="q8_0", batch=32, ctx_lo=700, ctx_hi=8192, n_lo=3,
             n_hi=16, shape=2),
        # a few long documents with wide trees
        dict(name="tree_long", op="tree", heads="long_gqa", kind="fp8_e4m3", batch=4, ctx_lo=65536, ctx_hi=65536,
             n_lo=32, n_hi=32, shape=3),
        # one short prompt: latency
        dict(name="prompt_short", op="prompt", heads="tiny", batch=1, len_lo=200, len_hi=200, shape=4),
        # a prefill batch of ragged prompts
        dict(name="prompt_packed", op="prompt", heads="qwen3_1p7b", batch=8, len_lo=150, len_hi=2048, shape=5),
        # one long document
        dict(name="prompt_long", op="prompt", heads="serving", batch=1, len_lo=16384, len_hi=16384, shape=6),
        # the copies that one beam step asks for
        dict(name="copy_beams", op="copy", heads="serving", kind="fp8_e4m3", pages=512, count=24, shape=7),
        # pages of a long context moved away
        dict(name="copy_context", op="copy", heads="long_gqa", kind="q8_0", pages=40000, count=16384, shape=8),
        # beams re-ordered: 16 prompts with 4 beams each
        dict(name="fork_beams", op="fork", heads="serving", kind="fp8_e4m3", batch=64, ctx_lo=300, ctx_hi=4096, beams=4,
             shape=9),
        # samples of long prompts
        dict(name="fork_samples", op="fork", heads="qwen3_1p7b", kind="q8_0", batch=32, ctx_lo=30000, ctx_hi=32768,
             beams=16, shape=10),
        # one chat accepts a path
        dict(name="accept_one_chat", op="accept", heads="qwen3_1p7b", kind="fp8_e4m3", batch=1, ctx_lo=1003, ctx_hi=1003,
             n_lo=8, n_hi=8, shape=11),
        # a serving batch accepts its paths
        dict(name="accept_serving", op="accept", heads="serving", kind="q8_0", batch=64, ctx_lo=300, ctx_hi=4096, n_lo=4,
             n_hi=64, shape=12),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "prompt", "prompt", "copy", "fork", "accept"))
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most[c["op"]], w["bytes"] / 7e12 + w["flops"] / 5e14)
    while True:
        c = dict(op=op, shape=rng.randrange(1 << 30))
        if op == "tree":
            c["heads"] = rng.choice(("tiny", "qwen3_1p7b", "long_gqa", "serving", "mla"))
            c["kind"] = rng.choice(KINDS)
            c["batch"] = _spread(rng, 1, 64)
            c["ctx_hi"] = _spread(rng, 1, 65536)
            c["ctx_lo"] = max(1, int(c["ctx_hi"] * rng.uniform(0.1, 1.0)))
            c["n_hi"] = _spread(rng, 1, 64)
            c["n_lo"] = max(1, int(c["n_hi"] * rng.uniform(0.1, 1.0)))
            if c["heads"] == "mla" and c["n_hi"] * c["batch"] * c["ctx_hi"] > 300000:
                continue
        elif op == "prompt":
            c["heads"] = rng.choice(("tiny", "qwen3_1p7b", "long_gqa", "serving"))
            c["batch"] = _spread(rng, 1, 16)
            c["len_hi"] = _spread(rng, 1, 8192)
            c["len_lo"] = max(1, int(c["len_hi"] * rng.uniform(0.05, 1.0)))
            if c["batch"] * HEADS[c["heads"]][0] * c["len_hi"] ** 2 > 32 * 16384 ** 2:
                continue
        elif op == "copy":
            c["heads"] = rng.choice(("qwen3_1p7b", "long_gqa", "serving", "mla"))
            c["kind"] = rng.choice(KINDS)
            c["count"] = _spread(rng, 1, 12000)
            c["pages"] = c["count"] * 2 + rng.randrange(1, 1000)
        else:
            c["heads"] = rng.choice(("qwen3_1p7b", "long_gqa", "serving", "mla"))
            c["kind"] = rng.choice(KINDS)
            c["batch"] = _spread(rng, 1, 64)
            c["ctx_hi"] = _spread(rng, 20, 32768)
            c["ctx_lo"] = max(1, int(c["ctx_hi"] * rng.uniform(0.1, 1.0)))
            if c["batch"] * c["ctx_hi"] > 32 * 32768:
                continue
            if op == "fork":
                c["beams"] = rng.choice((1, 2, 4, 5, 8))
                c["batch"] = max(c["beams"], c["batch"] // c["beams"] * c["beams"])
            else:
                c["n_hi"] = _spread(rng, 1, 64)
                c["n_lo"] = max(1, int(c["n_hi"] * rng.uniform(0.1, 1.0)))
        w = work(c)
        if w["bytes"] / 7e12 + w["flops"] / 5e14 <= most[op]:
            return c


# ---------------------------------------------------------------------------------------------- shapes
def _ints(case, what, lo, hi, count):
    r = random.Random("%d %s" % (case["shape"], what))
    return [r.randint(lo, hi) for _ in range(count)]


def _lens(case):
    """Context tokens and drafted tokens of each sequence (``tree``, ``accept``)."""
    ctx = _ints(case, "ctx", case["ctx_lo"], case["ctx_hi"], case["batch"])
    n = _ints(case, "n", case["n_lo"], case["n_hi"], case["batch"])
    return ctx, n


def _pages(tokens):
    return -(-tokens // PAGE)


def _token_bytes(case):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    return (1 if mla else 2) * hkv * (d + (0 if case["kind"].endswith("unscaled") else d // 16))


def work(case):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    if case["op"] == "tree":
        ctx, n = _lens(case)
        rows = sum(n)
        b = sum(c + m for c, m in zip(ctx, n)) * _token_bytes(case) + rows * hq * (d + dv) * 2 + rows * 8
        b += sum(_pages(c + m) for c, m in zip(ctx, n)) * 4
        return {"bytes": b, "flops": sum(2.0 * m * hq * (d + dv) * (c + m) for c, m in zip(ctx, n))}
    if case["op"] == "prompt":
        lens = _ints(case, "len", case["len_lo"], case["len_hi"], case["batch"])
        return {"bytes": sum(lens) * (2 * hq + 2 * hkv) * d * 2,
                "flops": sum(4.0 * hq * d * x * (x + 1) / 2 for x in lens)}
    if case["op"] == "copy":
        return {"bytes": case["count"] * (2 * PAGE * _token_bytes(case) + 8), "flops": 0}
    if case["op"] == "fork":
        # each row read, the new one written, both rows' counts changed; the last pages copied; the counts looked at
        src, lens, pages, copies = _fork_shape(case)
        rows = sum(_pages(lens[s]) for s in src)
        return {"bytes": rows * (4 + 4) + 4 * rows * 4 + pages * 4 + copies * 2 * PAGE * _token_bytes(case), "flops": 0}
    ctx, n = _lens(case)
    kept = _accepted(case)
    pages = _pages(max(ctx) + max(n)) * case["batch"]
    moved = sum(sum(k != i for i, k in enumerate(path)) for path in kept)
    return {"bytes": moved * 2 * _token_bytes(case) + sum(n) // 8 + 2 * pages * 4 + sum(_pages(m) for m in n) * 4 * 8,
            "flops": 0}


def _tree(r, n):
    """Parents of n drafted tokens (-1: the last token of the context), each before its children."""
    return [-1 if i == 0 else r.randint(max(-1, i - 9), i - 1) for i in range(n)]


def _path(parents, leaf):
    p = []
    while leaf >= 0:
        p.append(leaf)
        leaf = parents[leaf]
    return p[::-1]


def _accepted(case):
    """The accepted path of each sequence (drafted tokens' numbers, rising)."""
    ctx, n = _lens(case)
    r = random.Random("%d accepted" % case["shape"])
    return [_path(_tree(r, m), r.randrange(m)) for m in n]


def _fork_shape(case):
    """The parent of every sequence, the lengths, the pages in the pool and the copies needed."""
    b, k = case["batch"], case["beams"]
    lens = _ints(case, "ctx", case["ctx_lo"], case["ctx_hi"], b // k)
    lens = [x for x in lens for _ in range(k)]
    r = random.Random("%d parents" % case["shape"])
    src = [i // k * k + r.randrange(k) for i in range(b)]
    copies = sum(lens[s] % PAGE != 0 and s in src[:i] for i, s in enumerate(src))
    # every prompt's full pages are held once, the beams' last pages each on their own; room for the copies
    pages = sum(_pages(lens[i]) for i in range(0, b, k)) + 3 * b + 64
    return src, lens, pages, copies


# ---------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _fill(case, num_pages, g):
    """A pool of num_pages written as the store writes it: codes uint8 [pages][kv][heads][16][D], scales as
    fp16 bits [..][D / 32], from K with per-channel spread and V ~ N(0, 1)."""
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    nkv = 1 if mla else 2
    codes = torch.empty(num_pages, nkv, hkv, PAGE, d, dtype=torch.uint8, device=DEV)
    scales = torch.empty(num_pages, nkv, hkv, PAGE, d // 32, dtype=torch.int16, device=DEV)
    spread = torch.exp(0.5 * torch.randn(nkv, hkv, 1, d, generator=g, device=DEV))
    if not mla:
        spread[1] = 1.0
    step = max(1, (1 << 27) // (nkv * hkv * PAGE * d))
    for p in range(0, num_pages, step):
        m = min(step, num_pages - p)
        x = torch.randn(m, nkv, hkv, PAGE, d, generator=g, device=DEV) * spread
        if case["kind"] == "fp8_e4m3_unscaled":
            codes[p:p + m] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            continue
        if case["kind"] == "fp8_e5m2_unscaled":
            codes[p:p + m] = x.to(torch.float8_e5m2).view(torch.uint8)
            continue
        x = x.view(m, nkv, hkv, PAGE, d // 32, 32)
        top = 448.0 if case["kind"] == "fp8_e4m3" else 127.0
        s = (x.abs().amax(-1, keepdim=True) / top).to(torch.float16)
        y = x / s.float()
        y = (y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if case["kind"] == "fp8_e4m3"
             else torch.round(y).clamp(-127, 127).to(torch.int8).view(torch.uint8))
        codes[p:p + m] = y.view(m, nkv, hkv, PAGE, d)
        scales[p:p + m] = s.squeeze(-1).view(torch.int16)
    if case["kind"].endswith("unscaled"):
        scales = None
    return codes, scales


def _tables(lens, room, num_pages, seed):
    """Block tables of `room` pages a row over pages in an order drawn at random."""
    order = np.random.RandomState(seed % (1 << 31)).permutation(num_pages)
    t = np.full((len(lens), room), -1, np.int32)
    at = 0
    for b, x in enumerate(lens):
        t[b, :_pages(x)] = order[at:at + _pages(x)]
        at += _pages(x)
    return t


def _on(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).to(DEV)


def _prepare_tree(case, seed, g, s):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    ctx, n = _lens(case)
    lens = [c + m for c, m in zip(ctx, n)]
    s["pages"] = sum(_pages(x) for x in lens)
    s["codes"], s["scales"] = _fill(case, s["pages"], g)
    s["table"] = _on(_tables(lens, max(_pages(x) for x in lens), s["pages"], seed))
    s["lens"] = _on(lens, torch.int32)
    s["start"] = _on(np.concatenate([[0], np.cumsum(n)]), torch.int32)
    s["q"] = (torch.randn(sum(n), hq, d, generator=g, device=DEV) / math.sqrt(d)).to(torch.bfloat16)
    r = random.Random(seed)
    words = []
    for m in n:
        rows = []
        for i, p in enumerate(_tree(r, m)):
            rows.append((rows[p] if p >= 0 else 0) | 1 << i)
        words += rows
    s["mask"] = _on([w - (1 << 64) if w >> 63 else w for w in words], torch.int64).view(-1, 1)
    s["n_max"] = max(n)
    s["out"] = torch.empty(sum(n), hq, dv, dtype=torch.bfloat16, device=DEV)


def _prepare_prompt(case, seed, g, s):
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    lens = _ints(case, "len", case["len_lo"], case["len_hi"], case["batch"])
    t = sum(lens)
    s["start"] = _on(np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    s["longest"] = max(lens)
    s["q"] = (torch.randn(t, hq, d, generator=g, device=DEV)).to(torch.bfloat16)
    s["k"] = (torch.randn(t, hkv, d, generator=g, device=DEV)
              * torch.exp(0.5 * torch.randn(hkv, d, generator=g, device=DEV))).to(torch.bfloat16)
    s["v"] = torch.randn(t, hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)


def _prepare_copy(case, seed, g, s):
    s["pages"] = case["pages"]
    s["codes"], s["scales"] = _fill(case, case["pages"], g)
    order = np.random.RandomState(seed % (1 << 31)).permutation(case["pages"])
    n = case["count"]
    s["src"], s["dst"] = _on(order[:n], torch.int32), _on(order[n:2 * n], torch.int32)


def _prepare_fork(case, seed, g, s):
    src, lens, pages, copies = _fork_shape(case)
    b, k = case["batch"], case["beams"]
    s["pages"] = pages
    s["codes"], s["scales"] = _fill(case, pages, g)
    order = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    room = max(_pages(x) for x in lens) + 4
    t, at = np.full((b, room), -1, np.int32), 0
    for i in range(b):
        full, used = lens[i] // PAGE, _pages(lens[i])
        if i % k == 0:
            t[i, :full] = order[at:at + full]
            at += full
        else:
            t[i, :full] = t[i // k * k, :full]
        if used > full:
            t[i, full] = order[at]
            at += 1
    refs = np.zeros(pages, np.int32)
    np.add.at(refs, t[t >= 0], 1)
    s.update(table=_on(t), refs=_on(refs), lens=_on(lens, torch.int32), src=_on(src, torch.int32),
             dst=_on(range(b), torch.int32))
    s["copy_src"], s["copy_dst"] = torch.empty_like(s["src"]), torch.empty_like(s["dst"])


def _prepare_accept(case, seed, g, s):
    ctx, n = _lens(case)
    room = _pages(max(ctx) + max(n))
    s["pages"] = sum(_pages(c) + _pages(m) + 1 for c, m in zip(ctx, n))
    s["codes"], s["scales"] = _fill(case, s["pages"], g)
    t = _tables(ctx, room, s["pages"], seed)
    refs = np.zeros(s["pages"], np.int32)
    np.add.at(refs, t[t >= 0], 1)
    kept = _accepted(case)
    words = [sum(1 << j for j in path) for path in kept]
    s.update(table=_on(t), refs=_on(refs), lens=_on(ctx, torch.int32), seqs=_on(range(case["batch"]), torch.int32),
             drafted_lens=_on([c + m for c, m in zip(ctx, n)], torch.int32),
             start=_on(np.concatenate([[0], np.cumsum(n)]), torch.int32),
             keep=_on([w - (1 << 64) if w >> 63 else w for w in words], torch.int64).view(-1, 1))
    s["n_max"] = max(n)
    s["new_lens"] = torch.empty(case["batch"], dtype=torch.int32, device=DEV)


def prepare(case, seed):
    s = {"case": dict(case)}
    {"tree": _prepare_tree, "prompt": _prepare_prompt, "copy": _prepare_copy, "fork": _prepare_fork,
     "accept": _prepare_accept}[case["op"]](case, seed, _gen(seed), s)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _values(codes, scales, kind):
    """What the cache holds: value(code) * scale, rounded to bf16 by the operator's definition."""
    if kind == "q8_0":
        x = codes.view(torch.int8).float()
    elif kind == "fp8_e5m2_unscaled":
        x = codes.view(torch.float8_e5m2).float()
    else:
        x = codes.view(torch.float8_e4m3fn).float()
    if scales is not None:
        x = x.unflatten(-1, (-1, 32)) * scales.view(torch.float16).float().unsqueeze(-1)
        x = x.flatten(-2)
    return x.to(torch.bfloat16).float()


def _softmax_times(scores, seen, v):
    """softmax over the seen columns times v; rows that see nothing give zeros."""
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_tree(s):
    hq, hkv, d, dv, mla = HEADS[s["case"]["heads"]]
    table, lens, start = s["table"].long(), s["lens"].long(), s["start"].long()
    b, n_max, g = table.shape[0], s["n_max"], hq // hkv
    n = start[1:] - start[:-1]
    kv = _values(s["codes"][table.clamp(min=0)], None if s["scales"] is None else s["scales"][table.clamp(min=0)],
                 s["case"]["kind"])                                     # [B, P, kv, Hkv, 16, D]
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    v = k[..., :dv] if mla else kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, dv)
    i = torch.arange(n_max, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B, n_max]
    q = s["q"][row].float().view(b, n_max, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n_max * g, d)
    pos = torch.arange(k.shape[2], device=DEV)
    at = pos - (lens - n)[:, None]                                      # [B, S]: number among the drafted tokens
    bit = (s["mask"][:, 0][row][:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
    seen = ((at < 0)[:, None, :] | (bit == 1)) & (pos < lens[:, None])[:, None, :]
    seen &= (table.repeat_interleave(PAGE, 1) >= 0)[:, None, :]
    seen = seen[:, None, :, None, :].expand(b, 1, n_max, g, -1).reshape(b, 1, n_max * g, -1)
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)), seen, v)
    o = o.view(b, hkv, n_max, g, dv).permute(0, 2, 1, 3, 4).reshape(b, n_max, hq, dv)
    t = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return o[of, t - start[of]].to(torch.bfloat16)


def _plain_prompt(s):
    hq, hkv, d, dv, mla = HEADS[s["case"]["heads"]]
    start = s["start"].long()
    b, m, g = start.numel() - 1, s["longest"], hq // hkv
    lens = start[1:] - start[:-1]
    i = torch.arange(m, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(b, m, hkv, g, d).permute(0, 2, 3, 1, 4)
    k = s["k"][row].float().permute(0, 2, 1, 3).unsqueeze(2)
    v = s["v"][row].float().permute(0, 2, 1, 3).unsqueeze(2)
    seen = (i[None, :] <= i[:, None]) & (i < lens[:, None])[:, None, :]  # [B, m, m]
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]), seen[:, None, None], v)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)
    t = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return o[of, t - start[of]].to(torch.bfloat16)


def _copy_pages(s, src, dst, held=None):
    """Pages src to dst; where src is -1 the page `held`, which is no destination, is written to itself."""
    a, z = src.long(), dst.long()
    if held is not None:
        a, z = torch.where(src >= 0, a, held.long()), torch.where(src >= 0, z, held.long())
    s["codes"][z] = s["codes"][a]
    if s["scales"] is not None:
        s["scales"][z] = s["scales"][a]


def _lowest_free(refs):
    return torch.sort((refs != 0).to(torch.int8), stable=True).indices


def _count(refs, pages, by):
    """refs changed by `by` for every page >= 0 listed."""
    pages = pages.reshape(-1).long()
    ok = pages >= 0
    refs.index_add_(0, pages.clamp(min=0), torch.where(ok, by, 0).to(refs.dtype))


def _plain_fork(s):
    table, lens, refs, src, dst = s["table"], s["lens"], s["refs"], s["src"].long(), s["dst"].long()
    free = _lowest_free(refs)
    room = table.shape[1]
    col = torch.arange(room, device=DEV)
    new, old, new_lens = table[src], table[dst], lens[src].long()
    used = (new_lens + PAGE - 1) // PAGE
    new = torch.where(col < used[:, None], new, -1)
    old = torch.where(col < ((lens[dst].long() + PAGE - 1) // PAGE)[:, None], old, -1)
    tail = (used - 1).clamp(min=0)
    tail_page = new.gather(1, tail[:, None])[:, 0]
    j = torch.arange(src.numel(), device=DEV)
    gone = (src[:, None] == dst[None, :]).any(1)                          # the parent's row is itself replaced
    first = ~((src[:, None] == src[None, :]) & (j[None, :] < j[:, None])).any(1)
    fresh = (new_lens % PAGE != 0) & (tail_page >= 0) & ~(gone & first)
    page = free[(torch.cumsum(fresh, 0) - 1).clamp(min=0)].to(table.dtype)
    s["copy_src"] = torch.where(fresh, tail_page, -1)
    s["copy_dst"] = torch.where(fresh, page, -1)
    new = torch.where((col == tail[:, None]) & fresh[:, None], page[:, None], new)
    _count(refs, new, 1)
    _count(refs, old, -1)
    table[dst] = new
    lens[dst] = new_lens.to(lens.dtype)
    _copy_pages(s, s["copy_src"], s["copy_dst"], held=tail_page)
    return {"codes": s["codes"], "scales": s["scales"], "table": table, "lens": lens, "refs": refs}


def _resize(s, new_lens):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    seqs = s["seqs"].long()
    free = _lowest_free(refs)
    col = torch.arange(table.shape[1], device=DEV)
    rows = table[seqs]
    had = ((lens[seqs].long() + PAGE - 1) // PAGE)[:, None]
    want = ((new_lens.long() + PAGE - 1) // PAGE)[:, None]
    grow = (col >= had) & (col < want)
    rank = (torch.cumsum(grow.reshape(-1), 0) - 1).clamp(min=0).view_as(grow)
    drop = (col >= want) & (col < had)
    page = free[rank.clamp(max=free.numel() - 1)].to(table.dtype)
    _count(refs, torch.where(drop, rows, -1), -1)
    _count(refs, torch.where(grow, page, -1), 1)
    table[seqs] = torch.where(grow, page, torch.where(drop, -1, rows))
    lens[seqs] = new_lens.to(lens.dtype)


def _plain_accept(s):
    _resize(s, s["drafted_lens"])
    start, lens, table = s["start"].long(), s["lens"].long(), s["table"].long()
    n = start[1:] - start[:-1]
    base = lens - n
    j = torch.arange(s["n_max"], device=DEV)
    kept = ((s["keep"] >> j) & 1 == 1) & (j < n[:, None])                  # [B, n_max]
    count = kept.sum(1)
    order = torch.sort((~kept).to(torch.int8), dim=1, stable=True).indices
    moves = j < count[:, None]
    src = torch.where(moves, order, 0) + base[:, None]
    dst = torch.where(moves, j, 0) + base[:, None]
    # what moves nowhere repeats the first move, or stays: token 0 of the tail is then its own source
    first = torch.where(count > 0, order[:, 0], 0)
    src = torch.where(moves, src, (base + first)[:, None])
    sp, dp = table.gather(1, src // PAGE), table.gather(1, dst // PAGE)
    for x in (s["codes"], s["scales"]):
        if x is not None:
            x[dp, :, :, dst % PAGE] = x[sp, :, :, src % PAGE]
    s["new_lens"] = (base + count).to(torch.int32)
    _resize(s, s["new_lens"])
    return {"codes": s["codes"], "scales": s["scales"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}


# ---------------------------------------------------------------------------------------------- the library's calls
def _layout(s):
    from block_quantized_bit_gb300 import kvq
    hq, hkv, d, dv, mla = HEADS[s["case"]["heads"]]
    return kvq.Layout(s["pages"], PAGE, hkv, d, dv, mla)


def _own(s):
    from block_quantized_bit_gb300 import kvq
    op = s["case"]["op"]
    if op == "prompt":
        if "ws" not in s:
            s["ws"] = kvq.alloc_prompt_workspace(DEV)
        kvq.kvq_prompt(s["q"], s["k"], s["v"], s["start"], s["out"], s["ws"], sm_scale=s["scale"])
        return s["out"]
    kind = s["case"]["kind"]
    if "layout" not in s:
        s["layout"] = _layout(s)
    L = s["layout"]
    if op == "tree":
        if "ws" not in s:
            s["ws"] = kvq.alloc_tree_workspace(L, s["lens"].numel(), s["q"].shape[0], s["q"].shape[1],
                                               s["table"].shape[1], device=DEV)
        kvq.kvq_tree(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["start"], s["mask"], s["out"], s["ws"], L,
                     kind)
        return s["out"]
    if op == "copy":
        kvq.kvq_pages_copy(s["codes"], s["scales"], s["src"], s["dst"], L, kind)
        return {"codes": s["codes"], "scales": s["scales"]}
    if "ws" not in s:
        s["ws"] = kvq.alloc_pages_workspace(L, s["lens"].numel(), s["table"].shape[1], device=DEV)
    if op == "fork":
        kvq.kvq_pages_fork(s["table"], s["lens"], s["refs"], s["src"], s["dst"], s["copy_src"], s["copy_dst"], s["ws"], L)
        kvq.kvq_pages_copy(s["codes"], s["scales"], s["copy_src"], s["copy_dst"], L, kind)
    else:
        kvq.kvq_pages_resize(s["table"], s["lens"], s["refs"], s["seqs"], s["drafted_lens"], s["ws"], L)
        kvq.kvq_pages_compact(s["codes"], s["scales"], s["table"], s["lens"], s["start"], s["keep"], s["new_lens"],
                              s["ws"], L, kind, page_refs=s["refs"])
        kvq.kvq_pages_resize(s["table"], s["lens"], s["refs"], s["seqs"], s["new_lens"], s["ws"], L)
    return {"codes": s["codes"], "scales": s["scales"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tree":
        return _plain_tree(state)
    if op == "prompt":
        return _plain_prompt(state)
    if op == "copy":
        _copy_pages(state, state["src"], state["dst"])
        return {"codes": state["codes"], "scales": state["scales"]}
    return _plain_fork(state) if op == "fork" else _plain_accept(state)


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention from its definition in 64 bits, one sequence after the other.  Pages are copied, not computed:
    their outputs have no value of this kind."""
    if case["op"] not in ("tree", "prompt"):
        return None
    s = prepare(case, seed)
    hq, hkv, d, dv, mla = HEADS[case["heads"]]
    g = hq // hkv
    start = s["start"].tolist()
    out = torch.zeros(s["q"].shape[0], hq, dv, dtype=torch.float64, device=DEV)
    for b in range(len(start) - 1):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        if case["op"] == "prompt":
            k, v, length, scale = s["k"][lo:hi].double(), s["v"][lo:hi].double(), hi - lo, s["scale"]
        else:
            length, scale = int(s["lens"][b]), 1.0
            pages = s["table"][b, :_pages(length)].long()
            c = s["codes"][pages]
            c = (c.view(torch.int8) if case["kind"] == "q8_0" else c.view(torch.float8_e5m2) if "e5m2" in case["kind"]
                 else c.view(torch.float8_e4m3fn)).to(torch.float64)
            if s["scales"] is not None:
                c *= s["scales"][pages].view(torch.float16).double().repeat_interleave(32, -1)
            c = c.to(torch.bfloat16).double().permute(0, 3, 1, 2, 4).reshape(-1, c.shape[1], hkv, d)[:length]
            k, v = c[:, 0], c[:, 0, :, :dv] if mla else c[:, 1]
        step = max(1, (1 << 28) // (length * g))
        for h in range(hkv):
            for r in range(lo, hi, step):
                q = s["q"][r:min(r + step, hi), h * g:(h + 1) * g].double()
                a = torch.einsum("ngd,td->ngt", q, k[:, h]) * scale
                t = torch.arange(length, device=DEV)
                i = torch.arange(r - lo, r - lo + q.shape[0], device=DEV)
                if case["op"] == "prompt":
                    see = t[None, :] <= i[:, None]
                else:
                    at = t - (length - (hi - lo))
                    see = (at < 0) | ((s["mask"][r:r + q.shape[0]] >> at.clamp(min=0)) & 1 == 1)
                w = torch.softmax(a.masked_fill(~see[:, None, :], float("-inf")), -1)
                out[r:r + q.shape[0], h * g:(h + 1) * g] = torch.einsum("ngt,td->ngd", w, v[:, h])
    return out
