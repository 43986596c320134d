"""Attention from its definition in 64 bits (torch on whatever device the inputs are), for the tests of kvq_tree
and kvq_prompt."""
import torch


def cache_values(codes, scales, kind):
    """The pool's values: bf16(code * scale), as doubles, in the pool's own shape [pages][kv][heads][16][D]."""
    if kind == "q8_0":
        x = codes.view(torch.int8).double()
    elif kind == "fp8_e5m2_unscaled":
        x = codes.view(torch.float8_e5m2).double()
    else:
        x = codes.view(torch.float8_e4m3fn).double()
    if "unscaled" not in kind:
        x = (x.unflatten(-1, (-1, 32)) * scales.view(torch.float16).double().unsqueeze(-1)).flatten(-2)
    return x.float().to(torch.bfloat16).double()  # (code * scale is exact in fp32)


def attend(q, k, v, seen, scale):
    """q [n, H, D], k / v [T, Hkv, ...], seen [n, T]: (softmax(scale q.k) v, the same weights times |v|); zeros where
    nothing is seen."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("nhd,thd->hnt", q.double(), k) * scale
    s = s.masked_fill(~seen[None], float("-inf"))
    w = torch.softmax(s, -1)
    w = torch.where(seen.any(-1)[None, :, None], w, torch.zeros_like(w))
    return torch.einsum("hnt,thd->nhd", w, v), torch.einsum("hnt,thd->nhd", w, v.abs())


def tree64(q, codes, scales, kind, table, lens, start, mask, v_dim, mla, scale, out, skipped=()):
    """Rows of `out` (a double tensor [total_q, H, v_dim]) that sequences cover; returns (out, weights times |V|)."""
    mag = torch.zeros_like(out)
    vals = cache_values(codes, scales, kind)
    pages, nkv, hkv, P, d = codes.shape
    bits = (mask[:, :, None] >> torch.arange(64, device=mask.device)) & 1
    bits = bits.reshape(mask.shape[0], -1) == 1
    for b, L in enumerate(lens):
        r0, r1 = start[b], start[b + 1]
        n = r1 - r0
        if n <= 0 or b in skipped:
            continue
        row = table[b, :(L + P - 1) // P].long()
        ok = (row >= 0) & (row < pages)
        x = vals[row.clamp(0, pages - 1)].permute(0, 3, 1, 2, 4).reshape(-1, nkv, hkv, d)[:L]
        k, v = x[:, 0], (x[:, 0, :, :v_dim] if mla else x[:, 1])
        seen = torch.ones(n, L, dtype=torch.bool, device=q.device)
        seen[:, L - n:] = bits[r0:r1, :n]
        seen &= ok.repeat_interleave(P)[:L][None]
        out[r0:r1], mag[r0:r1] = attend(q[r0:r1], k, v, seen, scale)
    return out, mag


def prompt64(q, k, v, start, scale, out):
    mag = torch.zeros_like(out)
    for r0, r1 in zip(start[:-1], start[1:]):
        if r1 > r0:
            seen = torch.ones(r1 - r0, r1 - r0, dtype=torch.bool, device=q.device).tril()
            out[r0:r1], mag[r0:r1] = attend(q[r0:r1], k[r0:r1].double(), v[r0:r1].double(), seen, scale)
    return out, mag
