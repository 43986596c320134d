"""kvq_append on the CPU, row by row, and attention over a pool with a scale per page, for the tests.

fp32 with each product and sum rounded by itself, as the operator is defined, so pools compare bit for bit."""
import numpy as np
import torch

LOW, HIGH, PAGE = -32, 32, 16


def rotate(x, row, first, rot, pairs):
    """One token's rows x [heads, D] (fp32) turned by the angles of `row` (fp32 [rot]: cosines, then sines)."""
    x = x.clone()
    for i in range(rot // 2):
        a, b = (first + 2 * i, first + 2 * i + 1) if pairs else (first + i, first + rot // 2 + i)
        c, s = row[i], row[rot // 2 + i]
        u, v = x[:, a].clone(), x[:, b].clone()
        x[:, a], x[:, b] = u * c - v * s, v * c + u * s
    return x


def e4m3(y):
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def encode_row(x, kind):
    """Codes [heads, D] uint8 and fp16 scale bits [heads, D / 32] (or None) of fp32 rows."""
    if kind == "fp8_e4m3_unscaled":
        return e4m3(x), None
    if kind == "fp8_e5m2_unscaled":
        return x.clamp(-57344, 57344).to(torch.float8_e5m2).view(torch.uint8), None
    q = 448.0 if kind == "fp8_e4m3" else 127.0
    b = x.unflatten(-1, (-1, 32))
    s = torch.from_numpy(np.minimum(b.abs().amax(-1).numpy() / np.float32(q), np.float32(65504)).astype(np.float16))
    f = s.float().unsqueeze(-1)
    y = torch.where(f > 0, b / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(b)).flatten(-2)
    if kind == "fp8_e4m3":
        return e4m3(y), s.view(torch.int16)
    y = torch.sign(y) * torch.floor(y.double().abs() + 0.5)
    return y.clamp(-127, 127).to(torch.int8).view(torch.uint8), s.view(torch.int16)


def exponent(amax):
    if amax == 0:
        return LOW
    m, e = np.frexp(np.float32(amax))
    return int(min(max(e - 9 if m <= 0.875 else e - 8, LOW), HIGH))


def append(codes, scales, q, k, v, table, lens, start, layout, kind, angles=None, first=0, pairs=False, positions=None,
           q_out=None, skipped=()):
    """All on the CPU; codes, scales and q_out are changed."""
    P = layout.page_size
    rot = 0 if angles is None else angles.shape[1]
    pages = {}  # KVQ_FP8_E4M3_PAGE: (page, first new row) -> rows
    for b, length in enumerate(lens):
        n = start[b + 1] - start[b]
        if b in skipped or n <= 0:
            continue
        for i in range(n):
            t, at = start[b] + i, length - n + i
            pos = at if positions is None else positions[t]
            turn = (lambda x: x) if rot == 0 else (
                lambda x, p=min(max(int(pos), 0), angles.shape[0] - 1): rotate(x, angles[p], first, rot, pairs))
            if q is not None:
                q_out[t] = turn(q[t].float()).to(torch.bfloat16)
            rows = [turn(k[t].float())] + ([] if v is None else [v[t].float()])
            page = int(table[b, at // P])
            if page < 0 or page >= layout.num_pages:
                continue
            if kind == "fp8_e4m3_page":
                pages.setdefault(page, []).append((at % P, rows))
                continue
            for kv, x in enumerate(rows):
                c, s = encode_row(x, kind)
                codes[page, kv, :, at % P] = c
                if s is not None:
                    scales[page, kv, :, at % P] = s
    for page, new in pages.items():
        lo = new[0][0]
        for kv in range(2):
            for h in range(layout.num_kv_heads):
                x = torch.stack([rows[kv][h] for _, rows in new])
                e = exponent(float(x.abs().max()))
                if lo > 0:
                    old = int(np.frexp(float(scales[page, kv, h]))[1]) - 1
                    e = max(e, old)
                    was = codes[page, kv, h, :lo].view(torch.float8_e4m3fn).float()
                    codes[page, kv, h, :lo] = e4m3(was * 2.0 ** (old - e))
                scales[page, kv, h] = 2.0 ** e
                codes[page, kv, h, lo:lo + len(new)] = e4m3(x * 2.0 ** -e)


def angles_of(positions, rot, base=10000.0):
    a = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def page_values(codes, scales):
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None, None]


def attend64(q, codes, scales, table, lens, start, scale, out):
    """64-bit causal attention over a pool of fp8_e4m3_page (start None: one row per sequence); rows of `out` (double)
    that sequences cover, and the same weights times |V|."""
    mag = torch.zeros_like(out)
    pages, nkv, hkv, P, d = codes.shape
    g = q.shape[1] // hkv
    for b, length in enumerate(lens):
        r0, r1 = (b, b + 1) if start is None else (start[b], start[b + 1])
        if r1 <= r0 or (start is not None and r1 - r0 > length):
            continue
        row = table[b, :(length + P - 1) // P].long()
        ok = ((row >= 0) & (row < pages)).repeat_interleave(P)[:length]
        x = page_values(codes[row.clamp(0, pages - 1)], scales[row.clamp(0, pages - 1)])
        x = x.permute(1, 2, 0, 3, 4).reshape(nkv, hkv, -1, d)[:, :, :length]
        x = torch.where(ok[None, None, :, None], x, torch.zeros_like(x))
        step = max(1, (1 << 26) // max(1, length * q.shape[1]))
        for a in range(r0, r1, step):
            z = min(r1, a + step)
            last = length - (r1 - a) + torch.arange(z - a, device=q.device)
            seen = (torch.arange(length, device=q.device)[None] <= last[:, None]) & ok[None]
            s = torch.einsum("nhgd,htd->nhgt", q[a:z].double().unflatten(1, (hkv, g)), x[0]) * scale
            w = torch.softmax(s.masked_fill(~seen[:, None, None], float("-inf")), -1)
            w = torch.where(seen.any(-1)[:, None, None, None], w, torch.zeros_like(w))
            out[a:z] = torch.einsum("nhgt,htd->nhgd", w, x[1]).flatten(1, 2)
            mag[a:z] = torch.einsum("nhgt,htd->nhgd", w, x[1].abs()).flatten(1, 2)
    return out, mag
