"""Plain forms, in 64 bits, of the operators around the paged cache: the plan of a step, norm and
rotation with their gradients, rows in 4 bits, and decode over such rows. Values are bf16 bit
patterns (uint16) or float64 arrays; written from the definitions in include/gqa.h."""
import numpy as np

import gqa_inputs as gi


def f64(bits):
    return gi.bf16_bits_to_f32(np.ascontiguousarray(bits)).astype(np.float64).reshape(np.shape(bits))


def bf16_bits(x):
    """float32 values to bf16 bits, to nearest even (NaN stays NaN)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


# ---------------------------------------------------------------- plan
def plan(held, keep, new, table, free, count, page, num_pages, max_tokens):
    """(after, cu, positions, slots, table, free, count); None if the step is refused."""
    table, free = table.copy(), free.copy()
    S, max_pages = table.shape
    pages = lambda n: -(-n // page)
    held, new = [int(x) for x in held], [int(x) for x in new]
    keep = held if keep is None else [int(x) for x in keep]
    for h, k, n in zip(held, keep, new):
        if not (0 <= h <= max_pages * page and 0 <= k <= h and n >= 0 and k + n <= max_pages * page):
            return None
    after = [k + n for k, n in zip(keep, new)]
    stack = list(free[:count])
    if sum(new) > max_tokens or not 0 <= count <= len(free):
        return None
    for s in range(S):
        stack += [table[s, i] for i in range(pages(after[s]), pages(held[s]))]
    for s in range(S):
        for i in range(pages(held[s]), pages(after[s])):
            if not stack:
                return None
            table[s, i] = stack.pop()
    if len(stack) > len(free):
        return None
    free[:len(stack)] = stack
    pos, slots = np.zeros(max_tokens, np.int32), np.full(max_tokens, -1, np.int32)
    t = 0
    for s in range(S):
        for j in range(new[s]):
            p = keep[s] + j
            pg = table[s, p // page]
            pos[t], slots[t] = p, pg * page + p % page if 0 <= pg < num_pages else -1
            t += 1
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return np.array(after, np.int32), cu, pos, slots, table, free, len(stack)


# ---------------------------------------------------------------- norm and rotation
def angles(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** -(np.arange(rot // 2) * 2.0 / rot)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def turn(x, cos, sin, interleaved):
    """R x over the last axis; cos and sin broadcast over [..., rot/2] (None: x)."""
    if cos is None:
        return x
    h = cos.shape[-1]
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, w, eps, cos, sin, interleaved):
    """(z, size of the terms each element of z is the sum of)."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    z = turn(y, cos, sin, interleaved)
    if cos is None:
        return z, np.abs(y)
    return z, _pair_size(y, cos, interleaved)


def _pair_size(y, cos, interleaved):
    """|a| + |b| for both elements of a pair, |y| elsewhere."""
    h = cos.shape[-1]
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    m = np.abs(y)
    m[..., a] = m[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return m


def norm_rope_bwd(dz, x, w, eps, cos, sin, interleaved):
    """(dx, dw, size of dx's terms, size of dw's terms) for rows along the last axis."""
    g = turn(dz, cos, None if sin is None else -sin, interleaved)
    gs = _pair_size(dz, cos, interleaved) if cos is not None else np.abs(dz)
    if w is None:
        return g, None, gs, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, e = x * r, g * w
    es = gs * np.abs(w)
    axes = tuple(range(x.ndim - 1))
    return (r * (e - n * (e * n).mean(-1, keepdims=True)), (g * n).sum(axes),
            r * (es + np.abs(n) * (es * np.abs(n)).mean(-1, keepdims=True)), (gs * np.abs(n)).sum(axes))


# ---------------------------------------------------------------- rows in 4 bits
def kv4_pack(bits):
    """bf16 bits [..., D] -> uint8 [..., D/2 + 4]."""
    x = gi.bf16_bits_to_f32(np.ascontiguousarray(bits)).reshape(bits.shape)
    with np.errstate(all="ignore"):
        m = x.min(-1, keepdims=True)
        span = (x.max(-1, keepdims=True) - m).astype(np.float32)
        s_bits = bf16_bits(span / np.float32(15))
        m_bits = bf16_bits(m)
        bad = ~(span < np.inf)
        s_bits[bad] = m_bits[bad] = 0x7FC0
        s = gi.bf16_bits_to_f32(s_bits).reshape(s_bits.shape)
        s_bits[s < 2.0 ** -126] = 0
        inv = np.where(s >= 2.0 ** -126, np.float32(1) / s, np.float32(0)).astype(np.float32)
        code = np.rint((x - m).astype(np.float64) * inv.astype(np.float64))
        code = np.where(bad, 0, code).astype(np.uint8)
    head = np.concatenate([s_bits, m_bits], -1).astype(np.uint16).view(np.uint8)
    return np.concatenate([code[..., 0::2] | (code[..., 1::2] << 4), head], -1), bad[..., 0]


def kv4_parts(rows):
    """(codes, steps, minima) of packed rows, float64."""
    head = np.ascontiguousarray(rows[..., -4:]).view(np.uint16)
    c = rows[..., :-4]
    codes = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (2 * c.shape[-1],)).astype(np.float64)
    h = f64(head)
    return codes, h[..., :1], h[..., 1:]


def kv4_values(rows):
    c, s, m = kv4_parts(rows)
    return c * s + m


# ---------------------------------------------------------------- decode over 4-bit rows
def decode_kv4(q, k_pool, v_pool, lens, table, window=0, scale=None):
    """(o, largest error a right kernel can make) of q [B, Hq, Tq, D] bf16 bits, pools uint8.

    Error: the output's rounding to bf16, 2^-8 of it. The rounding of w = p * s to fp16, 2^-11 of
    sum w |code - 8| (the codes are summed about 8). fp32 sums of w * code: one rounding each 16
    keys, 2^-24 of at most 15 sum w, so 2^-10 of sum w up to 16000 keys. Scores: products of
    codes are exact and eight fp32 sums of 16 of them are off by 2^-21 * scale * s * 15 sum|q|, under
    2^-15 for these inputs, and the exponentials by 2^-21 more: 2^-13 of sum p |v|."""
    q = f64(q)
    B, Hq, Tq, D = q.shape
    pages, Hkv, page, _ = k_pool.shape
    scale = D ** -0.5 if scale is None else scale
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        at = table[b, np.arange(L) // page]
        ok = (at >= 0) & (at < pages)
        rows = lambda pool: np.where(ok[:, None, None], pool[np.where(ok, at, 0), :, np.arange(L) % page], 0)
        kr, vr = rows(k_pool).astype(np.uint8), rows(v_pool).astype(np.uint8)  # [L, Hkv, bytes]
        k = kv4_values(kr)
        vc, vs, vm = kv4_parts(vr)
        for a in range(Hq):
            h = a // (Hq // Hkv)
            for i in range(Tq):
                pos = L - Tq + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0:
                    continue
                see = slice(lo, pos + 1)
                sc = k[see, h] @ q[b, a, i] * scale
                p = np.exp(sc - sc.max())
                p /= p.sum()
                v = vc[see, h] * vs[see, h] + vm[see, h]
                out[b, a, i] = p @ v
                tol[b, a, i] = (2.0 ** -8 * np.abs(out[b, a, i]) + 2.0 ** -11 * (p @ (vs[see, h] * np.abs(vc[see, h] - 8)))
                                + 2.0 ** -10 * (p @ vs[see, h]) + 2.0 ** -13 * (p @ np.abs(v)))
    return out, tol
