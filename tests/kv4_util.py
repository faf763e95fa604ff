"""Plain 64-bit restatements of the rotary positions and of the 4-bit cache,
for the tests: torch on whatever device the inputs are on, no product code."""
import ctypes
import math

import torch

GROUP = 64


def longs(*values):
    """A C array of long long, as the strides of the C calls."""
    return (ctypes.c_longlong * len(values))(*values)


def rotary(x, positions, inv_freq, interleaved, amplitude, inverse=False):
    """x [B, H, N, d] -> float64, pairs turned by positions * inv_freq."""
    y = x.double().clone()
    rot = 2 * inv_freq.numel()
    ang = positions.double().reshape(-1, 1, x.shape[2], 1) * inv_freq.double()
    c, s = torch.cos(ang) * amplitude, torch.sin(ang) * amplitude * (-1 if inverse else 1)
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    xa, xb = y[..., a], y[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def word_places(d, value):
    """Place of each 8-channel word of a row."""
    w = range(d // 8)
    return [(i % 8) * (d // 64) + i // 8 if value else (i % 4) * (d // 32) + i // 4 for i in w]


def quantise(x):
    """(codes, scale, lowest) of x [..., d] bf16; float64, groups of 64."""
    z = x.double().unflatten(-1, (-1, GROUP))
    lo = z.amin(-1)
    span = z.amax(-1) - lo
    frac, exp = torch.frexp(span / 15.0)
    unit = torch.exp2(torch.clamp(exp - 8, min=-133).double())  # bf16 steps, subnormal ones too
    scale = torch.ceil(span / 15.0 / unit) * unit
    n = torch.floor((z - lo[..., None]) / scale.clamp_min(1e-300)[..., None] + 0.5)
    n = torch.where(scale[..., None] > 0, n.clamp(0, 15), torch.zeros_like(n))
    return n, scale, lo


def dequantised(x):
    """float64 values that x [..., d] has once it went through the cache."""
    n, scale, lo = quantise(x)
    return (lo[..., None] + scale[..., None] * n).flatten(-2)


def tiles_of(k, v):
    """Tile bytes [16-token blocks, 18 d] of one head's keys and values [tokens, d]
    (tokens a multiple of 16)."""
    d = k.shape[-1]
    parts = []
    for x, value in ((k, False), (v, True)):
        n, scale, lo = quantise(x)
        n = n.flatten(-2).to(torch.uint8)
        words = (n[:, 0::2] | (n[:, 1::2] << 4)).reshape(-1, d // 8, 4)
        code = torch.empty_like(words)
        code[:, torch.tensor(word_places(d, value), device=x.device)] = words
        par = torch.stack([scale, lo], -1).to(torch.bfloat16).reshape(-1, d // 32)
        parts += [code.reshape(-1, 16 * d // 2), par.view(torch.uint8).reshape(-1, 16 * d // 16)]
    return torch.cat(parts, 1)


def read_tiles(tiles, d):
    """(keys, values, half ranges of the values) float64 [tokens, d] of tile bytes."""
    out, at = [], 0
    for value in (False, True):
        code = tiles[:, at:at + 8 * d].reshape(-1, d // 8, 4)
        par = tiles[:, at + 8 * d:at + 9 * d].contiguous().view(torch.bfloat16)
        par = par.reshape(-1, d // 64, 2).double().repeat_interleave(GROUP, 1)
        at += 9 * d
        words = code[:, torch.tensor(word_places(d, value), device=tiles.device)].reshape(-1, d // 2)
        n = torch.stack([words & 15, words >> 4], -1).reshape(-1, d).double()
        out.append(par[..., 1] + par[..., 0] * n)
        out.append(8.0 * par[..., 0].abs())
    return out[0], out[2], out[1], out[3]


def attention(q, cache, table, lengths, cu, causal, scale, rounded=False):
    """O, LSE in 64 bits and the largest errors the kernel's roundings allow.

    Where each term of the bounds comes from (u = half a step, eps / 2):
      * scores: fp32 sums of at most 128 products of a code with q and a few
        more operations: 2^-17 of the sum of the terms' sizes, eta; it moves P by
        the same relative amount;
      * P s in fp16: 2^-11 of P times at most 15 s a key, and, below fp16's
        smallest normal number, 2^-25 of the largest 15 s a key, twice that if s is
        half its reference (the sum of P is at least 1 at that scale);
      * the output's type: u |O|;
      * `rounded`: keys and values go through fp16, 2^-11 of themselves, or, below
        its smallest normal number in units of 2^7 of the tile's largest, 2^-18 of
        the largest: scores by 2^-11 of the sum of their terms' sizes and 2^-18 of
        the largest key times the sum of q, the output by the same shares of V.
    """
    T, H, d = q.shape
    pages, G, blocks, _ = cache.shape
    ps = blocks * 16
    o = torch.full((T, H, d), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), float("nan"), dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    u = torch.finfo(q.dtype).eps / 2
    for b in range(len(lengths)):
        first, last, n = int(cu[b]), int(cu[b + 1]), int(lengths[b])
        new = last - first
        if not new:
            continue
        for h in range(G):
            if n:
                tiles = cache[table[b, :-(-n // ps)].long(), h].reshape(-1, 18 * d)
                k, v, k8, v8 = (x[:n] for x in read_tiles(tiles, d))
            rows = slice(h * (H // G), (h + 1) * (H // G))
            qq = q[first:last, rows].double().reshape(-1, d)
            see = torch.full((new,), n, device=q.device)
            if causal:
                see = (n - new + 1 + torch.arange(new, device=q.device)).clamp(0, n)
            see = see.repeat_interleave(H // G)
            if not n:
                oo, ll = torch.zeros_like(qq), torch.full_like(qq[:, 0], -math.inf)
                to, tl = torch.zeros_like(qq), torch.zeros_like(ll)
            else:
                hidden = torch.arange(n, device=q.device) >= see[:, None]
                s = (qq @ k.T * scale).masked_fill(hidden, -math.inf)
                ll = torch.logsumexp(s, 1)
                p = torch.exp(s - torch.where(see > 0, ll, 0.0)[:, None]).masked_fill(hidden, 0.0)
                vz = torch.where(hidden.all(0)[:, None], 0.0, v)
                oo = p @ vz
                size = (qq.abs() @ (k.abs() + 2 * k8).T * abs(scale)).masked_fill(hidden, 0.0)
                eta = 2.0 ** -17 * size.amax(1, keepdim=True)
                if rounded:
                    eta = eta + 2.0 ** -11 * size.amax(1, keepdim=True) + \
                        2.0 ** -18 * k.abs().amax() * qq.abs().sum(1, keepdim=True) * abs(scale)
                v8 = torch.where(hidden.all(0)[:, None], 0.0, v8)
                to = (u * oo.abs() + 2.0 ** -11 * (p @ v8) * 15 / 8 + n * 2.0 ** -24 * v8.amax() * 15 / 8 +
                      eta * (p @ vz.abs() + oo.abs()) + 2.0 ** -20 * (p @ (vz.abs() + v8)))
                if rounded:
                    to = to + 2.0 ** -11 * (p @ vz.abs()) + 2.0 ** -18 * vz.abs().amax()
                tl = eta[:, 0] + 2.0 ** -20 + 2.0 ** -22 * ll.abs()
            shape = (new, H // G)
            o[first:last, rows] = oo.reshape(*shape, d)
            lse[first:last, rows] = ll.reshape(shape)
            tol_o[first:last, rows] = to.reshape(*shape, d)
            tol_l[first:last, rows] = tl.reshape(shape)
    return o, lse, tol_o, tol_l


def plan(lengths, new_lengths, table, ring, head, tail, page, max_tokens):
    """The plan of a step on plain lists: (lengths, head, tail, cu, slots, positions,
    status); table and ring are changed in place."""
    width, size = len(table[0]), len(ring)
    status = 0
    ok_len = all(0 <= n <= width * page for n in list(lengths) + list(new_lengths))
    pages = lambda n: -(-n // page)  # noqa: E731
    rows = [(o, n) for o, n in zip(lengths, new_lengths)
            if 0 <= o <= width * page and 0 <= n <= width * page]
    need = sum(max(0, pages(n) - pages(o)) for o, n in rows)
    back = sum(max(0, pages(o) - pages(n)) for o, n in rows)
    grow = sum(max(0, n - o) for o, n in rows)
    status += 1 if need > tail - head else 0
    status += 2 if grow > max_tokens else 0
    status += 0 if ok_len else 4
    status += 8 if head < 0 or tail < head or tail - head > size or tail - head + back > size else 0
    cu, slots, positions = [0], [], []
    if status:
        return (list(lengths), head, tail, [0] * (len(lengths) + 1), [-1] * max_tokens,
                [0] * max_tokens, status)
    for b, (o, n) in enumerate(zip(lengths, new_lengths)):
        for i in range(pages(o), pages(n)):
            table[b][i] = ring[head % size]
            head += 1
        for i in range(pages(n), pages(o)):
            ring[tail % size] = table[b][i]
            tail += 1
        for pos in range(o, n):
            positions.append(pos)
            slots.append(table[b][pos // page] * page + pos % page)
        cu.append(len(slots))
    pad = max_tokens - len(slots)
    return (list(new_lengths), head, tail, cu, slots + [-1] * pad, positions + [0] * pad, 0)
