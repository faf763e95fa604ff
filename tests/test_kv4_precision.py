"""What a row of the attention over the 4-bit cache may depend on: the tokens that it
sees, each to its own precision.  Tokens behind a row's limit change none of its bits,
and a large token or a large group of 64 channels takes none from the others."""
import math

import pytest
import torch

from exact_attention_117_b200 import fa
import kv4_util as ref
from test_kv4_attention import Case

# d, heads, kv heads, page, lengths, new tokens; rows a kv head below 48 (d = 64: 80) go to the
# mma kernel in 1 to 4 tiles of 8, others to the tcgen05 kernel
MMA = [
    (128, 4, 2, 16, [90], [3]),
    (128, 8, 2, 16, [300], [4]),
    (64, 8, 2, 32, [500], [5]),
    (128, 8, 1, 16, [260], [5]),
    (64, 4, 1, 64, [1100], [19]),
]
TCGEN = [
    (128, 8, 2, 16, [150], [50]),
    (64, 16, 2, 32, [700], [60]),
    (128, 4, 4, 64, [600], [300]),
    (64, 1, 1, 16, [400], [400]),
]


def on_tcgen(c):
    rows = c.most * (c.q.shape[1] // c.cache.shape[1])
    return rows >= (80 if c.d == 64 else 48)


def parameters(c, value):
    """A view of the cache's K or V parameters: bf16 [pages, kv heads, blocks, 16, groups, 2]."""
    at = (17 if value else 8) * c.d
    return c.cache[..., at:at + c.d].view(torch.bfloat16).unflatten(-1, (16, c.d // 64, 2))


def token(c, value, b, i):
    """Token i of request b in that view: [kv heads, groups, 2]."""
    slot = int(c.table[b, i // c.page]) * c.page + i % c.page
    return parameters(c, value)[slot // c.page, :, slot % c.page // 16, slot % 16]


def opposed(c, b, i, size):
    """Token i of request b gets the keys -size, size, -size, ... (size a multiple of
    15 / 4 by a power of two): the code bytes f0 whatever the order of the words."""
    slot = int(c.table[b, i // c.page]) * c.page + i % c.page
    rows = c.cache[slot // c.page, :, slot % c.page // 16, :8 * c.d].unflatten(-1, (16, -1))
    rows[:, slot % 16] = 0xf0
    token(c, False, b, i).copy_(torch.tensor([size * 2 / 15, -size], device="cuda"))


def balanced(c, least):
    """Queries of which every even channel is positive, every odd one negative."""
    c.q.abs_().clamp_min_(least)
    c.q[..., 1::2] *= -1


def attend(c, causal=True, scale=None):
    out = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=c.most, causal=causal, scale=scale)
    fa.check_device_error()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("shape", MMA + TCGEN, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
@pytest.mark.parametrize("value", [False, True], ids=["key", "value"])
def test_rows_do_not_depend_on_tokens_they_do_not_see(shape, value):
    """One of a request's new tokens grows by powers of two up to the largest floats,
    then its lowest values become infinite and no number: the rows before it keep
    every bit."""
    c = Case(*shape, seed=61)
    n, new = shape[4][0], shape[5][0]
    clean = c.cache.clone()
    want = attend(c)
    for query in (1, new // 2, new - 1):
        for power in (10, 20, 60, 122, "inf", "nan"):
            c.cache.copy_(clean)
            t = token(c, value, 0, n - new + query)
            if isinstance(power, str):
                t[..., 1] = float(power)
            else:
                t.mul_(2.0 ** power)
            o, lse = attend(c)
            assert torch.equal(o[:query], want[0][:query]), (query, power)
            assert torch.equal(lse[:query], want[1][:query]), (query, power)


def check(c, o, lse, causal=True, scale=None):
    """O and LSE against the definition in 64 bits, each row and group of channels to
    what its own keys allow.

    Terms (half a step: 2^-8 bf16, 2^-11 fp16, 2^-24 fp32; p: the row's weights):
      * scores, both kernels: fp32 sums of products, 2^-17 of their sizes;
      * scores, tcgen05: K is lowest, rounded to fp16, plus scale n, rounded to
        fp16: in each channel at most 2^-11 of |k|, independent of each other, and
        in each group of 64 at most 2^-11 of |lowest|, the same in all its
        channels.  Independent errors of at most b_i sum up to more than six times
        the root of the sum of b_i^2 once in 10^7;
      * P: mma 2^-11 of p times 15 steps of the key's group, below fp16's normal
        numbers 2^-25 in a unit that brings the largest P s so far to 8 at least;
        tcgen05 2^-11 of p |v|, or 2^-25 where the largest is 1; in the last
        tiles, with keys that some rows do not see, that of 2^9 times a unit of
        2^-8 of the largest |v| seen;
      * V, tcgen05: 2^-11 of |lowest| and of |v|, and 2^-33 of the largest seen (in
        units that bring that one to 2^8 at least), twice;
      * O: its rounding (2^-25 where fp16 holds it as a subnormal number, below
        2^-14), and 2^-20 of its terms for fp32 sums.
    """
    d, tc = c.d, on_tcgen(c)
    scale = d ** -0.5 if scale is None else scale
    u = torch.finfo(c.q.dtype).eps / 2
    T, H, _ = c.q.shape
    G = c.cache.shape[1]
    groups = lambda x: x.unflatten(-1, (-1, 64))  # noqa: E731
    for b, n in enumerate(c.lens.tolist()):
        first, last = int(c.cu[b]), int(c.cu[b + 1])
        new = last - first
        for h in range(G if n and new else 0):
            tiles = c.cache[c.table[b, :-(-n // c.page)].long(), h].reshape(-1, 18 * d)
            k, v, k8, v8 = (x[:n] for x in ref.read_tiles(tiles, d))
            par = tiles[:, 8 * d:9 * d].contiguous().view(torch.bfloat16).reshape(-1, d // 64, 2)[:n].double()
            klo = par[..., 1]
            vlo = tiles[:, 17 * d:].contiguous().view(torch.bfloat16).reshape(-1, d // 64, 2)[:n].double()[..., 1]
            heads = slice(h * (H // G), (h + 1) * (H // G))
            q = c.q[first:last, heads].double().reshape(-1, d)
            see = torch.full((new,), n, device="cuda")
            if causal:
                see = (n - new + 1 + torch.arange(new, device="cuda")).clamp(0, n)
            see = see.repeat_interleave(H // G)
            got_o = o[first:last, heads].double().reshape(-1, d)
            got_l = lse[first:last, heads].double().reshape(-1)
            assert not got_o[see == 0].any() and (got_l[see == 0] == -math.inf).all()
            q, got_o, got_l, see = q[see > 0], got_o[see > 0], got_l[see > 0], see[see > 0]
            hidden = torch.arange(n, device="cuda") >= see[:, None]
            seen = (~hidden).double()
            s = (q @ k.T * scale).masked_fill(hidden, -math.inf)
            ll = torch.logsumexp(s, 1)
            p = torch.exp(s - ll[:, None]).masked_fill(hidden, 0.0)
            eta = 2.0 ** -17 * (q.abs() @ (k.abs() + 2 * k8).T) * abs(scale)
            if tc:
                lows = (groups(q).sum(-1) ** 2) @ (klo ** 2).T
                eta = eta + 6 * 2.0 ** -11 * torch.sqrt((q ** 2) @ (k ** 2).T + lows) * abs(scale)
            eta = eta.masked_fill(hidden, 0.0)
            # scores off by at most eta: sum p' v - o = sum p (e^delta - 1) (v - o) / sum p e^delta
            pe = p * torch.expm1(eta)
            assert float(pe.sum(1).max()) < 0.1  # (a wider bound would say little)
            pe = pe / (1 - pe.sum(1, keepdim=True))
            tl = -torch.log1p(-(p * torch.expm1(eta)).sum(1)) + 2.0 ** -20 + 2.0 ** -22 * ll.abs()
            oo = p @ v
            spans = v8 * 15 / 8
            tiny = 2.0 ** -25 if c.q.dtype == torch.float16 else 0.0
            to = (u * oo.abs()).clamp_min(tiny) + pe @ v.abs() + pe.sum(1, keepdim=True) * oo.abs() + 2.0 ** -20 * (p @ (v.abs() + spans))
            most = p.amax(1, keepdim=True)
            if tc:
                low = vlo.abs().repeat_interleave(64, 1)
                to = to + 2.0 ** -11 * (p @ (2 * v.abs() + low)) + 2.0 ** -25 * most * (seen @ v.abs())
                top = torch.stack([(v.abs().amax(1) * seen[i]).amax() for i in range(len(seen))])[:, None]
                late = min(n, n - int(see[0]) + 128) if int(see[0]) < n else 0
                to = to + (late * most * 2.0 ** -24 + 2.0 ** -32) * top
            else:
                step = groups(spans)[..., 0]  # 15 scales of each key and group
                big = (p[:, :, None] * step[None]).amax(1).repeat_interleave(64, 1)
                to = to + 2.0 ** -11 * (p @ spans) + n * 2.0 ** -28 * big
            over = ((got_o - oo).abs() / to.clamp_min(1e-300)).amax()
            assert ((got_o - oo).abs() <= to).all(), f"O off by {float(over):.2f} of the bound"
            over = ((got_l - ll).abs() / tl).amax()
            assert ((got_l - ll).abs() <= tl).all(), f"LSE off by {float(over):.2f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [4, 64], ids=["mma", "tcgen05"])
@pytest.mark.parametrize("ratio", [0, 10, 16])
@pytest.mark.parametrize("keys", [1, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_groups_of_unlike_sizes_keep_their_bits(heads, ratio, keys, dtype):
    """The second 64 channels are 2^-ratio of the first in K and V, and q's are that
    much larger in turn: each group counts alike in the scores, and O's groups are
    held to their own sizes."""
    c = Case(128, heads, 1, 16, [keys] * 9, [1] * 9, dtype=dtype, seed=62 + ratio)
    for value in (False, True):
        parameters(c, value)[..., 1, :] *= 2.0 ** -ratio
    c.q[..., 64:] *= 2.0 ** (ratio / 2)
    c.q[..., :64] *= 2.0 ** -(ratio / 2)
    o, lse = attend(c, scale=2.0 ** (ratio / 2) / math.sqrt(128))
    check(c, o, lse, scale=2.0 ** (ratio / 2) / math.sqrt(128))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(128, 4, 1, 16, [1000, 90], [1, 3]), (64, 8, 2, 16, [600], [4]),
                                   (128, 16, 2, 32, [700], [5]), (128, 16, 2, 16, [1000, 200], [8, 60]),
                                   (64, 32, 2, 64, [900], [40])],
                         ids=["mma128", "mma64", "mma128x5", "tcgen128", "tcgen64"])
@pytest.mark.parametrize("power", [8, 12, 16, 20])
def test_a_large_token_of_no_weight_takes_no_bits(shape, power):
    """A token that all rows see has values 2^power larger than all others and a
    weight of e^-30 and less: O stays as exact as the others' values are."""
    c = Case(*shape, seed=63)
    balanced(c, 0.6)
    c.q *= 2.0  # the large tokens' scores: below -3.75 * 1.2 * sqrt(d)
    for b in range(len(shape[4])):
        for at in (33, 70):
            opposed(c, b, at, 3.75)
            token(c, True, b, at).mul_(2.0 ** power)
    check(c, *attend(c))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [4, 64], ids=["mma", "tcgen05"])
def test_a_large_key_takes_no_bits_from_its_tile(heads):
    """Every eighth token's keys are 2^12 larger and opposed to the queries (no weight):
    the others' scores keep their precision."""
    c = Case(128, heads, 1, 16, [300, 64], [1, 1], seed=64)
    balanced(c, 0.1)
    for b, n in enumerate((300, 64)):
        for at in range(5, n, 8):
            opposed(c, b, at, 3840.0)
    check(c, *attend(c))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [4, 64], ids=["mma", "tcgen05"])
def test_values_and_keys_near_the_ends_of_the_floats(heads):
    """One key: O is its value and LSE its score, from 2^-90 to 2^120."""
    for power in (-90, -40, 60, 100, 120):
        c = Case(128, heads, 1, 16, [1] * 5, [1] * 5, seed=65)
        parameters(c, True).mul_(2.0 ** power)
        check(c, *attend(c))
        c = Case(128, heads, 1, 16, [1] * 5, [1] * 5, seed=65)
        parameters(c, False).mul_(2.0 ** power)
        c.q *= 2.0 ** -(power - power % 2) * 2.0 ** -(power % 2)
        check(c, *attend(c))
