"""Attention over the paged 4-bit cache against the 64-bit definition, and the
whole serving step: plan, rotary, append, attention."""
import math
import random

import pytest
import torch

from exact_attention_117_b200 import fa
import kv4_util as ref

P = 0x10000


def _raw(q=P, cache=P, table=P, lens=P, cu=P, o=P, lse=P, R=2, T=3, H=4, G=2, d=64, pages=5, page=16,
         width=3, stride=3, strides=(256, 64, 256, 64), most=2, scale=0.1, dtype=0, ws=P, size=None):
    lib = fa.load()
    if size is None:
        size = lib.fa_kv4_attention_workspace_size(max(H, 1), max(G, 1), 64, max(most, 1)) or 1 << 30
    return lib.fa_kv4_attention(q, cache, table, lens, cu, o, lse, R, T, H, G, d, pages, page, width,
                                stride, ref.longs(*strides), most, 1, scale, dtype, ws, size, None)


def test_refusals():
    from exact_attention_117_b200 import build
    build.build()
    for name in ("q", "cache", "table", "lens", "cu", "o", "lse"):
        assert _raw(**{name: None}) == 1, name
    for bad in (dict(R=0), dict(T=-1), dict(H=0), dict(G=0), dict(H=3), dict(pages=0), dict(page=8),
                dict(page=17), dict(width=0), dict(stride=2), dict(most=0), dict(dtype=2),
                dict(width=1 << 28, stride=1 << 28), dict(T=1 << 30)):
        assert _raw(**bad) == 2, bad
    for d in (0, 32, 96, 256):
        assert _raw(d=d) == 3
    for bad in (dict(q=P + 8), dict(cache=P + 4), dict(o=P + 2), dict(lse=P + 2), dict(lens=P + 1),
                dict(strides=(256, 60, 256, 64)), dict(strides=(256, 64, -256, 64)), dict(ws=P + 8)):
        assert _raw(**bad) == 4, bad
    for scale in (math.nan, math.inf):
        assert _raw(scale=scale) == 5
    need = fa.load().fa_kv4_attention_workspace_size(4, 2, 64, 2)
    assert need > 0 and _raw(ws=None) == 6 and _raw(size=need - 1) == 6
    assert _raw(T=0) == 0 and _raw(T=0, q=None, o=None, lse=None) == 0
    size = fa.load().fa_kv4_attention_workspace_size
    assert size(4, 3, 64, 1) == 0 and size(4, 2, 80, 1) == 0 and size(4, 2, 64, 0) == 0


def test_binding_refuses():
    c = torch.zeros(4, 2, 1, 18 * 64, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    tab, ln, cu = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for args in ((q.float(), c, tab, ln, cu), (q[:, :3], c, tab, ln, cu), (q, c[:, :, :, :100], tab, ln, cu),
                 (q, c, tab.long(), ln, cu), (q, c, tab[0], ln, cu), (q, c, tab, ln[:1], cu),
                 (q, c, tab, ln, cu[:2]), (q.transpose(1, 2), c, tab, ln, cu)):
        with pytest.raises(ValueError):
            fa.kv4_attention(*args, max_tokens=1)


class Case:
    """A cache filled through the definition (not the product), pages shuffled."""

    def __init__(self, d, H, G, page, lens, new, dtype=torch.bfloat16, seed=0, q_mult=1.0, extra=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width = max(1, max(-(-n // page) for n in lens)) + 1
        held = [-(-n // page) for n in lens]
        self.pages = sum(held) + extra
        order = torch.randperm(self.pages, generator=g, device="cuda", dtype=torch.int32)
        tab, at = torch.full((len(lens), self.width), -1, dtype=torch.int32, device="cuda"), 0
        for b, h in enumerate(held):
            tab[b, :h] = order[at:at + h]
            at += h
        n = self.pages * page
        k = torch.randn(n, G, d, generator=g, device="cuda") * torch.exp(
            0.5 * torch.randn(d, generator=g, device="cuda"))
        v = torch.randn(n, G, d, generator=g, device="cuda")
        self.cache = torch.stack([ref.tiles_of(k[:, h].bfloat16(), v[:, h].bfloat16()).reshape(
            self.pages, page // 16, 18 * d) for h in range(G)], 1).contiguous()
        self.table, self.page, self.d = tab, page, d
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().cuda()
        self.q = (torch.randn(sum(new), H, d, generator=g, device="cuda") * q_mult).to(dtype)
        self.most = max(max(new), 1)

    def check(self, causal=True, scale=None, most=None, **kw):
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        o, lse = fa.kv4_attention(self.q, self.cache, self.table, self.lens, self.cu,
                                  max_tokens=most or self.most, causal=causal, scale=scale, **kw)
        fa.check_device_error()
        group = self.q.shape[1] // self.cache.shape[1]
        # (many rows go to the tcgen05 kernel, whose keys and values are fp16)
        self.compare(o, lse, causal, scale, (most or self.most) * group >= (80 if self.d == 64 else 48))
        return o, lse

    def compare(self, o, lse, causal, scale, rounded=False):
        wo, wl, to, tl = ref.attention(self.q, self.cache, self.table, self.lens.tolist(),
                                       self.cu.tolist(), causal, scale, rounded)
        T = int(self.cu[-1])
        o, lse, wo, wl, to, tl = o[:T].double(), lse[:T].double(), wo[:T], wl[:T], to[:T], tl[:T]
        empty = wl == -math.inf
        assert torch.equal(lse == -math.inf, empty) and not o[empty].any()
        assert ((o - wo).abs() <= to).all(), f"O off by {float(((o - wo).abs() - to).max()):.3e} too much"
        err = (lse - wl).abs()[~empty]
        assert (err <= tl[~empty]).all(), f"LSE off by {float((err - tl[~empty]).max()):.3e} too much"


SHAPES = [
    # d, heads, kv heads, page, lengths, new tokens
    (64, 1, 1, 16, [1], [1]),
    (128, 8, 8, 16, [17], [1]),
    (128, 4, 1, 64, [16, 1, 300], [1, 1, 1]),
    (64, 16, 2, 32, [1000, 0, 33, 1], [1, 1, 0, 1]),
    (128, 32, 4, 128, [129, 2000, 5], [1, 1, 1]),
    (64, 5, 1, 48, [100, 47, 49], [3, 1, 2]),
    (128, 14, 2, 16, [65, 64, 63], [2, 5, 1]),
    (64, 24, 8, 16, [777], [7]),
    (128, 3, 3, 64, [500, 20], [33, 20]),
    (64, 32, 1, 64, [90, 4096], [1, 2]),
    (128, 8, 2, 16, [260, 130], [260, 130]),
    (64, 2, 1, 16, [7, 3], [10, 9]),        # more queries than keys: rows that see nothing
    # 48 rows (d = 64: 80) and more: the tcgen05 kernel
    (128, 64, 1, 16, [1], [1]),
    (64, 1, 1, 64, [84, 0, 700], [84, 0, 85]),
    (64, 20, 5, 64, [100, 19], [19, 1]),     # 76 rows: still the other one
    (128, 1, 1, 16, [257], [257]),
    (128, 4, 2, 48, [1000, 129, 2049], [33, 129, 1]),
    (64, 6, 2, 16, [2000, 31], [100, 300]),  # rows that see nothing
    (64, 16, 2, 128, [5000], [500]),
    (128, 24, 8, 32, [300, 77, 1500, 2], [300, 50, 64, 2]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_definition(shape, dtype, causal):
    Case(*shape, dtype=dtype, seed=len(shape[4])).check(causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,G,R", [(128, 32, 8, 1), (64, 16, 16, 2), (128, 8, 1, 300)])
def test_long_and_many(d, H, G, R):
    """One long context over many CTAs, and more requests than threads of a block."""
    rng = random.Random(R)
    lens = [20011] * R if R < 3 else [rng.randint(0, 90) for _ in range(R)]
    Case(d, H, G, 64 if R < 3 else 16, lens, [1] * R, seed=R).check()


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,G,new", [(128, 8, 4, 1), (64, 4, 2, 3), (128, 8, 2, 20), (64, 4, 1, 30)])
def test_many_uneven_jobs(d, H, G, new):
    """More jobs than CTAs, of unlike lengths and some without a key, so that ranges
    begin and end anywhere in them."""
    rng = random.Random(d + new)
    lens = [rng.choice([0, 1, 5, 17, 255, 256, 257, 300, 900, 2000]) for _ in range(170)]
    lens[40:44] = [6000, 0, 0, 0]
    Case(d, H, G, 16, lens, [rng.choice([0, 1, new]) for _ in lens], seed=new).check(most=new)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 64])
def test_a_long_context_keeps_its_small_output(heads):
    """Half a million keys of nearly equal weight: O is their values' mean, two hundred
    times smaller than they are, and still off by little more than its rounding (bf16
    2^-8 at most, 2^-9.2 in root mean square; P in fp16 adds at most 2^-11 of 15 s a
    key, of either sign: below 2^-11 of O)."""
    c = Case(64, heads, 1, 64, [500_000], [1], seed=50, q_mult=0.25)
    o, _ = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1)
    tiles = c.cache[c.table[0, :-(-500_000 // 64)].long(), 0].reshape(-1, 18 * 64)
    k, v, _, _ = (x[:500_000] for x in ref.read_tiles(tiles, 64))
    w = torch.softmax(c.q[0].double() @ k.T / 8.0, -1) @ v
    off = float((o[0].double() - w).norm() / w.norm())
    assert off <= 2.0 ** -9, off


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0])
@pytest.mark.parametrize("q_mult", [1.0, 2.0 ** -40, 2.0 ** 30])
def test_scales_and_sizes_of_q(scale, q_mult):
    """Sharp, flat and reversed rows; queries far from 1 (their power of two is split
    off exactly), with the scale that undoes it."""
    c = Case(128, 4, 2, 16, [200, 31], [2, 1], seed=9, q_mult=q_mult)
    c.check(scale=scale / q_mult)


@pytest.mark.gpu
def test_values_of_unlike_sizes():
    """V scales that grow and shrink by 2^60 along the keys, keys that grow."""
    c = Case(64, 4, 1, 16, [320], [4], seed=2)
    par = c.cache[..., 17 * 64:].clone().view(torch.bfloat16)
    mult = torch.exp2(torch.randint(-30, 30, par.shape[:3] + (16, 1), device="cuda").float()).bfloat16()
    c.cache[..., 17 * 64:] = (par.unflatten(-1, (16, -1)) * mult).flatten(-2).view(torch.uint8)
    kp = c.cache[..., 8 * 64:9 * 64].clone().view(torch.bfloat16)
    c.cache[..., 8 * 64:9 * 64] = (kp * 8).view(torch.uint8)
    c.check()


@pytest.mark.gpu
def test_masked_places_may_hold_anything():
    """Rows behind a length, unused pages and table entries, and later tokens of the
    same request hold NaN and infinities."""
    H, d, page = 4, 128, 16
    c = Case(d, H, 2, page, [37, 16, 90], [1, 1, 3], seed=4)
    clean = c.cache.clone()
    want = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=3)
    bad = torch.tensor([0x7f, 0xc0, 0x80, 0x7f], dtype=torch.uint8, device="cuda")  # NaN, infinity
    used = torch.zeros(c.pages * page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens.tolist()):
        for t in range(n):
            used[int(c.table[b, t // page]) * page + t % page] = True
    for at in (8 * d, 17 * d):
        rows = c.cache[..., at:at + d].unflatten(-1, (16, d // 64, 4))
        mask = ~used.reshape(c.pages, 1, 1, 16).expand(rows.shape[:4])
        rows[mask] = bad
    got = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the newest token of the third request is no number: only its own row sees it
    c.cache.copy_(clean)
    slot = int(c.table[2, 89 // page]) * page + 89 % page
    for at in (8 * d, 17 * d):
        c.cache[slot // page, :, slot % page // 16, at:at + d].unflatten(-1, (16, -1))[:, slot % 16] = \
            bad.repeat(d // 64)
    got = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=3)
    assert torch.equal(got[0][:4], want[0][:4]) and torch.equal(got[1][:4], want[1][:4])
    assert got[0][4].isnan().all() and got[1][4].isnan().all()
    fa.check_device_error()


@pytest.mark.gpu
def test_no_number_in_seen_places():
    c = Case(64, 2, 2, 16, [40, 40], [1, 1], seed=8)
    c.q[1, 0, 3] = float("nan")
    o, lse = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1)
    assert o[1, 0].isnan().all() and lse[1, 0].isnan()
    assert o[0].isfinite().all() and o[1, 1].isfinite().all() and lse[0].isfinite().all()


@pytest.mark.gpu
def test_max_tokens_only_chooses_the_kernel():
    c = Case(64, 8, 2, 16, [300, 77], [9, 4], seed=6)
    for most in (1, 3, 5, 9, 4000):
        c.check(most=most)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_one_long_request(d):
    """Row tiles cut over many CTAs and joined."""
    Case(d, 4, 1, 64, [9000], [70], seed=30).check()
    Case(d, 8, 8, 64, [3000, 100], [3000, 100], seed=31).check()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0])
@pytest.mark.parametrize("q_mult", [1.0, 2.0 ** -40, 2.0 ** 30])
def test_many_rows_scales_and_sizes_of_q(scale, q_mult):
    c = Case(128, 4, 2, 16, [500, 131], [60, 100], seed=9, q_mult=q_mult)
    c.check(scale=scale / q_mult)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 40])
def test_scores_beyond_all_exponents(new):
    """Scores of 2^40 and more: one key takes each row, or, where the difference to the
    next is lost in 32 bits, some of the largest do; nothing overflows."""
    c = Case(128, 4, 2, 16, [300, 77], [new, new], seed=21)
    for scale in (2.0 ** 40, -(2.0 ** 70)):
        o, lse = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=new, scale=scale)
        fa.check_device_error()
        assert o.isfinite().all() and lse.isfinite().all()
        wl = ref.attention(c.q, c.cache, c.table, c.lens.tolist(), c.cu.tolist(), True, scale)[1]
        # scores from fp16 keys are off by at most 2^-11 of their terms' sizes, here
        # below 2^-3 of the largest score
        assert ((lse.double() - wl).abs() <= 2.0 ** -3 * wl.abs().amax()).all()


@pytest.mark.gpu
def test_many_rows_values_of_unlike_sizes():
    """V's scales grow along the keys by up to 2^20 (O follows the unit of V), then
    shrink; the keys' sizes change from page to page."""
    c = Case(64, 8, 1, 16, [1100], [20], seed=12)
    pages = (1100 + 15) // 16
    for i in range(pages):
        tile = c.cache[int(c.table[0, i])]
        for at, power in ((8 * 64, (i * 7) % 4), (17 * 64, 20 * i // 40 if i < 40 else 20 - (i - 40))):
            par = tile[..., at:at + 64].clone().view(torch.bfloat16)
            tile[..., at:at + 64] = (par * 2.0 ** power).view(torch.uint8)
    c.check()
    c.check(causal=False)


@pytest.mark.gpu
def test_many_rows_masked_places_may_hold_anything():
    H, d, page = 8, 128, 16
    c = Case(d, H, 2, page, [150, 40], [50, 20], seed=14)
    clean = c.cache.clone()
    want = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=50)
    c.compare(*want, True, d ** -0.5, True)
    bad = torch.tensor([0x7f, 0xc0, 0x80, 0x7f], dtype=torch.uint8, device="cuda")  # NaN, infinity
    used = torch.zeros(c.pages * page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens.tolist()):
        for t in range(n):
            used[int(c.table[b, t // page]) * page + t % page] = True
    for at in (8 * d, 17 * d):
        rows = c.cache[..., at:at + d].unflatten(-1, (16, d // 64, 4))
        rows[~used.reshape(c.pages, 1, 1, 16).expand(rows.shape[:4])] = bad
    got = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=50)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # token 130 of the first request (its query 30) is no number, in K and V, then in V
    for places in ((8 * d, 17 * d), (17 * d,)):
        c.cache.copy_(clean)
        slot = int(c.table[0, 130 // page]) * page + 130 % page
        for at in places:
            c.cache[slot // page, :, slot % page // 16, at:at + d].unflatten(-1, (16, -1))[:, slot % 16] = \
                bad.repeat(d // 64)
        got = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=50)
        seen = torch.zeros(70, dtype=torch.bool, device="cuda")
        seen[30:50] = True
        assert torch.equal(got[0][~seen], want[0][~seen]) and torch.equal(got[1][~seen], want[1][~seen])
        assert got[0][seen].isnan().all()
    fa.check_device_error()


@pytest.mark.gpu
def test_many_rows_pages_outside_the_cache_are_reported():
    c = Case(64, 8, 1, 16, [300], [20], seed=15)
    keep = c.table.clone()
    for page in (-1, c.pages, 1 << 30):
        c.table.copy_(keep)
        c.table[0, 3] = page
        o, lse = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=20, causal=False)
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == 10
        left = torch.cat([keep[0, :3], keep[0, 4:19]])
        k, v, _, _ = (x[:284] for x in ref.read_tiles(c.cache[left.long(), 0].reshape(-1, 18 * 64), 64))
        s = c.q.double() @ k.T / 8.0
        # fp16 keys and values, output rounding: a few 2^-9 of values up to 4
        assert (o.double() - torch.softmax(s, -1) @ v).abs().max() <= 2.0 ** -6
        assert (lse.double() - torch.logsumexp(s, -1)).abs().max() <= 2.0 ** -8
    c.table.copy_(keep)
    c.check()


@pytest.mark.gpu
def test_strides_untouched_rows_workspace_and_repeats():
    c = Case(128, 8, 2, 32, [3000, 65], [1, 2], seed=7)
    T, H, d = c.q.shape
    big = torch.full((T + 5, H + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:T, :H] = c.q
    out = torch.full((T + 5, 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 5, H), 7.0, device="cuda")
    ws = torch.full((fa.kv4_attention_workspace_size(H, 2, d, 2) // 4,), float("nan"), device="cuda")
    fa.kv4_attention(big[:, :H], c.cache, c.table, c.lens, c.cu, max_tokens=2, out=out[:, :H],
                     lse=lse, workspace=ws)
    fa.check_device_error()
    c.compare(out[:, :H], lse, True, d ** -0.5)
    assert (out[T:] == 7).all() and (out[:, H:] == 7).all() and (lse[T:] == 7).all()
    a, b = (fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=2) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], out[:T, :H])
    with pytest.raises(fa.FaError):
        fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=2, workspace=ws[:-4])
    e = fa.kv4_attention(c.q[:0], c.cache, c.table, c.lens, c.cu * 0, max_tokens=1)
    assert e[0].shape == (0, H, d)


@pytest.mark.gpu
def test_pages_outside_the_cache_are_reported():
    c = Case(64, 2, 1, 16, [40], [1], seed=3)
    keep = c.table.clone()
    for page in (-1, c.pages, 1 << 30):
        c.table.copy_(keep)
        c.table[0, 1] = page
        o, lse = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1)
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == 10
        fa.check_device_error()
        # the keys of that page count as absent
        k, v, _, _ = ref.read_tiles(c.cache[keep[0, [0, 2]].long(), 0].reshape(-1, 18 * 64), 64)
        k, v = k[:24], v[:24]
        for h in range(2):
            s = c.q[0, h].double() @ k.T / 8.0
            assert (o[0, h].double() - torch.softmax(s, 0) @ v).abs().max() <= 2.0 ** -6
            assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) <= 1e-3
    c.table.copy_(keep)
    c.check()


@pytest.mark.gpu
def test_two_streams_and_a_replayed_graph():
    cases = [Case(128, 8, 2, 16, [500 + 30 * i, 90], [1, 1], seed=20 + i) for i in range(2)]
    want = [fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    c = cases[0]
    out, lse = torch.empty_like(c.q), torch.empty(2, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1, out=out, lse=lse)
    for n in ([500, 90], [1, 0], [333, 17]):
        c.lens.copy_(torch.tensor(n, dtype=torch.int32))
        c.q.copy_(torch.randn_like(c.q.float()))
        graph.replay()
        c.compare(out, lse, True, 128 ** -0.5)
    fa.check_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 40])
def test_what_a_call_on_another_stream_allocates_stays_its_own(new):
    """The call runs on a side stream that is still busy; memory it allocated itself
    (the workspace, here at once free again) is not handed out meanwhile."""
    c = Case(128, 8, 2, 16, [4000, 900], [new, new], seed=41)
    kw = dict(max_tokens=new)
    want = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, **kw)
    size = fa.kv4_attention_workspace_size(8, 2, 128, new)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, stream=side, **kw)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        for _ in range(20):
            for j in junk:
                j.fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del junk


@pytest.mark.gpu
def test_axes_of_length_one_may_have_any_stride():
    c = Case(128, 4, 1, 16, [50], [1], seed=42)
    flat = torch.zeros(4 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((1, 4, 128), (3, 128, 1))
    q.copy_(c.q)
    want = fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=1)
    got = fa.kv4_attention(q, c.cache, c.table, c.lens, c.cu, max_tokens=1)
    assert torch.equal(got[0], want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 64])
def test_one_page_of_more_than_2_to_the_31_bytes(new):
    """A key far behind in a page of its own takes all the weight (its score is
    above 180, all others are 0): O is its value."""
    page, far = 1 << 24, (1 << 24) - 33
    cache = fa.kv4_cache(1, 1, page, 128)
    k = torch.full((1, 1, 128), 4.0, device="cuda").bfloat16()
    v = torch.randn(1, 1, 128, device="cuda").bfloat16()
    fa.kv4_append(k, v, cache, torch.tensor([far], device="cuda"))
    q = k.expand(new, 1, 128).contiguous()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    o, lse = fa.kv4_attention(q, cache, ints(0)[None], ints(page), ints(0, new), max_tokens=new,
                              causal=False)
    _, want = fa.kv4_gather(cache, torch.tensor([far], device="cuda"))
    # bf16's rounding of the value and of O, P's and V's to fp16
    assert torch.allclose(o.float(), want[0].float().expand(new, 1, 128).reshape(o.shape),
                          rtol=2.0 ** -7 + 2.0 ** -10, atol=2.0 ** -9 * float(v.abs().max()))
    assert torch.allclose(lse, torch.full_like(lse, 128 * 16 / math.sqrt(128)), rtol=1e-4)
    fa.check_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,G,page,interleaved", [(128, 8, 2, 64, False), (64, 6, 3, 16, True)])
def test_serving_steps(d, H, G, page, interleaved):
    """Requests that come, grow and go: each step plans its pages, turns q and k,
    appends and attends; the cache a request sees is the one its tokens made."""
    R, width = 4, 6
    rng, g = random.Random(d), torch.Generator(device="cuda").manual_seed(d)
    cache = fa.kv4_cache(R * width, G, page, d)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    ring = torch.randperm(R * width, device="cuda", dtype=torch.int32)
    fr = torch.tensor([0, R * width], device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    f, amp = fa.rotary_frequencies(d, factor=4.0, original_length=64)
    held = [[] for _ in range(R)]  # per request: (key, value) rows as the cache has them
    for step in range(9):
        old = lens.tolist()
        want = [0 if n and rng.random() < 0.15 else min(n + (rng.randint(1, 40) if n == 0 else rng.choice([1, 1, 4])),
                                                        page * width) for n in old]
        room = 170
        plan = fa.kv4_plan(lens, torch.tensor(want, dtype=torch.int32, device="cuda"), table, ring, fr, page,
                           room, lengths_out=lens, free_range_out=fr)
        assert plan.status.item() == 0
        x = torch.randn(room, (H + 2 * G) * d, generator=g, device="cuda").bfloat16()
        q = x[:, :H * d].unflatten(-1, (H, d))
        k, v = (x[:, (H + i * G) * d:(H + (i + 1) * G) * d].unflatten(-1, (G, d)) for i in range(2))
        yq, yk = fa.rotary(q.transpose(0, 1)[None], k.transpose(0, 1)[None], plan.positions, f,
                           interleaved=interleaved, amplitude=amp)
        yq, yk = yq[0].transpose(0, 1), yk[0].transpose(0, 1)
        fa.kv4_append(yk, v, cache, plan.slots)
        o, lse = fa.kv4_attention(yq, cache, table, plan.lengths, plan.cu_tokens, max_tokens=40)
        fa.check_device_error()
        cu = plan.cu_tokens.tolist()
        dk, dv = ref.dequantised(yk), ref.dequantised(v)
        for b in range(R):
            held[b] = held[b][:want[b]]
            for t in range(cu[b], cu[b + 1]):
                held[b].append((dk[t], dv[t]))
            if not held[b]:
                continue
            K, V = (torch.stack([r[i] for r in held[b]]) for i in range(2))
            n, new = want[b], cu[b + 1] - cu[b]
            for i in range(new):
                for h in range(H):
                    s = yq[cu[b] + i, h].double() @ K[:n - new + i + 1, h // (H // G)].T * d ** -0.5
                    p = torch.softmax(s, 0)
                    w = p @ V[:n - new + i + 1, h // (H // G)]
                    # output and P roundings, and 2^-10 of the values for the scores'
                    tol = 2.0 ** -8 * w.abs() + 2.0 ** -9 * (p @ V[:n - new + i + 1, h // (H // G)].abs()) + 2.0 ** -10
                    assert ((o[cu[b] + i, h].double() - w).abs() <= tol).all()
                    assert abs(float(lse[cu[b] + i, h]) - float(torch.logsumexp(s, 0))) <= 1e-3
