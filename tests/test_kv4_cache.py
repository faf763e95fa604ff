"""The paged 4-bit cache: its plan of pages, writing and reading it back."""
import random

import pytest
import torch

from exact_attention_117_b200 import fa
import kv4_util as ref

P = 0x10000


def _plan_raw(lens=P, new=P, table=P, stride=4, width=4, ring=P, size=9, rng=P, R=3, page=16,
              most=8, lo=P, ro=P, cu=P, slots=P, pos=P, status=P):
    return fa.load().fa_kv4_plan(lens, new, table, stride, width, ring, size, rng, R, page, most,
                                 lo, ro, cu, slots, pos, status, None)


def test_plan_refusals():
    from exact_attention_117_b200 import build
    build.build()
    for name in ("lens", "new", "table", "ring", "rng", "lo", "ro", "cu", "slots", "pos", "status"):
        assert _plan_raw(**{name: None}) == 1, name
    for bad in (dict(R=0), dict(width=0), dict(size=0), dict(page=8), dict(page=24), dict(most=-1),
                dict(stride=3), dict(most=(1 << 30) + 1), dict(R=1 << 28, width=16, stride=16),
                dict(width=1 << 27, stride=1 << 27)):
        assert _plan_raw(**bad) == 2, bad
    for name in ("lens", "table", "cu", "pos", "status"):
        assert _plan_raw(**{name: P + 2}) == 4, name
    for name in ("rng", "ro", "slots"):
        assert _plan_raw(**{name: P + 4}) == 4, name


def _store_raw(call, k=P, v=P, cache=P, slots=P, T=3, H=2, d=64, pages=4, page=16, strides=(128, 64, 128, 64)):
    lib = fa.load()
    st = ref.longs(*strides)
    if call == "append":
        return lib.fa_kv4_append(k, v, cache, slots, T, H, d, pages, page, st, None)
    return lib.fa_kv4_gather(cache, slots, k, v, T, H, d, pages, page, st, None)


@pytest.mark.parametrize("call", ["append", "gather"])
def test_store_refusals(call):
    for name in ("k", "v", "cache", "slots"):
        assert _store_raw(call, **{name: None}) == 1, name
    for bad in (dict(T=-1), dict(H=0), dict(pages=0), dict(page=0), dict(page=20)):
        assert _store_raw(call, **bad) == 2, bad
    assert _store_raw(call, d=96) == 3
    for bad in (dict(k=P + 8), dict(v=P + 2), dict(cache=P + 8), dict(slots=P + 4),
                dict(strides=(128, 60, 128, 64)), dict(strides=(128, 64, -128, 64))):
        assert _store_raw(call, **bad) == 4, bad
    assert _store_raw(call, T=0) == 0 and _store_raw(call, T=0, k=None, v=None, slots=None) == 0


def test_binding_refuses():
    c = torch.zeros(2, 3, 1, 18 * 64, dtype=torch.uint8)
    x = torch.zeros(5, 3, 64, dtype=torch.bfloat16)
    s = torch.zeros(5, dtype=torch.int64)
    for k, v, cache, slots in ((x.float(), x, c, s), (x, x[:, :2], c, s), (x[:, :2], x[:, :2], c, s),
                               (x, x, c.int(), s), (x, x, c[..., :64], s), (x, x, c, s.int()),
                               (x, x, c, s[:4]), (x.transpose(1, 2), x.transpose(1, 2), c, s),
                               (x, x, c, s)):  # the last: not on a GPU
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            fa.kv4_append(k, v, cache, slots)
    with pytest.raises(ValueError):
        fa.kv4_gather(c[..., :-1], s)
    for bad in ((0, 1, 16, 64), (1, 0, 16, 64), (1, 1, 20, 64), (1, 1, 16, 80)):
        with pytest.raises(ValueError):
            fa.kv4_cache(*bad, device="cpu")
    assert fa.kv4_cache(2, 3, 32, 128, device="cpu").shape == (2, 3, 2, 18 * 128)


# ------------------------------------------------------------------ the plan
def _random_step(rng, R, page, width, idle=0.2, end=0.2, prompt=0.2):
    old = [rng.randint(0, page * width - 1) if rng.random() > 0.1 else 0 for _ in range(R)]
    new = []
    for o in old:
        x = rng.random()
        new.append(o if x < idle else 0 if x < idle + end else
                   rng.randint(o, page * width) if x < idle + end + prompt else
                   rng.randint(0, o) if x < idle + end + prompt + 0.1 else min(o + 1, page * width))
    return old, new


def _plan_state(rng, old, page, width, spare):
    held = [-(-o // page) for o in old]
    P_ = sum(held) + spare
    ids = list(range(P_))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (width - h))
        at += h
    head = rng.randint(0, 1 << 40)
    ring = [-9] * P_
    for i in range(spare):
        ring[(head + i) % P_] = ids[at + i]
    return table, ring, head, head + spare


def _run_plan(old, new, table, ring, head, tail, page, most, in_place=False):
    t = torch.tensor
    lens, tab = t(old, dtype=torch.int32, device="cuda"), t(table, dtype=torch.int32, device="cuda")
    rg, fr = t(ring, dtype=torch.int32, device="cuda"), t([head, tail], device="cuda")
    p = fa.kv4_plan(lens, t(new, dtype=torch.int32, device="cuda"), tab, rg, fr, page, most,
                    **(dict(lengths_out=lens, free_range_out=fr) if in_place else {}))
    return p, tab, rg


def _check_plan(old, new, table, ring, head, tail, page, most, in_place=False):
    p, tab, rg = _run_plan(old, new, table, ring, head, tail, page, most, in_place)
    table, ring = [list(r) for r in table], list(ring)
    lens, head, tail, cu, slots, positions, status = ref.plan(old, new, table, ring, head, tail, page, most)
    assert p.status.item() == status
    assert p.lengths.tolist() == lens and p.free_range.tolist() == [head, tail]
    assert p.cu_tokens.tolist() == cu and p.slots.tolist() == slots and p.positions.tolist() == positions
    assert tab.tolist() == table and rg.tolist() == ring
    return status


@pytest.mark.gpu
@pytest.mark.parametrize("R,page,width", [(1, 16, 1), (1, 64, 40), (8, 16, 9), (33, 48, 7), (1024, 16, 5),
                                          (1025, 32, 3), (2500, 16, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_lists(R, page, width, in_place):
    rng = random.Random(R * 7 + width)
    for spare_more in (0, 5):
        old, new = _random_step(rng, R, page, width)
        need = sum(max(0, -(-n // page) - -(-o // page)) for o, n in zip(old, new))
        grow = sum(max(0, n - o) for o, n in zip(old, new))
        table, ring, head, tail = _plan_state(rng, old, page, width, need + spare_more)
        if not ring:
            ring = [0]
        assert _check_plan(old, new, table, ring, head, tail, page, grow + spare_more, in_place) == 0


@pytest.mark.gpu
def test_plan_refuses_a_step_as_a_whole():
    rng = random.Random(11)
    old, new = [16, 0, 31, 5], [17, 40, 0, 5]  # 1 + 3 pages needed, 2 given back, 41 tokens
    table, ring, head, tail = _plan_state(rng, old, 16, 4, 4)
    ring, size = ring + [-9] * 3, len(ring) + 3
    ring = [-9] * size
    for i in range(4):
        ring[(head + i) % size] = 100 + i
    tail = head + 4
    assert _check_plan(old, new, table, ring, head, tail, 16, 41) == 0
    assert _check_plan(old, new, table, ring, head, tail - 1, 16, 41) == 1
    assert _check_plan(old, new, table, ring, head, tail, 16, 40) == 2
    assert _check_plan(old, new, table, ring, head, tail - 1, 16, 0) == 3
    assert _check_plan([16, 0, 31, -1], new, table, ring, head, tail, 16, 41) & 4
    assert _check_plan(old, [17, 40, 0, 65], table, ring, head, tail, 16, 101) & 4
    assert _check_plan(old, new, table, ring, -5, -1, 16, 41) & 8
    assert _check_plan(old, new, table, ring, head, head + size, 16, 41) & 8  # released pages do not fit
    assert _check_plan(old, old, table, ring, head, head + size + 1, 16, 0) & 8


@pytest.mark.gpu
def test_plan_replays_in_a_graph():
    """Lengths, ring range, table and ring live on the device: a captured step serves
    every later one."""
    page, width, R = 16, 6, 3
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    ring = torch.arange(18, dtype=torch.int32, device="cuda")
    fr = torch.tensor([0, 18], device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    target = torch.zeros(R, dtype=torch.int32, device="cuda")
    fa.kv4_plan(lens, target, table, ring, fr, page, 40)  # loads the kernel before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = fa.kv4_plan(lens, target, table, ring, fr, page, 40, lengths_out=lens, free_range_out=fr)
    host = dict(lens=[0] * R, table=[[-1] * width for _ in range(R)], ring=list(range(18)), head=0, tail=18)
    rng = random.Random(2)
    for step in range(40):
        want = [rng.choice([0, min(n + 1, 96), min(n + rng.randint(1, 13), 96), n]) for n in host["lens"]]
        target.copy_(torch.tensor(want, dtype=torch.int32))
        graph.replay()
        host["lens"], host["head"], host["tail"], cu, slots, positions, status = ref.plan(
            host["lens"], want, host["table"], host["ring"], host["head"], host["tail"], page, 40)
        assert status == 0 and p.status.item() == 0
        assert p.slots.tolist() == slots and p.cu_tokens.tolist() == cu
        assert lens.tolist() == host["lens"] and fr.tolist() == [host["head"], host["tail"]]
        assert table.tolist() == host["table"] and ring.tolist() == host["ring"]


# ------------------------------------------------------------------ write and read
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (5, 3, 16), (33, 2, 48), (300, 8, 64), (129, 7, 128)])
def test_append_and_gather_match_definition(d, T, H, page):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    pages = -(-T // page) * 2 + 3
    k, v = (torch.randn(T, H, d, generator=g, device="cuda").bfloat16() * (i + 1) for i in range(2))
    k[0, 0, :64] = 2.5                      # a group of equal values: scale 0
    v[T // 2, H - 1, :64] *= 1e-38          # subnormal numbers
    k[T - 1, 0, :64] *= 2.0 ** 100
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    cache = torch.randint(0, 256, (pages, H, page // 16, 18 * d), generator=g, device="cuda",
                          dtype=torch.uint8)
    before = cache.clone()
    fa.kv4_append(k, v, cache, slots)
    # the bytes: every written row as defined, everything else as it was
    for h in range(H):
        want = before[:, h].reshape(-1, 18 * d).clone()
        pad = torch.zeros(16 - 1, d, dtype=torch.bfloat16, device="cuda")
        for i, s in enumerate(slots.tolist()):
            if i > 40 and i % 16:
                continue
            tile, r = divmod(s, 16)
            one = ref.tiles_of(torch.cat([k[i, h][None], pad]), torch.cat([v[i, h][None], pad]))[0]
            got = cache[s // page, h, s % page // 16]
            for at, width in ((0, d // 2), (8 * d, d // 16), (9 * d, d // 2), (17 * d, d // 16)):
                a = got[at + r * width:at + (r + 1) * width]
                assert torch.equal(a, one[at:at + width]), (i, h, at)
        assert want is not None
    rows = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    rows[slots] = True
    view = lambda c: [c[..., a:a + 16 * w].unflatten(-1, (16, w)).transpose(0, 1).flatten(1, 3)  # noqa: E731
                      for a, w in ((0, d // 2), (8 * d, d // 16), (9 * d, d // 2), (17 * d, d // 16))]
    for a, b in zip(view(cache), view(before)):
        assert torch.equal(a[:, ~rows], b[:, ~rows])
    # the values
    gk, gv = fa.kv4_gather(cache, slots)
    for got, x in ((gk, k), (gv, v)):
        want = ref.dequantised(x)
        # rounded to 32 bits, then to bf16
        assert torch.equal(got, want.float().bfloat16())
        # and no further from x than half a step of the group (steps are at most
        # 2^-7 above a fifteenth of the span, or the smallest bf16)
        span = x.double().unflatten(-1, (-1, 64))
        span = (span.amax(-1) - span.amin(-1))[..., None]
        err = (want.unflatten(-1, (-1, 64)) - x.double().unflatten(-1, (-1, 64))).abs()
        assert (err <= span / 30 * (1 + 2.0 ** -6) + 2.0 ** -134).all()


@pytest.mark.gpu
def test_append_borders_and_odd_values():
    """Values on and next to the borders between two codes, and groups that hold no number."""
    d = 64
    lo, s = -2.0, 2.0 ** -2
    base = torch.full((64,), lo, device="cuda")
    base[1] = lo + 15 * s                                   # scale exactly s
    half = lo + s * (torch.arange(15, device="cuda") + 0.5)  # exact in bf16: goes up
    base[2:17] = half
    base[17:32] = half - 2.0 ** -6
    k = base.bfloat16().reshape(1, 1, 64).repeat(4, 1, 1)
    k[1, 0, 5] = float("nan")
    k[2, 0, 9] = float("inf")
    k[3, 0, 0], k[3, 0, 1] = -3e38, 3e38                    # a span that no float holds
    v = torch.randn(4, 1, 64, device="cuda").bfloat16()
    cache = fa.kv4_cache(1, 1, 16, d)
    slots = torch.arange(4, device="cuda")
    fa.kv4_append(k, v, cache, slots)
    gk, gv = fa.kv4_gather(cache, slots)
    assert torch.equal(gk[0], ref.dequantised(k[:1])[0].bfloat16())
    assert torch.equal(gk[0, 0, 2:17].double(), (half + s / 2).double())
    assert gk[1:].isnan().all() and torch.equal(gv, ref.dequantised(v).float().bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("lift", [0, -100])
def test_append_values_a_hair_from_a_border(lift):
    """Tiny values in a group whose lowest is a whole border below 0: their distances
    from it are that border give or take less than 32 bits hold."""
    x = torch.zeros(64, dtype=torch.float64)
    x[0], x[1] = -2.875, 0.875  # scale 1/4; 0 is the border 11 1/2 steps above the lowest
    tiny = [2.0 ** -e for e in (10, 18, 20, 21, 22, 23, 30)]
    x[2:9], x[9:16] = torch.tensor(tiny, dtype=torch.float64), -torch.tensor(tiny, dtype=torch.float64)
    x = (x * 2.0 ** lift).bfloat16().reshape(1, 1, 64).cuda()
    cache = fa.kv4_cache(1, 1, 16, 64)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    fa.kv4_append(x, x, cache, slots)
    for got in fa.kv4_gather(cache, slots):
        want = ref.dequantised(x)
        assert torch.equal(got.double(), want)  # multiples of 1/8: exact in bf16
        up = (got[0, 0].double() * 2.0 ** -lift + 2.875) / 0.25
        assert up[2:9].tolist() == [12.0] * 7 and up[9:16].tolist() == [11.0] * 7


@pytest.mark.gpu
def test_append_skips_slots_outside_and_reads_zeros_there():
    H, d, page = 2, 128, 32
    cache = torch.randint(0, 255, (3, H, 2, 18 * d), device="cuda", dtype=torch.uint8)
    before = cache.clone()
    k, v = (torch.randn(4, H, d, device="cuda").bfloat16() for _ in range(2))
    outside = torch.tensor([-1, 3 * page, 1 << 40, -(1 << 40)], device="cuda")
    fa.kv4_append(k, v, cache, outside)
    assert torch.equal(cache, before)
    gk, gv = fa.kv4_gather(cache, outside)
    assert not gk.any() and not gv.any()
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    fa.kv4_append(k[:0], v[:0], cache, e)
    assert fa.kv4_gather(cache, e)[0].shape == (0, H, d) and torch.equal(cache, before)


@pytest.mark.gpu
def test_append_strided_inputs_stream_and_graph():
    T, H, d, page = 21, 3, 64, 16
    x = torch.randn(T, 3 * H * d, device="cuda").bfloat16()
    k, v = (x[:, i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in (1, 2))
    slots = torch.randperm(64, device="cuda")[:T]
    a, b = fa.kv4_cache(4, H, page, d), fa.kv4_cache(4, H, page, d)
    fa.kv4_append(k, v, a, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.kv4_append(k.contiguous(), v.contiguous(), b, slots, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    ok = torch.empty(T, 2 * H, d, dtype=torch.bfloat16, device="cuda")
    gk, gv = fa.kv4_gather(a, slots, out_k=ok[:, :H], out_v=ok[:, H:])
    fk, fv = fa.kv4_gather(a, slots)
    assert torch.equal(gk, fk) and torch.equal(ok[:, H:], fv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv4_append(k, v, b, slots)
        rk, rv = fa.kv4_gather(b, slots)
    x.copy_(torch.randn_like(x.float()))
    slots.copy_(torch.randperm(64, device="cuda")[:T])
    graph.replay()
    assert torch.equal(rk, ref.dequantised(k).float().bfloat16())
    assert torch.equal(rv, ref.dequantised(v).float().bfloat16())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Slots whose bytes lie past 2^32 of the cache."""
    H, d, page = 8, 128, 64
    pages = (1 << 32) // (H * 4 * 18 * d) + 3
    cache = torch.empty((pages, H, 4, 18 * d), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * page - 1, (pages - 2) * page + 17, 5], device="cuda")
    k, v = (torch.randn(3, H, d, device="cuda").bfloat16() for _ in range(2))
    fa.kv4_append(k, v, cache, slots)
    gk, gv = fa.kv4_gather(cache, slots)
    assert torch.equal(gk, ref.dequantised(k).float().bfloat16())
    assert torch.equal(gv, ref.dequantised(v).float().bfloat16())
