"""Calls of the 4-bit attention on the tcgen05 kernel and on both kernels as a server
makes them: strided outputs, padded batches, dirty workspaces, replayed graphs, shared
pages, prompts beside single tokens, a captured step."""
import pytest
import torch

from exact_attention_117_b200 import fa
import kv4_util as ref
from test_kv4_attention import Case
from test_kv4_precision import attend, check, on_tcgen

# jobs cut over several CTAs (one row tile of each kv head over up to 37 of them) and
# jobs of their own
CUT = [(128, 8, 2, 32, [3000, 65], [40, 20]), (64, 32, 2, 64, [5000, 300, 40], [10, 5, 40])]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CUT, ids=["128", "64"])
def test_strides_padding_workspace_and_repeats(shape):
    c = Case(*shape, seed=71)
    assert on_tcgen(c)
    T, H, d = c.q.shape
    G = c.cache.shape[1]
    big = torch.full((T + 5, H + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:T, :H] = c.q
    a, b = attend(c), attend(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(c, *a)
    size = fa.kv4_attention_workspace_size(H, G, d, c.most)
    for fill in (0xff, 0x7f, 0):  # no numbers, large numbers, zeros: also as the cuts' integers
        out = torch.full((T + 5, 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T + 5, H), 7.0, device="cuda")
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        fa.kv4_attention(big[:, :H], c.cache, c.table, c.lens, c.cu, max_tokens=c.most, out=out[:, :H],
                         lse=lse, workspace=ws)
        fa.check_device_error()
        assert torch.equal(out[:T, :H], a[0]) and torch.equal(lse[:T], a[1])
        assert (out[T:] == 7).all() and (out[:, H:] == 7).all() and (lse[T:] == 7).all()
    with pytest.raises(fa.FaError):
        fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=c.most, workspace=ws[:-16])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CUT, ids=["128", "64"])
def test_replayed_with_other_lengths(shape):
    """One graph, lengths that shrink to one and to none and grow again, in one workspace:
    what an earlier replay left there (partial results, cuts) is never read."""
    c = Case(*shape, seed=72)
    T, H, d = c.q.shape
    size = fa.kv4_attention_workspace_size(H, c.cache.shape[1], d, c.most)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(T, H, device="cuda")
    call = lambda: fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=c.most, out=out,  # noqa: E731
                                    lse=lse, workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = c.lens.tolist()
    for lens in (full, [1] * len(full), [0] * len(full), [full[0]] + [0] * (len(full) - 1), [7] + full[1:], full):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.q.copy_(torch.randn_like(c.q.float()))
        out.fill_(float("nan"))
        graph.replay()
        fa.check_device_error()
        check(c, out, lse)
        for b, n in enumerate(lens):  # rows that see nothing
            first, last = int(c.cu[b]), int(c.cu[b + 1])
            none = out[first:max(first, last - n)]
            assert not none.any() and (lse[first:max(first, last - n)] == float("-inf")).all()


@pytest.mark.gpu
def test_two_streams_and_two_graphs():
    cases = [Case(128, 8, 2, 16, [900 + 300 * i, 90], [30, 25], seed=73 + i) for i in range(2)]
    want = [attend(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, got = [], []
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(fa.kv4_attention(c.q, c.cache, c.table, c.lens, c.cu, max_tokens=c.most))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    fa.check_device_error()
    for (o, lse), w in zip(got, want):
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,G", [(128, 8, 2), (64, 16, 2), (128, 5, 5)])
@pytest.mark.parametrize("order", ["prompt first", "prompt last"])
def test_prompts_beside_single_tokens(d, H, G, order):
    """A mixed step; and the same call with too small a bound on the tokens, which
    takes the other kernel."""
    lens, new = [700, 300, 1, 45, 513, 128], [200, 1, 1, 1, 1, 1]
    if order == "prompt last":
        lens, new = lens[::-1], new[::-1]
    c = Case(d, H, G, 16, lens, new, seed=75)
    assert on_tcgen(c)
    check(c, *attend(c))
    c.most = 1
    check(c, *attend(c))


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 50])
def test_requests_that_share_pages(new):
    """Two requests with the same first pages (a common prefix) and one whose table
    names a page twice."""
    c = Case(128, 8, 2, 16, [400, 400, 320], [new] * 3, seed=76)
    c.table[1, :20] = c.table[0, :20]
    c.table[2, 5] = c.table[2, 4]
    check(c, *attend(c))


@pytest.mark.gpu
@pytest.mark.parametrize("H,G,new", [(128, 1, 1), (128, 1, 3), (96, 2, 2), (7, 7, 3)])
def test_wide_groups(H, G, new):
    c = Case(64, H, G, 32, [333, 20], [new, new], seed=77)
    check(c, *attend(c))
    check(c, *attend(c, causal=False), causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,G,chunk", [(128, 8, 2, 1), (128, 8, 2, 30), (64, 8, 1, 12)])
def test_a_captured_step_replayed(d, H, G, chunk):
    """Plan, rotary, append and attention captured once and replayed as requests grow
    page by page, against the same steps made one call after another."""
    R, page, width, steps = 3, 16, 12, 5

    def state():
        g = torch.Generator(device="cuda").manual_seed(78)
        s = dict(cache=fa.kv4_cache(R * width, G, page, d),
                 table=torch.full((R, width), -1, dtype=torch.int32, device="cuda"),
                 ring=torch.randperm(R * width, generator=g, device="cuda", dtype=torch.int32),
                 range=torch.tensor([0, R * width], device="cuda"),
                 lens=torch.zeros(R, dtype=torch.int32, device="cuda"),
                 want=torch.zeros(R, dtype=torch.int32, device="cuda"),
                 x=torch.zeros(R * chunk + 2, (H + 2 * G) * d, dtype=torch.bfloat16, device="cuda"))
        return s

    f, amp = fa.rotary_frequencies(d)

    def step(s):
        room = R * chunk + 2
        p = fa.kv4_plan(s["lens"], s["want"], s["table"], s["ring"], s["range"], page, room,
                        lengths_out=s["lens"], free_range_out=s["range"])
        q = s["x"][:, :H * d].unflatten(-1, (H, d))
        k, v = (s["x"][:, (H + i * G) * d:(H + (i + 1) * G) * d].unflatten(-1, (G, d)) for i in range(2))
        yq, yk = fa.rotary(q.transpose(0, 1)[None], k.transpose(0, 1)[None], p.positions, f, amplitude=amp)
        fa.kv4_append(yk[0].transpose(0, 1), v, s["cache"], p.slots)
        o, lse = fa.kv4_attention(yq[0].transpose(0, 1), s["cache"], s["table"], p.lengths, p.cu_tokens,
                                  max_tokens=chunk)
        return o, lse, p.status, p.cu_tokens

    eager, replayed = state(), state()
    step(state())  # (loads the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(replayed)
    for i in range(steps):
        grow = torch.tensor([chunk, max(1, chunk // 2), chunk if i % 2 else 0], dtype=torch.int32, device="cuda")
        x = torch.randn(R * chunk + 2, (H + 2 * G) * d, device="cuda").bfloat16()
        for s in (eager, replayed):
            s["want"].copy_(s["lens"] + grow)
            s["x"].copy_(x)
        want = step(eager)
        graph.replay()
        fa.check_device_error()
        assert out[2].item() == 0 and torch.equal(out[3], want[3])
        T = int(out[3][-1])
        assert T > 0 and torch.equal(out[0][:T], want[0][:T]) and torch.equal(out[1][:T], want[1][:T])
        for name in ("cache", "table", "ring", "range", "lens"):
            assert torch.equal(eager[name], replayed[name]), name


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_writes_every_head_and_token_as_defined(d):
    """The whole cache after one call, byte by byte."""
    T, H, page = 37, 3, 32
    pages = 5
    k, v = (torch.randn(T, H, d, device="cuda").bfloat16() for _ in range(2))
    slots = torch.randperm(pages * page, device="cuda")[:T]
    cache = torch.randint(0, 256, (pages, H, page // 16, 18 * d), device="cuda", dtype=torch.uint8)
    want = cache.clone()
    fa.kv4_append(k, v, cache, slots)
    at = [(0, d // 2), (8 * d, d // 16), (9 * d, d // 2), (17 * d, d // 16)]
    for h in range(H):
        pad = (-T) % 16
        rows = ref.tiles_of(*(torch.cat([x[:, h], x[:1, h].expand(pad, d)]) for x in (k, v)))
        for i, s in enumerate(slots.tolist()):
            tile = want[s // page, h, s % page // 16]
            for a, w in at:
                tile[a + s % 16 * w:a + (s % 16 + 1) * w] = rows[i // 16, a + i % 16 * w:a + (i % 16 + 1) * w]
    assert torch.equal(cache, want)
