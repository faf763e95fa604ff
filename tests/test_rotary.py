"""Rotary positions and their gradient against the 64-bit definition."""
import math

import pytest
import torch

from exact_attention_117_b200 import fa
import kv4_util as ref

P = 0x10000  # fake, never-dereferenced, 16-byte aligned address


def _raw(q=P, k=P, qo=P, ko=P, B=1, Hq=1, Hk=1, N=4, d=64, strides=None, pos=P, p64=0, ps=0,
         inv=P, rot=64, inter=0, amp=1.0, dtype=0):
    st = strides or [256, 256, 64] * 4
    return fa.load().fa_rotary(q, k, qo, ko, B, Hq, Hk, N, d, ref.longs(*st), pos, p64, ps, inv,
                               rot, inter, amp, 0, dtype, None)


def test_refusals():
    from exact_attention_117_b200 import build
    build.build()
    for name in ("q", "qo", "k", "ko", "pos", "inv"):
        assert _raw(**{name: None}) == 1, name
    for bad in (dict(B=0), dict(Hq=0), dict(N=-1), dict(rot=0), dict(rot=63), dict(rot=66),
                dict(dtype=3), dict(dtype=-1), dict(ps=-1), dict(Hk=-1)):
        assert _raw(**bad) == 2, bad
    for d in (0, 32, 96, 256):
        assert _raw(d=d) == 3
    assert _raw(q=P + 1) == 4 and _raw(inv=P + 4) == 4 and _raw(pos=P + 4, p64=1) == 4
    assert _raw(qo=P + 2, inter=1) == 4  # a pair is one access
    assert _raw(strides=[256, 256, 63] + [256, 256, 64] * 3, inter=1) == 4
    assert _raw(strides=[-256, 256, 64] + [256, 256, 64] * 3) == 4
    assert _raw(amp=math.inf) == 5
    assert _raw(N=0) == 0 and _raw(N=0, q=None, qo=None, pos=None) == 0


def test_an_output_at_its_inputs_address_lies_as_it_does():
    from exact_attention_117_b200 import build
    build.build()
    q, other = [1024, 256, 64], [1024, 64, 256]
    k = [512, 256, 64]
    heads = dict(Hq=4, Hk=2, B=2, N=4)
    assert _raw(strides=q + other + k + k, **heads) == 2
    assert _raw(strides=q + q + k + [512, 64, 128], **heads) == 2
    assert _raw(strides=q + other + k + k, Hq=4, Hk=2, B=2, N=0) == 0


def test_binding_refuses():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.ones(32, dtype=torch.float64)
    for q, k, pos, inv in ((x[0], None, torch.arange(3), f), (x.double(), None, torch.arange(3), f),
                           (x, x[:, :, :2], torch.arange(3), f), (x, x.float(), torch.arange(3), f),
                           (x, None, torch.arange(4), f), (x, None, torch.arange(3.0), f),
                           (x, None, torch.arange(3), f.float()),
                           (x.transpose(2, 3), None, torch.arange(64), f)):
        with pytest.raises(ValueError):
            fa.rotary(q, k, pos, inv)


def test_frequencies():
    f, a = fa.rotary_frequencies(128, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    assert torch.equal(f, 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128))
    g, a = fa.rotary_frequencies(128, factor=4.0, device="cpu")
    assert a == 1.0 and torch.equal(g, f / 4.0)
    g, a = fa.rotary_frequencies(128, factor=4.0, original_length=8192, device="cpu")
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32])
    assert torch.equal(g[turns < 1], f[turns < 1] / 4.0)
    mid = (turns > 1) & (turns < 32)
    assert ((g[mid] < f[mid]) & (g[mid] > f[mid] / 4.0)).all()
    assert a == pytest.approx(0.1 * math.log(4.0) + 1.0)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, base=0.0)):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(device="cpu", **bad)


def _check(y, x, want, what):
    """One rounding to the type, and 32-bit arithmetic before it: sin and cos of
    a phase rounded to 2^-25 turns and two products, 2^-20 of the pair's size."""
    size = x.double().abs().amax(-1, keepdim=True) * 2
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 2.0 ** -20 * size
    err = (y.double() - want).abs()
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3e} over"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,B,H,Hk,N", [
    (64, 64, 1, 1, 1, 1), (128, 128, 2, 5, 1, 7), (128, 64, 1, 8, 2, 300), (64, 32, 3, 2, 2, 33),
    (128, 90, 1, 3, 2, 17), (64, 2, 2, 4, 0, 5), (128, 126, 1, 1, 3, 129), (64, 64, 2, 16, 16, 1000)])
def test_rotary_matches_definition(dtype, interleaved, d, rot, B, H, Hk, N):
    g = torch.Generator(device="cuda").manual_seed(d + rot + N)
    q = torch.randn(B, H, N, d, generator=g, device="cuda").to(dtype)
    k = torch.randn(B, Hk, N, d, generator=g, device="cuda").to(dtype) if Hk else None
    pos = torch.randint(-5, 1 << 20, (B, N), generator=g, device="cuda")
    f, amp = fa.rotary_frequencies(rot, factor=8.0, original_length=4096)
    for inverse, call in ((False, fa.rotary), (True, fa.rotary_backward)):
        yq, yk = call(q, k, pos, f, interleaved=interleaved, amplitude=amp)
        _check(yq, q, ref.rotary(q, pos, f, interleaved, amp, inverse), "q")
        assert torch.equal(yq[..., rot:], q[..., rot:])
        if Hk:
            _check(yk, k, ref.rotary(k, pos, f, interleaved, amp, inverse), "k")
        else:
            assert yk is None


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,N", [(32, 8, 800), (32, 8, 2048), (5, 2, 8191), (1, 0, 70001)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes_between_a_decode_step_and_a_training_batch(H, Hk, N, interleaved):
    f, a = fa.rotary_frequencies(128)
    g = torch.Generator(device="cuda").manual_seed(N)
    q = torch.randn(1, H, N, 128, generator=g, device="cuda").bfloat16()
    k = torch.randn(1, Hk, N, 128, generator=g, device="cuda").bfloat16() if Hk else None
    pos = torch.randint(0, 100000, (N,), generator=g, device="cuda", dtype=torch.int32)
    y, z = fa.rotary(q, k, pos, f, interleaved)
    _check(y, q, ref.rotary(q, pos, f, interleaved, a), "q")
    if Hk:
        _check(z, k, ref.rotary(k, pos, f, interleaved, a), "k")


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_keep_their_phase(interleaved):
    q = torch.randn(1, 2, 6, 128, device="cuda")
    pos = torch.tensor([0, 1, 131071, 10 ** 7, 2 ** 31 - 1, -(2 ** 31)], device="cuda")
    f, _ = fa.rotary_frequencies(128)
    for p in (pos, pos.int()):
        y, _ = fa.rotary(q, None, p, f, interleaved=interleaved)
        _check(y, q, ref.rotary(q, pos, f, interleaved, 1.0), "q")


@pytest.mark.gpu
def test_strides_packed_in_place_and_unaligned():
    f, _ = fa.rotary_frequencies(128)
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, Hk, d = 37, 6, 2, 128
    x = torch.randn(T, (H + 2 * Hk) * d, generator=g, device="cuda").bfloat16()
    keep = x.clone()
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    q = x[:, :H * d].unflatten(-1, (H, d)).transpose(0, 1)[None]
    k = x[:, H * d:(H + Hk) * d].unflatten(-1, (Hk, d)).transpose(0, 1)[None]
    wq, wk = ref.rotary(q, pos, f, False, 1.0), ref.rotary(k, pos, f, False, 1.0)
    yq, yk = fa.rotary(q, k, pos, f)
    _check(yq, q, wq, "q")
    _check(yk, k, wk, "k")
    assert torch.equal(x, keep)
    zq, zk = fa.rotary(q, k, pos, f, out_q=q, out_k=k)  # in place, strided
    assert zq is q and torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(x[:, (H + Hk) * d:], keep[:, (H + Hk) * d:])
    # a start and a row pitch that 16-byte accesses do not divide
    flat = torch.randn(2 * 3 * 5 * 71 + 9, generator=g, device="cuda").half()
    u = torch.as_strided(flat, (2, 3, 5, 64), (3 * 5 * 71, 5 * 71, 71, 1), 1)
    f64, _ = fa.rotary_frequencies(64)
    y, _ = fa.rotary(u, None, torch.arange(5, device="cuda"), f64)
    _check(y, u, ref.rotary(u, torch.arange(5, device="cuda"), f64, False, 1.0), "odd start")
    with pytest.raises(fa.FaError):
        fa.rotary(u, None, torch.arange(5, device="cuda"), f64, interleaved=True)
    # heads shared by broadcasting are read, not written
    shared = torch.randn(1, 1, 9, 64, generator=g, device="cuda").bfloat16().expand(1, 4, 9, 64)
    y, _ = fa.rotary(shared, None, torch.arange(9, device="cuda"), f64,
                     out_q=torch.empty(1, 4, 9, 64, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(y[:, 0], y[:, 3])
    with pytest.raises(ValueError):
        fa.rotary(shared, None, torch.arange(9, device="cuda"), f64, out_q=shared)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_transposed_map_and_matches_differences(interleaved):
    f, amp = fa.rotary_frequencies(48, factor=4.0, original_length=64)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(2, 3, 11, 64, generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(0, 999, (11,), generator=g, device="cuda")
    kw = dict(interleaved=interleaved, amplitude=amp)
    grad, _ = fa.rotary_backward(w, None, pos, f, **kw)
    # <w, R x> = <R^T w, x>: sums of 4224 products of normal numbers, each side off by
    # at most 2^-20 of the sum of sizes
    a = (w.double() * fa.rotary(x, None, pos, f, **kw)[0].double()).sum()
    b = (grad.double() * x.double()).sum()
    assert abs(float(a - b)) <= 2.0 ** -20 * float((w.abs() * 2 * x.abs().amax(-1, keepdim=True)).sum())
    # differences of the loss along single channels (the map is linear: any step will
    # do; 1 keeps the cancellation error of 4224 terms below 2^-20 of their sizes)
    for idx in ((0, 0, 0, 0), (1, 2, 10, 47), (0, 1, 5, 30), (1, 0, 3, 60)):
        hi, lo = x.clone(), x.clone()
        hi[idx] += 1.0
        lo[idx] -= 1.0
        up, down = (fa.rotary(z, None, pos, f, **kw)[0].double() for z in (hi, lo))
        diff = float((w.double() * (up - down)).sum()) / 2
        assert abs(diff - float(grad[idx])) <= 2.0 ** -16


@pytest.mark.gpu
def test_empty_stream_and_graph():
    f, _ = fa.rotary_frequencies(64)
    e = torch.empty(1, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = fa.rotary(e, e, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert y.shape == e.shape
    x = torch.randn(1, 4, 50, 64, device="cuda").bfloat16()
    pos = torch.arange(50, device="cuda")
    want, _ = fa.rotary(x, None, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = fa.rotary(x, None, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        fa.rotary(x, None, pos, f, out_q=out)
    x.copy_(torch.randn(1, 4, 50, 64, device="cuda"))
    pos += 3
    graph.replay()
    want, _ = fa.rotary(x, None, pos, f)
    assert torch.equal(out, want)
