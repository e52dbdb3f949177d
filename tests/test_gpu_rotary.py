"""rotary against its 64-bit form: types, layouts, widths that fill no vector,
strided and in-place rows, far positions, the gradient, and a whole layer
(rotary, attention with shared heads, their gradients, the paged cache)."""
import pytest
import torch

import online_softmax_forward_gb300 as pkg
from grad_ref import assert_gradients, backward64, rotary64
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def allowed(x, theta, amplitude, dt):
    """Half a step of the output, and fp32 arithmetic: three roundings of products with sines and
    cosines of 2 units in the last place, on |x| + |y| of the pair (8 units of 2^-24 in all)."""
    big = x.double().abs().amax(-1, keepdim=True) * 2 * amplitude
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    return lambda want: want.abs() * torch.finfo(dt).eps / 2 * (1 + 1e-6) + big * 2.0 ** -21 + tiny


def compare(got, x, pos, rot, transpose=False):
    theta = torch.tensor(rot.frequencies, dtype=torch.float64)
    want = rotary64(x.cpu(), pos.cpu(), theta, rot.layout, rot.amplitude, transpose)
    err = (got.cpu().double() - want).abs()
    assert (err <= allowed(x.cpu(), theta, rot.amplitude, got.dtype)(want)).all(), err.max()
    assert torch.equal(got[..., rot.width:], x[..., rot.width:])


def rows(*shape, dt, seed=0):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def positions(B, S, top, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, top + 1, (B, S), generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("dt", [BF, HF, F], ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hkv,S,d,width", [
    (1, 1, 1, 1, 64, 64), (2, 4, 2, 37, 128, 128), (3, 5, 1, 9, 128, 64), (2, 3, 3, 50, 64, 24),
    (1, 2, 1, 200, 64, 10), (4, 32, 8, 1, 128, 128), (1, 6, 2, 65, 80, 32), (1, 1, 1, 3, 6, 2),
    (1, 150, 30, 4, 256, 256), (2, 1, 1, 700, 16, 16), (1, 2, 2, 5, 1024, 1024),
])
def test_rows(dt, layout, B, H, Hkv, S, d, width):
    q, k = rows(B, H, S, d, dt=dt), rows(B, Hkv, S, d, dt=dt, seed=2)
    rot = pkg.Rotary(width, layout=layout)
    pos = positions(B, S, 5000)
    for transpose in (False, True):
        q2, k2 = pkg.rotary(q, k, rot, pos, transpose=transpose)
        assert q2.is_contiguous() and k2.is_contiguous()
        compare(q2, q, pos, rot, transpose)
        compare(k2, k, pos, rot, transpose)
    alone, none = pkg.rotary(q, None, rot, pos, transpose=True)
    assert none is None and torch.equal(alone, q2)
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("dt,width,layout", [(BF, 128, "half"), (HF, 24, "interleaved"), (F, 64, "half"),
                                             (BF, 10, "half")])
def test_bounds_checking_build(dt, width, layout, monkeypatch):
    q, k = rows(3, 7, 41, 128, dt=dt), rows(3, 2, 41, 128, dt=dt, seed=2)
    rot, pos = pkg.Rotary(width, layout=layout), positions(3, 41, 5000)
    lib = pkg.load_checked_library()
    monkeypatch.setattr(pkg, "load_library", lambda: lib)
    # with outputs given the call goes through load_library()
    q2, k2 = pkg.rotary(q, k, rot, pos, out=(torch.empty_like(q), torch.empty_like(k)))
    assert lib.attn_check_status(None) == pkg.ATTN_OK
    compare(q2, q, pos, rot)
    compare(k2, k, pos, rot)


@pytest.mark.parametrize("dt,width,layout", [(BF, 128, "half"), (HF, 64, "interleaved"), (F, 48, "half"),
                                             (BF, 10, "half")])
def test_strides_and_in_place(dt, width, layout):
    """Rows of a packed projection, read, written and overwritten where they lie; the rest stays."""
    B, H, Hkv, S, d = 2, 6, 2, 33, 128
    packed = rows(B, S, H + 2 * Hkv, d, dt=dt)
    q, k = packed[:, :, :H].transpose(1, 2), packed[:, :, H:H + Hkv].transpose(1, 2)
    rot, pos = pkg.Rotary(width, layout=layout), positions(B, S, 900)
    q2, k2 = pkg.rotary(q, k, rot, pos)
    compare(q2, q, pos, rot)
    compare(k2, k, pos, rot)
    same = pkg.rotary(q.contiguous(), k.contiguous(), rot, pos)
    assert torch.equal(same[0], q2) and torch.equal(same[1], k2)
    place = torch.full_like(packed, 7.0)
    out = place[:, :, :H].transpose(1, 2), place[:, :, H:H + Hkv].transpose(1, 2)
    pkg.rotary(q, k, rot, pos, out=out)
    assert torch.equal(out[0], q2) and torch.equal(out[1], k2) and (place[:, :, H + Hkv:] == 7.0).all()
    values = packed[:, :, H + Hkv:].clone()
    pkg.rotary(q, k, rot, pos, out=(q, k))
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(packed[:, :, H + Hkv:], values)
    # channels that start between two vectors, and a broadcast input
    odd = rows(B, H, S, d + 3, dt=dt)[..., 1:1 + d]
    compare(pkg.rotary(odd, None, rot, pos)[0], odd, pos, rot)
    one = rows(1, 1, S, d, dt=dt).expand(B, H, S, d)
    compare(pkg.rotary(one, None, rot, pos)[0], one, pos, rot)


@pytest.mark.parametrize("top", [4096, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(top):
    """The angle's error does not grow with the position (float64 angles: p * 2^-53 of them)."""
    rot = pkg.Rotary(64)
    x = rows(1, 2, 300, 64, dt=F)
    pos = (top - torch.arange(300, device="cuda")).to(torch.int32)[None]
    got, _ = pkg.rotary(x, None, rot, pos)
    theta = torch.tensor(rot.frequencies, dtype=torch.float64)
    want = rotary64(x.cpu(), pos.cpu(), theta)
    slack = x.cpu().double().abs().amax(-1, keepdim=True) * 2 * (2.0 ** -21 + top * 2.0 ** -52)
    assert ((got.cpu().double() - want).abs() <= want.abs() * 2.0 ** -24 + slack).all()


def test_negative_and_counted_positions():
    rot = pkg.Rotary(64, layout="interleaved")
    x = rows(3, 2, 40, 64, dt=F)
    start = torch.tensor([-70, 0, 12345], dtype=torch.int32, device="cuda")
    pos = start[:, None] + torch.arange(40, device="cuda", dtype=torch.int32)
    got, _ = pkg.rotary(x, None, rot, start)
    compare(got, x, pos, rot)
    assert torch.equal(got, pkg.rotary(x, None, rot, pos.contiguous())[0])


def test_scalings():
    x, pos = rows(1, 2, 64, 128, dt=F), positions(1, 64, 100000)
    theta = [10000.0 ** (-2 * i / 128) for i in range(64)]
    lin = pkg.Rotary(128, scaling="linear", factor=4.0)
    assert lin.frequencies == tuple(t / 4 for t in theta) and lin.amplitude == 1.0
    base = pkg.Rotary(128, scaling="base", factor=4.0)
    assert base.frequencies[0] == 1.0 and abs(base.frequencies[-1] * 4 / theta[-1] - 1) < 1e-12
    parts = pkg.Rotary(128, scaling="parts", factor=8.0, context=4096)
    assert parts.frequencies[:10] == tuple(theta[:10]) and parts.frequencies[-1] == theta[-1] / 8
    assert all(a >= b for a, b in zip(theta, parts.frequencies)) and parts.amplitude > 1.2
    own = pkg.Rotary(128, frequencies=theta, amplitude=0.5)
    for rot in (lin, base, parts, own):
        compare(pkg.rotary(x, None, rot, pos)[0], x, pos, rot)


def test_back_and_forth_and_differences():
    """transpose is the inverse at amplitude 1 and the gradient at any: <rotary(x), y> = <x, transpose(y)>."""
    rot, pos = pkg.Rotary(96, amplitude=1.25), positions(2, 50, 70000)
    x, y = rows(2, 3, 50, 128, dt=F), rows(2, 3, 50, 128, dt=F, seed=5)
    fx, _ = pkg.rotary(x, None, rot, pos)
    ty, _ = pkg.rotary(y, None, rot, pos, transpose=True)
    a, b = (fx.double() * y.double()).sum(), (x.double() * ty.double()).sum()
    # 2 n products of relative error 2^-21 each, independent: far below 1e-6 of |x| |y|
    assert (a - b).abs() <= 1e-6 * x.double().norm() * y.double().norm() * 1.25
    one = pkg.Rotary(96)
    back, _ = pkg.rotary(pkg.rotary(x, None, one, pos)[0], None, one, pos, transpose=True)
    assert (back - x).abs().max() <= x.abs().max() * 2.0 ** -19


def test_captured_streams_and_empty():
    rot, pos = pkg.Rotary(128), positions(2, 9, 500)
    q, k = rows(2, 4, 9, 128, dt=BF), rows(2, 2, 9, 128, dt=BF)
    want = pkg.rotary(q, k, rot, pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pkg.rotary(q, k, rot, pos)
    pos.add_(11)
    g.replay()
    moved = pkg.rotary(q, k, rot, pos, stream=(side := torch.cuda.Stream()))
    torch.cuda.synchronize()
    side.synchronize()
    assert torch.equal(got[0], moved[0]) and torch.equal(got[1], moved[1])
    assert not torch.equal(got[0], want[0])
    for shape in ((0, 4, 9, 128), (2, 4, 0, 128)):
        e = torch.empty(shape, dtype=BF, device="cuda")
        p = torch.empty((shape[0], shape[2]), dtype=torch.int32, device="cuda")
        assert pkg.rotary(e, None, rot, p)[0].shape == shape


def test_offsets_past_32_bits():
    rot = pkg.Rotary(64)
    S, H, d = 9000, 4000, 64  # 2.3e9 elements
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    x = torch.zeros(1, H, S, d, dtype=BF, device="cuda")
    x[0, -1] = rows(S, d, dt=BF)
    pos = torch.arange(S, device="cuda", dtype=torch.int32)[None]
    got, _ = pkg.rotary(x, None, rot, pos)
    compare(got[:, -1:], x[:, -1:], pos, rot)
    assert (got[0, :-1] == 0).all()


@pytest.mark.parametrize("dt,layout", [(BF, "half"), (HF, "interleaved"), (F, "half")])
def test_a_layer_there_and_back(dt, layout):
    """Packed projection -> rotary -> attention with shared heads -> their gradients -> packed
    gradient, against the 64-bit formulas on what each step was given; then the rotated keys go
    through the paged cache and one more token is decoded."""
    B, H, Hkv, S, d = 2, 8, 2, 300, 64
    packed = rows(B, S, H + 2 * Hkv, d, dt=dt)
    rot, pos = pkg.Rotary(d, layout=layout), positions(B, S, 0) + torch.arange(S, device="cuda", dtype=torch.int32)
    heads = lambda a, b: packed[:, :, a:b].transpose(1, 2)  # noqa: E731
    q, k = pkg.rotary(heads(0, H), heads(H, H + Hkv), rot, pos)
    v = heads(H + Hkv, H + 2 * Hkv).contiguous()
    o, lse = pkg.attention(q, k, v, causal=True)
    do = rows(B, H, S, d, dt=dt, seed=9)
    dq, dk, dv = pkg.attention_bwd(q, k, v, o, lse, do, causal=True)
    c = lambda t: t.cpu()  # noqa: E731
    want, errors = backward64(c(q), c(k), c(v), c(o), c(lse), c(do), causal=True)
    assert_gradients((dq, dk, dv), want, errors)
    grad = torch.empty_like(packed)
    place = lambda a, b: grad[:, :, a:b].transpose(1, 2)  # noqa: E731
    pkg.rotary(dq, dk, rot, pos, transpose=True, out=(place(0, H), place(H, H + Hkv)))
    place(H + Hkv, H + 2 * Hkv).copy_(dv)
    compare(place(0, H), dq, pos, rot, transpose=True)
    compare(place(H, H + Hkv), dk, pos, rot, transpose=True)
    # serving: the prompt into the cache, then one token at its own position
    cache = pkg.KVCache.empty(B * 5, Hkv, 64, d)
    table = torch.arange(B * 5, device="cuda", dtype=torch.int32).view(B, 5)
    at = lambda n: torch.full((B,), n, device="cuda", dtype=torch.int32)  # noqa: E731
    pkg.cache_append(cache, k, v, table, at(0))
    new = rows(B, 1, H + 2 * Hkv, d, dt=dt, seed=10)
    q1, k1 = pkg.rotary(new[:, :, :H].transpose(1, 2), new[:, :, H:H + Hkv].transpose(1, 2), rot, at(S))
    pkg.cache_append(cache, k1, new[:, :, H + Hkv:].transpose(1, 2).contiguous(), table, at(S))
    o1, _ = pkg.attention_cache(q1, cache, table, at(S + 1))
    kc, vc = pkg.cache_read(cache, table, at(S + 1), S + 1, dtype=dt)
    o2, _ = pkg.attention(q1, kc, vc, causal=True)
    assert (o1.float() - o2.float()).abs().max() <= 2e-2
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("dt", [BF, HF, F], ids=str)
def test_both_ways_through_the_wrapper(dt):
    """The host side in C++ takes ordinary calls and gives the bits of the Python one; what it does
    not take, it leaves alone."""
    x = rows(3, 41, 9, 64, dt=dt)
    q, k = x[:, :, :6].transpose(1, 2), x[:, :, 6:].transpose(1, 2)
    rot, pos = pkg.Rotary(48, layout="interleaved"), positions(3, 41, 5000)
    fast = lambda *a: pkg._fast().rotary(*a, *rot._args)  # noqa: E731
    for transpose in (False, True):
        for kk, p in ((k, pos), (None, pos[:, 0].contiguous())):
            a = fast(q, kk, p, transpose)
            out = (torch.empty(q.shape, dtype=dt, device="cuda"),
                   None if kk is None else torch.empty(k.shape, dtype=dt, device="cuda"))
            b = pkg.rotary(q, kk, rot, p, transpose=transpose, out=out)
            assert type(a) is tuple and a[0].is_contiguous() and torch.equal(a[0], b[0])
            assert a[1] is None if kk is None else torch.equal(a[1], b[1])
    class Rows(torch.Tensor):
        pass
    for args in ((q.cpu(), k, pos), (q, k.cpu(), pos), (q, k, pos.cpu()), (q, k, pos.long()), (q, k, pos[:2]),
                 (q, k, pos.t()), (q, k[:, :, :5], pos), (q.double(), None, pos), (q[0], None, pos),
                 (q[..., ::2], None, pos), (q[..., :32], None, pos), (q.as_subclass(Rows), None, pos), (q, 3, pos),
                 (q, k, pos[:, :, None])):
        assert fast(*args, False) is None
    host = pkg.Rotary(48, device="cpu")
    assert pkg._fast().rotary(q, k, pos, False, *host._args) is None
    with pytest.raises(ValueError):
        pkg.rotary(q, k, host, pos)
