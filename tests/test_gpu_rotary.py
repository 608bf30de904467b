"""Rotary positions against complex rotations in 64 bits.

Bound, with u = 2^-24: the reduced angle is rounded to fp32 (2 pi times 2^-26 of
a turn, 1.6 u), sine and cosine are off by two steps (4 u) and by the scale's
product (u), each of the two products and their sum by u more: 10 u times
(|u| + |v|) scale covers them; then half a step of the type."""

import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _values(gen, tokens, heads, dim, dtype, pad=0, shift=0):
    flat = torch.randn(tokens * heads * (dim + pad) + shift, generator=gen, device=DEV).to(dtype)
    return flat[shift:].view(tokens, heads, dim + pad)[..., :dim]


def _positions(gen, tokens, far=100000):
    return torch.randint(0, far, (tokens,), generator=gen, device=DEV, dtype=torch.int32)


def _pairs(first, n, interleaved):
    i = torch.arange(n, device=DEV)
    return (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + n + i)


def _check(x, y, positions, freq, first=0, interleaved=False, scale=1.0, transpose=False):
    n = freq.numel()
    one, two = _pairs(first, n, interleaved)
    a = positions.double()[:, None, None] * freq.to(DEV) * (-1.0 if transpose else 1.0)
    z = torch.complex(x[..., one].double(), x[..., two].double()) * torch.polar(torch.full_like(a, scale), a)
    off = 10 * U * abs(scale) * (x[..., one].double().abs() + x[..., two].double().abs())
    half = torch.finfo(x.dtype).eps / 2
    for got, want in ((y[..., one], z.real), (y[..., two], z.imag)):
        assert bool(((got.double() - want).abs() <= off + half * (want.abs() + off)).all())
    rest = torch.ones(x.shape[-1], dtype=torch.bool, device=DEV)
    rest[one] = rest[two] = False
    assert torch.equal(y[..., rest], x[..., rest])


def _turn(x, positions, freq, out=None, **kw):
    y = torch.full_like(x, 7.0) if out is None else out
    mu.muon_rotary(Handle.get(), x, y, positions, freq.to(DEV), **kw)
    return y


HEAD = [(2, 0, 1), (64, 0, 32), (128, 0, 64), (128, 0, 32), (192, 128, 32), (80, 0, 40), (100, 3, 17), (70, 1, 3),
        (256, 0, 128), (36, 7, 13), (600, 11, 290)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,first,pairs", HEAD)
def test_head_layouts(dim, first, pairs, interleaved, dtype):
    gen = _gen(dim)
    freq = mu.muon_rotary_frequencies(pairs)
    for tokens, heads in ((1, 1), (37, 3), (5, 64)):
        x, pos = _values(gen, tokens, heads, dim, dtype), _positions(gen, tokens)
        for kw in (dict(), dict(transpose=True, scale=1.25)):
            kw.update(first=first, interleaved=interleaved)
            _check(x, _turn(x, pos, freq, **kw), pos, freq, **kw)
            into = x.clone()
            assert torch.equal(_turn(into, pos, freq, out=into, **kw), _turn(x, pos, freq, **kw))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [1, 2, 3, 16, 63, 130, 1025, 4099])
def test_tokens_of_several_tensors(tokens, dtype):
    gen = _gen(tokens)
    freq, pos = mu.muon_rotary_frequencies(64), _positions(gen, tokens)
    xs = [_values(gen, tokens, n, 128, dtype) for n in (16, 4, 1, 7)]
    for n in (1, 2, 3, 4):
        ys = [torch.full_like(x, 7.0) for x in xs[:n]]
        mu.muon_rotary(Handle.get(), xs[:n], ys, pos, freq.to(DEV))
        for x, y in zip(xs, ys):
            _check(x, y, pos, freq)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_token_with_more_heads_than_a_workgroup_takes(dtype):
    gen, freq = _gen(1), mu.muon_rotary_frequencies(64)
    for heads in (128, 129, 1000):
        x, pos = _values(gen, 3, heads, 192, dtype), _positions(gen, 3)
        _check(x, _turn(x, pos, freq, first=64), pos, freq, first=64)
        x = x[:, :, 64:]
        _check(x, _turn(x, pos, freq), pos, freq)


@pytest.mark.parametrize("pairs", [1000, 2048])
def test_the_widest_heads(pairs):
    gen, freq = _gen(2), mu.muon_rotary_frequencies(pairs)
    x, pos = _values(gen, 9, 2, 2 * pairs + 5, F32), _positions(gen, 9)
    _check(x, _turn(x, pos, freq, first=2), pos, freq, first=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (5, 3), (64, 8)])
def test_strides_and_alignments(pad, shift, dtype):
    gen, freq = _gen(3), mu.muon_rotary_frequencies(32)
    pos = _positions(gen, 60)
    wide = _values(gen, 60, 9, 64, dtype, pad, shift)
    for x in (wide, wide[:, 2:6], wide[:, 4:5], wide.permute(1, 0, 2)[:, :60].permute(1, 0, 2),
              wide.transpose(0, 1).contiguous().transpose(0, 1), wide[:1].expand(60, 9, 64)):
        _check(x, _turn(x, pos, freq, out=torch.zeros(60, x.shape[1], 64, device=DEV, dtype=dtype)), pos, freq)
    _check(wide[:, :1], _turn(wide[:, 0], pos, freq)[:, None], pos, freq)          # (tokens, width)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_within_a_fused_tensor(dtype):
    gen, freq = _gen(4), mu.muon_rotary_frequencies(32)
    pos = _positions(gen, 77)
    buf = _values(gen, 77, 12, 64, dtype, pad=6)
    q, k = buf[:, 1:7], buf[:, 7:9]
    want = [_turn(t.contiguous(), pos, freq) for t in (q, k)]
    whole = torch.as_strided(buf, (77 * 12 * 70 - 6,), (1,), buf.storage_offset())
    before = whole.clone()
    mu.muon_rotary(Handle.get(), [q, k], [q, k], pos, freq.to(DEV))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    for t in (q, k):
        t.copy_(torch.as_strided(before, t.shape, t.stride(), t.storage_offset() - buf.storage_offset()))
    assert torch.equal(whole, before)
    # the turning part of a wider head, and a shared key head of that part alone
    wide, shared = _values(gen, 77, 5, 192, dtype), _values(gen, 77, 1, 64, dtype)
    a, b, rest = wide[..., 128:], shared, wide[..., :128].clone()
    want = [_turn(t.contiguous(), pos, freq, interleaved=True) for t in (a, b)]
    mu.muon_rotary(Handle.get(), [a, b], [a, b], pos, freq.to(DEV), interleaved=True)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(wide[..., :128], rest)


def test_far_and_negative_positions():
    gen = _gen(5)
    freq = mu.muon_rotary_frequencies(64, base=1e6, scaling="parts", factor=16.0, context=32768.0)
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7], dtype=torch.int32, device=DEV)
    x = _values(gen, 8, 4, 128, F32)
    # in 64 bits the angle itself is off by 2^-53 of itself twice: 5e-7 at 2^31
    one, two = _pairs(0, 64, False)
    y = _turn(x, pos, freq)
    a = pos.double()[:, None, None] * freq.to(DEV)
    z = torch.complex(x[..., one].double(), x[..., two].double()) * torch.polar(torch.ones_like(a), a)
    off = (10 * U + a.abs() * 2.0 ** -51) * (x[..., one].double().abs() + x[..., two].double().abs())
    assert bool(((y[..., one].double() - z.real).abs() <= off + U * z.real.abs()).all())
    assert bool(((y[..., two].double() - z.imag).abs() <= off + U * z.imag.abs()).all())
    assert torch.equal(y[0], x[0])                              # position 0 turns nothing


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_gradient_is_the_transposed_turn(interleaved):
    # <y, R x> = <R^T y, x>: whole numbers and quarter turns, so that every product is exact
    gen = _gen(6)
    freq = torch.full((32,), 0.5 * torch.pi, dtype=torch.float64)
    x, g = (torch.randint(-8, 9, (50, 3, 64), generator=gen, device=DEV).float() for _ in range(2))
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    y, dx = _turn(x, pos, freq, interleaved=interleaved), _turn(g, pos, freq, interleaved=interleaved, transpose=True)
    assert torch.equal(y.round(), y) and torch.equal(dx.round(), dx)
    assert float((y.double() * g.double()).sum()) == float((x.double() * dx.double()).sum())
    # and against differences: the turn is linear, so its difference quotient along v is itself
    v = torch.randint(-8, 9, (50, 3, 64), generator=gen, device=DEV).float()
    moved = _turn(x + v, pos, freq, interleaved=interleaved)
    assert float(((moved - y).double() * g.double()).sum()) == float((dx.double() * v.double()).sum())


def test_values_that_are_not_finite_stay_in_their_pair():
    gen, freq = _gen(7), mu.muon_rotary_frequencies(32)
    x, pos = _values(gen, 20, 2, 80, F32), _positions(gen, 20)
    want = _turn(x, pos, freq, first=8)
    x[7, 1, 8 + 5], x[9, 0, 3], x[11, 0, 79] = float("nan"), float("inf"), float("nan")
    y = _turn(x, pos, freq, first=8)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[7, 1, 8 + 5] = hit[7, 1, 8 + 5 + 32] = hit[9, 0, 3] = hit[11, 0, 79] = True
    assert torch.equal(y[~hit], want[~hit]) and bool(torch.isnan(y[7, 1, 13]) & torch.isnan(y[7, 1, 45]))
    assert float(y[9, 0, 3]) == float("inf")


def test_streams_and_a_captured_graph():
    gen, freq = _gen(8), mu.muon_rotary_frequencies(64).to(DEV)
    q, k, pos = _values(gen, 300, 8, 128, BF16), _values(gen, 300, 2, 128, BF16), _positions(gen, 300)
    h = Handle.get()
    outs = [torch.zeros_like(t) for t in (q, k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mu.muon_rotary(h, [q, k], outs, pos, freq, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((q, k), outs):
        assert torch.equal(y, _turn(x, pos, freq))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mu.muon_rotary(h, [q, k], outs, pos, freq)
    for seed in (1, 2, 3):
        pos.copy_(_positions(_gen(seed), 300))
        q.copy_(_values(_gen(seed + 10), 300, 8, 128, BF16))
        [t.zero_() for t in outs]
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((q, k), outs):
            assert torch.equal(y, _turn(x, pos, freq))
    mu.muon_rotary(h, q[:0], outs[0][:0], pos[:0], freq)


@pytest.mark.parametrize("dtype,tokens,interleaved,first", [(BF16, 20011, False, 0), (F32, 9001, True, 0),
                                                            (BF16, 20011, True, 32), (F32, 9001, False, 3)])
def test_large_tensors_are_their_parts(dtype, tokens, interleaved, first):
    # beyond 96 MiB the tensors are read around the caches
    gen, freq = _gen(tokens), mu.muon_rotary_frequencies(32).to(DEV)
    q, k = _values(gen, tokens, 24, 128, dtype), _values(gen, tokens, 3, 128, dtype)
    assert q.nbytes + k.nbytes >= 96 << 20
    pos = _positions(gen, tokens)
    kw = dict(first=first, interleaved=interleaved)
    y = [torch.zeros_like(q), torch.zeros_like(k)]
    mu.muon_rotary(Handle.get(), [q, k], y, pos, freq, **kw)
    for a in range(0, tokens, tokens // 3):
        cut = slice(a, a + 1001)
        for x, got in zip((q, k), y):
            assert torch.equal(got[cut], _turn(x[cut], pos[cut].contiguous(), freq, **kw))
    mu.muon_rotary(Handle.get(), [q, k], [q, k], pos, freq, **kw)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])


def test_tokens_far_apart():
    # 2^31 elements and more between a tensor's first and last token
    far, freq = (1 << 30) + 8, mu.muon_rotary_frequencies(32).to(DEV)
    buf = torch.zeros(2 * far + 4 * 64, device=DEV, dtype=BF16)
    x = torch.as_strided(buf, (3, 4, 64), (far, 64, 1))
    small = _values(_gen(1), 3, 4, 64, BF16)
    x.copy_(small)
    pos = _positions(_gen(2), 3)
    want = _turn(small, pos, freq)
    assert torch.equal(_turn(x, pos, freq, out=torch.zeros_like(small)), want)
    assert torch.equal(_turn(x, pos, freq, out=x), want)


# parts that end within a unit of 4 or 8, that have just one, or less than one
CUT = [(80, 0, 10, 3), (80, 5, 10, 300), (200, 0, 61, 70), (200, 9, 61, 129), (32, 8, 8, 5), (30, 8, 9, 5), (28, 4, 8, 2),
       (31, 8, 8, 65), (41, 15, 9, 40), (36, 16, 4, 40), (24, 0, 12, 513), (18, 0, 7, 600), (60, 0, 5, 200), (4096, 0, 2047, 3)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,first,pairs,heads", CUT)
def test_parts_that_end_within_a_unit(dim, first, pairs, heads, interleaved, dtype):
    gen, freq = _gen(dim + pairs), mu.muon_rotary_frequencies(pairs)
    kw = dict(first=first, interleaved=interleaved)
    for tokens, pad, shift in ((1, 0, 0), (83, 3, 1)):
        x, pos = _values(gen, tokens, heads, dim, dtype, pad, shift), _positions(gen, tokens)
        y = _turn(x, pos, freq, **kw)
        _check(x, y, pos, freq, **kw)
        # in place, in a tensor whose other elements stay as they were
        buf = torch.full((tokens, heads, dim + 3), 5.0, device=DEV, dtype=dtype)
        buf[..., 1:1 + dim] = x
        into = buf[..., 1:1 + dim]
        for _ in range(2):
            assert torch.equal(_turn(into, pos, freq, out=into, **kw), y)
            into.copy_(x)
        assert bool((buf[..., 0] == 5).all()) and bool((buf[..., 1 + dim:] == 5).all())
        # one tensor in place beside one that is copied
        into, other = x.clone(), torch.full_like(x, 7.0)
        mu.muon_rotary(Handle.get(), [into, x], [into, other], pos, freq.to(DEV), **kw)
        assert torch.equal(into, y) and torch.equal(other, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [1, 50])
def test_an_input_that_is_listed_again(tokens, dtype):
    gen, freq = _gen(11), mu.muon_rotary_frequencies(32)
    q, k, pos = _values(gen, tokens, 16, 64, dtype), _values(gen, tokens, 2, 64, dtype), _positions(gen, tokens)
    for xs in ([q, k, q], [k, q, k], [q, q, k, k], [k, q, q, k]):
        guard = [torch.full((tokens + 2, x.shape[1], 64), 7.0, device=DEV, dtype=dtype) for x in xs]
        ys = [t[1:-1] for t in guard]
        mu.muon_rotary(Handle.get(), xs, ys, pos, freq.to(DEV))
        for x, y, t in zip(xs, ys, guard):
            _check(x, y, pos, freq)
            assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())


# parts that end evenly, within a unit (so that units share elements), and with one shorter than a unit
AROUND = [(64, 0, 32), (80, 0, 10), (100, 8, 17), (100, 3, 17)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,first,pairs", AROUND)
def test_loads_around_the_caches_in_place_and_copied(dim, first, pairs, interleaved, dtype):
    # from 112 MiB that a call reads on: in place the turning elements alone count
    heads, size = (24, 3), torch.finfo(dtype).bits // 8
    tokens = -(-(112 << 20) // (sum(heads) * 2 * pairs * size)) + 5
    gen, freq = _gen(dim), mu.muon_rotary_frequencies(pairs).to(DEV)
    q, k = (_values(gen, tokens, n, dim, dtype) for n in heads)
    pos = _positions(gen, tokens)
    kw = dict(first=first, interleaved=interleaved)
    y = [torch.zeros_like(q), torch.zeros_like(k)]
    mu.muon_rotary(Handle.get(), [q, k], y, pos, freq, **kw)
    for a in range(0, tokens, tokens // 3):
        cut = slice(a, a + 501)
        for x, got in zip((q, k), y):
            assert torch.equal(got[cut], _turn(x[cut], pos[cut].contiguous(), freq, **kw))
    mu.muon_rotary(Handle.get(), [q, k], [q, k], pos, freq, **kw)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])
    # and back, in place: what is copied has not changed
    mu.muon_rotary(Handle.get(), [q, k], [q, k], pos, freq, transpose=True, **kw)
    one, two = _pairs(first, pairs, interleaved)
    rest = torch.ones(dim, dtype=torch.bool, device=DEV)
    rest[one] = rest[two] = False
    for x, got in zip((q, k), y):
        assert torch.equal(x[:700, :, rest], got[:700, :, rest]) and torch.equal(x[-700:, :, rest], got[-700:, :, rest])
        _check(got[-700:], x[-700:], pos[-700:], freq, transpose=True, **kw)
