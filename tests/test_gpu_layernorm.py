"""Layer norm and its gradient against their formulas in 64 bits.

Bounds, with u = 2^-24 (half a step of fp32, relative): the longest chain of
fp32 additions in a row's sum is 32 values of a lane, 6 steps over lanes and 8
over waves, so a sum of C values is off by at most 64 u times the sum of their
magnitudes.  Forward: the mean by dm = 65 u mean|x|; the variance by 66 u of
itself and dm^2 (the differences' first order cancels in the sum); rstd by half
of that and 3 u; y by its three roundings, and by half a step of its type.
Gradient: xhat is two roundings off, each row sum 66 u of its magnitudes.  A
column sum adds fewer than `rows` values in fp32: (rows + 4) u of its
magnitudes; that every row is in it is seen with whole numbers, whose sums are
exact."""

import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _values(gen, *shape, dtype=F32, pad=0, shift=0):
    """Values in rows padded by `pad`, from `shift` elements into their buffer on."""
    *lead, cols = shape
    rows = 1
    for n in lead:
        rows *= n
    flat = torch.randn(rows * (cols + pad) + shift, generator=gen, device=DEV) * 2 + 0.3
    return flat.to(dtype)[shift:].view(*lead, cols + pad)[..., :cols]


def _weights(gen, cols, dtype, bias=True):
    w = (1 + 0.3 * torch.randn(cols, generator=gen, device=DEV)).to(dtype)
    return w, (0.2 * torch.randn(cols, generator=gen, device=DEV)).to(dtype) if bias else None


def _stats(x, eps, center):
    x = x.double()
    mean = x.mean(-1) if center else torch.zeros_like(x[..., 0])
    return mean, 1.0 / ((x - mean[..., None]).square().mean(-1) + eps).sqrt()


def _check_forward(x, w, b, eps, center, y, mean, rstd):
    m, r = _stats(x, eps, center)
    dm = 65 * U * x.double().abs().mean(-1) if center else torch.zeros_like(m)
    rel = 0.5 * (66 * U + dm.square() * r.square()) + 3 * U
    if center:
        assert bool(((mean.double() - m).abs() <= dm).all())
    assert bool(((rstd.double() - r).abs() <= r * rel).all())
    hat = (x.double() - m[..., None]) * r[..., None]
    wd = w.double() if w is not None else 1.0
    bd = b.double() if b is not None else 0.0
    want = hat * wd + bd
    off = (hat.abs() * rel[..., None] + (dm * r)[..., None] + 3 * U * hat.abs()) * abs(wd) + U * want.abs()
    assert bool(((y.double() - want).abs() <= off + _half(x.dtype) * (want.abs() + off)).all())


def _forward(x, w=None, b=None, eps=1e-5, center=True, out=None, **kw):
    y = torch.full_like(x, 7.0) if out is None else out
    mean, rstd = (torch.full(x.shape[:-1], 7.0, device=DEV) for _ in range(2))
    mu.muon_layernorm_forward(Handle.get(), x, y, weight=w, bias=b, mean=mean, rstd=rstd, eps=eps, center=center, **kw)
    return y, mean, rstd


COLS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 31, 33, 64, 65, 128, 129, 250, 256, 257, 511, 512, 513, 1000, 1001, 1024, 1025, 2048, 2049, 4096,
        4097, 7168, 8192, 8193, 16383, 16384, 100, 600, 769, 1536, 1537, 2560, 2999, 5120, 6145, 10000, 12288, 12289]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", COLS)
def test_forward_widths(cols, dtype):
    gen = _gen(cols)
    x = _values(gen, 37, cols, dtype=dtype)
    for center, wide in ((True, F32), (False, dtype)):
        w, b = _weights(gen, cols, wide, center)
        _check_forward(x, w, b, 1e-5, center, *_forward(x, w, b, center=center))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 31, 33, 255, 2049, 9001])
def test_forward_rows(rows, dtype):
    gen = _gen(rows)
    for cols in (64, 192, 1000):
        x = _values(gen, rows, cols, dtype=dtype)
        w, b = _weights(gen, cols, BF16)
        _check_forward(x, w, b, 1e-6, True, *_forward(x, w, b, eps=1e-6))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,pad,shift", [(64, 0, 1), (64, 3, 0), (128, 8, 8), (100, 1, 3), (1024, 5, 2), (1001, 0, 7)])
def test_forward_alignments_and_strides(cols, pad, shift, dtype):
    gen = _gen(1)
    w, b = _weights(gen, cols + 1, F32)
    w, b = w[1:], b[1:]                                       # off 16 bytes
    x = _values(gen, 50, cols, dtype=dtype, pad=pad, shift=shift)
    for out in (None, _values(gen, 50, cols, dtype=dtype, pad=pad + 2, shift=1)):
        _check_forward(x, w, b, 1e-5, True, *_forward(x, w, b, out=out))
    # heads of a wider tensor, tokens before heads and heads before tokens
    wide = _values(gen, 23, 9, cols, dtype=dtype, pad=pad, shift=shift)
    for t in (wide[:, 2:7], wide[:, 3:4], wide[5:6], wide.transpose(0, 1)[2:7], wide.transpose(0, 1)):
        _check_forward(t, w, b, 1e-5, False, *_forward(t, w, b, center=False))
    # one row for every head and token: strides of zero
    t = wide[:1, :1].expand(23, 5, cols)
    y, mean, rstd = _forward(t, w, b, out=torch.zeros(23, 5, cols, device=DEV, dtype=dtype))
    _check_forward(t, w, b, 1e-5, True, y, mean, rstd)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_writes_its_rows_only_and_takes_them_in_place(dtype):
    gen = _gen(2)
    for cols, heads in ((64, 3), (100, 3), (2049, 1)):
        buf = _values(gen, 40, heads + 2, cols, dtype=dtype, pad=5)
        whole = torch.as_strided(buf, (40 * (heads + 2) * (cols + 5) - 5,), (1,), buf.storage_offset())
        x = buf[:, 1:1 + heads]
        w, b = _weights(gen, cols, dtype)
        want = _forward(x.contiguous(), w, b)[0]
        before = whole.clone()
        y = _forward(x, w, b, out=x)[0]
        assert torch.equal(y, want)
        x.copy_(torch.as_strided(before, x.shape, x.stride(), x.storage_offset() - buf.storage_offset()))
        assert torch.equal(whole, before)


def test_forward_without_weights_statistics_or_rows():
    x = _values(_gen(3), 20, 300)
    _check_forward(x, None, None, 1e-5, True, *_forward(x))
    y = torch.zeros_like(x)
    mu.muon_layernorm_forward(Handle.get(), x, y)
    assert torch.equal(y, _forward(x)[0])
    mu.muon_layernorm_forward(Handle.get(), x[:0], y[:0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_one_value_and_far_from_zero(dtype):
    # no variance: xhat is zero and y the bias, with the mean exact
    x = torch.full((5, 256), 3.0, device=DEV, dtype=dtype)
    w, b = _weights(_gen(4), 256, dtype)
    y, mean, rstd = _forward(x, w, b, eps=1e-5)
    assert torch.equal(y, b.expand(5, 256)) and bool((mean == 3.0).all())
    assert bool(((rstd.double() * 1e-5 ** 0.5 - 1).abs() < 4 * U).all())
    # differences far below the mean: whole numbers, whose sums are exact
    x = (4096.0 + 32.0 * torch.arange(256, device=DEV).remainder(2) * torch.ones(3, 1, device=DEV)).to(dtype)
    y, mean, rstd = _forward(x, eps=0.0)
    assert bool((mean == 4112.0).all()) and bool((rstd == 1.0 / 16).all())
    assert torch.equal(y.float(), torch.where(torch.arange(256, device=DEV).remainder(2) == 1, 1.0, -1.0).expand(3, 256))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_stays_alone(value):
    for cols in (64, 100, 1000, 5000):
        x = _values(_gen(5), 70, cols)
        want = _forward(x)
        x[33, cols // 2] = value
        got = _forward(x)
        keep = torch.arange(70, device=DEV) != 33
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep])
        assert bool(torch.isnan(got[0][33, cols // 2])) and bool(torch.isnan(got[2][33]) | (got[2][33] == 0))


# ---- gradient ----------------------------------------------------------------------

def _grad(x, dy, mean, rstd, w, center, dw=None, db=None, dx=None, accumulate=False, wide=F32, **kw):
    cols = x.shape[-1]
    h = Handle.get()
    dx = torch.full_like(x, 7.0) if dx is None else dx
    dw = torch.full((cols,), 7.0, device=DEV, dtype=wide) if dw is None else dw
    db = torch.full((cols,), 7.0, device=DEV, dtype=wide) if db is None else db
    ws = torch.full((mu.muon_layernorm_workspace_size(h, x),), 255, dtype=torch.uint8, device=DEV)
    mu.muon_layernorm_grad(h, x, dy, rstd, ws, mean=mean if center else None, weight=w, dx=dx, dweight=dw, dbias=db,
                           accumulate=accumulate, center=center, **kw)
    return dx, dw, db


def _check_grad(x, dy, mean, rstd, w, center, dx, dw, db, held=None):
    n, cols = x.shape[0] * (x.shape[1] if x.dim() == 3 else 1), x.shape[-1]
    r = rstd.double()[..., None]
    hat = (x.double() - (mean.double()[..., None] if center else 0.0)) * r
    d = dy.double()
    g = d * (w.double() if w is not None else 1.0)
    s1, s2 = (g * hat).mean(-1, keepdim=True), g.mean(-1, keepdim=True) if center else torch.zeros_like(r)
    want = r * (g - s2 - hat * s1)
    a1 = (g * hat).abs().mean(-1, keepdim=True)
    off = r * (U * (6 * (g.abs() + s2.abs() + 2 * (hat * s1).abs())
                    + 70 * (hat.abs() * a1 + (g.abs().mean(-1, keepdim=True) if center else 0.0))))
    assert bool(((dx.double() - want).abs() <= off + _half(x.dtype) * (want.abs() + off)).all())
    rows = tuple(range(x.dim() - 1))
    for got, term, k in ((dw, d * hat, 0), (db, d, 1)):
        want = term.sum(rows) + (held[k].double() if held is not None else 0.0)
        off = (n + 4) * U * term.abs().sum(rows)
        assert bool(((got.double() - want).abs() <= off + _half(got.dtype) * (want.abs() + off)).all())


def _case(seed, *shape, dtype, center, pad=0, shift=0, wide=F32):
    gen = _gen(seed)
    x, dy = _values(gen, *shape, dtype=dtype, pad=pad, shift=shift), _values(gen, *shape, dtype=dtype, pad=pad)
    mean, rstd = (t.float() for t in _stats(x, 1e-5, center))
    return x, dy, mean, rstd, _weights(gen, shape[-1], wide)[0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", COLS)
def test_grad_widths(cols, dtype):
    for center, wide in ((True, F32), (False, dtype)):
        args = _case(cols, 37, cols, dtype=dtype, center=center, wide=wide)
        _check_grad(*args, center, *_grad(*args, center, wide=wide))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 31, 33, 255, 2049, 9001])
def test_grad_rows(rows, dtype):
    for cols in (64, 192, 1000):
        args = _case(rows, rows, cols, dtype=dtype, center=True)
        _check_grad(*args, True, *_grad(*args, True))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 40), (17, 128), (1000, 64), (4099, 100), (777, 1001), (3000, 513), (600, 4096),
                                       (520, 7168), (300, 16384)])
def test_every_row_is_in_the_column_sums(rows, cols, dtype):
    # whole numbers: every sum is below 2^24, and so exact in any order
    gen = _gen(rows)
    x, dy = (torch.randint(-3, 4, (rows, cols), generator=gen, device=DEV).to(dtype) for _ in range(2))
    one, zero = torch.ones(rows, device=DEV), torch.zeros(rows, device=DEV)
    _, dw, db = _grad(x, dy, zero, one, None, True)
    assert torch.equal(dw, (x.double() * dy.double()).sum(0).float())
    assert torch.equal(db, dy.double().sum(0).float())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,pad,shift", [(64, 0, 1), (64, 3, 0), (128, 8, 8), (100, 1, 3), (1024, 5, 2), (1001, 0, 7)])
def test_grad_alignments_and_strides(cols, pad, shift, dtype):
    args = _case(1, 50, cols, dtype=dtype, center=True, pad=pad, shift=shift)
    _check_grad(*args, True, *_grad(*args, True, dx=_values(_gen(9), 50, cols, dtype=dtype, pad=pad + 2, shift=1)))
    x, dy, mean, rstd, w = _case(2, 23, 9, cols, dtype=dtype, center=False, pad=pad, shift=shift)
    for cut in (lambda t: t[:, 2:7], lambda t: t[:, 3:4], lambda t: t[5:6], lambda t: t.transpose(0, 1)[2:7]):
        args = cut(x), cut(dy), cut(mean).contiguous(), cut(rstd).contiguous(), w
        _check_grad(*args, False, *_grad(*args, False))
    # one gradient for every row, as that of a sum: strides of zero
    args = x[:, 2:7], dy[:1, :1].expand(23, 5, cols), mean[:, 2:7].contiguous(), rstd[:, 2:7].contiguous(), w
    _check_grad(*args, False, *_grad(*args, False, dx=torch.zeros(23, 5, cols, device=DEV, dtype=dtype)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [64, 100, 1000, 7168])
def test_grad_in_place_alone_and_added(cols, dtype):
    args = _case(3, 300, cols, dtype=dtype, center=True)
    x, dy, mean, rstd, w = args
    dx, dw, db = _grad(*args, True)
    again = _grad(*args, True)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))     # a fixed order
    for into in (0, 1):
        a = [t.clone() for t in args]
        got = _grad(*a, True, dx=a[into])
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
    h = Handle.get()
    ws = torch.empty(mu.muon_layernorm_workspace_size(h, x), dtype=torch.uint8, device=DEV)
    for kw in (dict(dx=dx), dict(dweight=dw), dict(dbias=db)):
        (name, want), = kw.items()
        out = torch.full_like(want, 7.0)
        mu.muon_layernorm_grad(h, x, dy, rstd, ws, mean=mean, weight=w, **{name: out})
        assert torch.equal(out, want)
    held = torch.randn(2, cols, generator=_gen(4), device=DEV).to(dtype)
    got = _grad(*args, True, dw=held[0].clone(), db=held[1].clone(), accumulate=True)
    _check_grad(*args, True, *got, held=held)


def test_grad_without_rows():
    args = _case(5, 4, 50, dtype=F32, center=True)
    none = tuple(t[:0] for t in args[:4]) + (args[4],)
    _, dw, db = _grad(*none, True)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0
    _, dw, db = _grad(*none, True, accumulate=True)
    assert bool((dw == 7.0).all()) and bool((db == 7.0).all())


def test_grad_of_a_row_that_is_not_finite_stays_alone():
    for cols in (64, 1000):
        args = _case(6, 70, cols, dtype=F32, center=True)
        want = _grad(*args, True)[0]
        args[1][33, 5] = float("nan")
        dx, dw, db = _grad(*args, True)
        keep = torch.arange(70, device=DEV) != 33
        assert torch.equal(dx[keep], want[keep]) and bool(torch.isnan(dx[33]).all())
        at = torch.arange(cols, device=DEV) == 5
        assert torch.equal(torch.isnan(dw), at) and torch.equal(torch.isnan(db), at)


@pytest.mark.parametrize("center", [True, False])
def test_grad_against_differences(center):
    # L = sum(y * dy): central differences of the formula in 64 bits along random directions
    x, dy, mean, rstd, w = _case(7, 6, 96, dtype=F32, center=center)
    b = torch.zeros_like(w)
    dx, dw, db = _grad(x, dy, mean, rstd, w, center)

    def loss(x, w, b):
        m, r = _stats(x, 1e-5, center)
        return float((((x.double() - m[..., None]) * r[..., None] * w.double() + b.double()) * dy.double()).sum())

    gen, t = _gen(8), 1e-5
    for k, grad in enumerate((dx, dw, db)):
        at = [x.double(), w.double(), b.double()]
        v = torch.randn(at[k].shape, generator=gen, device=DEV, dtype=torch.float64)
        ends = []
        for s in (t, -t):
            moved = list(at)
            moved[k] = at[k] + s * v
            ends.append(loss(*moved))
        slope, scale = (ends[0] - ends[1]) / (2 * t), float((grad.double() * v).abs().sum())
        # the differences' own error: t^2 times third derivatives, and 2^-52 |L| / t
        assert abs(float((grad.double() * v).sum()) - slope) <= 1e-5 * scale


def test_streams_and_a_captured_graph():
    args = _case(11, 500, 1000, dtype=BF16, center=True)
    x, dy, mean, rstd, w = args
    h = Handle.get()
    y, m, r = _forward(x, w)
    dx, dw, db = _grad(*args, True)
    outs = [torch.zeros_like(t) for t in (y, m, r, dx, dw, db)]
    ws = torch.empty(mu.muon_layernorm_workspace_size(h, x), dtype=torch.uint8, device=DEV)

    def both(stream):
        mu.muon_layernorm_forward(h, x, outs[0], weight=w, mean=outs[1], rstd=outs[2], stream=stream)
        mu.muon_layernorm_grad(h, x, dy, rstd, ws, mean=mean, weight=w, dx=outs[3], dweight=outs[4], dbias=outs[5],
                               stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(outs, (y, m, r, dx, dw, db)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(None)
    for seed in (20, 21, 22):
        new = _case(seed, 500, 1000, dtype=BF16, center=True)
        for a, b in zip(args, new):
            a.copy_(b)
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, _forward(x, w) + _grad(*args, True)):
            assert torch.equal(a, b)


# ---- large tensors --------------------------------------------------------------------

@pytest.mark.parametrize("dtype,rows,cols", [(BF16, 500003, 128), (F32, 200001, 130), (BF16, 70001, 1000),
                                             (F32, 26001, 1001), (BF16, 9001, 7168)])
def test_large_tensors_are_their_parts(dtype, rows, cols):
    # beyond 96 MiB rows are read around the caches, and workgroups take many of them
    gen = _gen(rows)
    x, dy = (torch.randint(-4, 5, (rows, cols), generator=gen, device=DEV, dtype=torch.int8).to(dtype) for _ in range(2))
    assert x.nbytes >= 96 << 20
    w, b = _weights(gen, cols, F32)
    y, mean, rstd = _forward(x, w, b)
    one = torch.ones(rows, device=DEV)
    dx, dw, db = _grad(x, dy, mean, one, w, True)
    step = 7001
    for a in range(0, rows, rows // 3):
        cut = slice(a, min(a + step, rows))
        for got, want in zip((y, mean, rstd), _forward(x[cut], w, b)):
            assert torch.equal(got[cut], want)
        assert torch.equal(dx[cut], _grad(x[cut], dy[cut], mean[cut], one[cut], w, True)[0])
    # whole numbers below 2^24: exact in any order
    zero = torch.zeros(rows, device=DEV)
    _, dw, db = _grad(x, dy, zero, one, None, True)
    assert torch.equal(db, dy.sum(0, dtype=torch.float64).float())
    want = torch.zeros(cols, device=DEV, dtype=torch.float64)
    for a in range(0, rows, 100000):
        want += (x[a:a + 100000].float() * dy[a:a + 100000].float()).sum(0, dtype=torch.float64)
    assert torch.equal(dw, want.float())


def test_rows_far_apart():
    # 2^31 elements and more between a tensor's first and last row
    cols, far = 200, (1 << 30) + 8
    buf = torch.zeros(2 * far + cols, device=DEV, dtype=BF16)
    x = torch.as_strided(buf, (3, cols), (far, 1))
    small = _values(_gen(1), 3, cols, dtype=BF16)
    w, b = _weights(_gen(2), cols, BF16)
    x.copy_(small)
    want = _forward(small, w, b)
    for got, ref in zip(_forward(x, w, b), want):
        assert torch.equal(got, ref)
    args = small, _values(_gen(3), 3, cols, dtype=BF16), want[1], want[2], w
    ref = _grad(*args, True)
    into = torch.as_strided(buf, (3, cols), (far, 1))
    got = _grad(x, *args[1:], True, dx=into)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("cols", [64, 100, 1000, 7168])
def test_grad_of_tiny_and_of_huge_rows(cols):
    # rstd^2 and rstd^3 leave fp32, dx does not
    for size in (1e-25, 1e25):
        gen = _gen(cols)
        x, dy = (torch.randn(30, cols, generator=gen, device=DEV) for _ in range(2))
        x *= size
        rstd = torch.full((30,), 1.0 / size, device=DEV)
        mean = x.double().mean(1).float()
        args = x, dy, mean, rstd, _weights(gen, cols, F32)[0]
        got = _grad(*args, True)
        assert all(bool(torch.isfinite(t).all()) for t in got)
        _check_grad(*args, True, *got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_row_for_every_token_next_to_its_output(dtype):
    # a gradient as that of a sum, and its output right behind it in one buffer
    tokens, cols = 500, 64
    buf = _values(_gen(12), tokens + 2, cols, dtype=dtype).contiguous()
    w, b = _weights(_gen(13), cols, F32)
    one, out = buf[:1].expand(tokens, cols), buf[1:tokens + 1]
    first, last = buf[0].clone(), buf[-1].clone()
    _check_forward(one, w, b, 1e-5, True, *_forward(one, w, b, out=out))
    x = _values(_gen(14), tokens, cols, dtype=dtype)
    mean, rstd = (t.float() for t in _stats(x, 1e-5, True))
    _check_grad(x, one, mean, rstd, w, True, *_grad(x, one, mean, rstd, w, True, dx=out))
    assert torch.equal(buf[0], first) and torch.equal(buf[-1], last)
    with pytest.raises(mu.MuonError, match="MUON_ERR_OVERLAP"):
        _forward(one, w, b, out=buf[:tokens])


@pytest.mark.parametrize("cols", [64, 100, 1000, 7168])
def test_rows_beyond_what_fp32_squares_and_sums(cols):
    sign = torch.where(torch.arange(cols, device=DEV) % 2 == 0, 1.0, -1.0)
    w, b = _weights(_gen(15), cols, F32)
    x = _values(_gen(16), 40, cols)
    want = _forward(x, w, b)
    x[5] = 1e25 * sign              # squares beyond fp32
    x[6] = 3e38                     # the sum itself
    x[7] = 1e-25 * sign             # no squares left: eps alone
    y, mean, rstd = _forward(x, w, b)
    assert float(rstd[5]) == 0.0 and torch.equal(y[5], b)
    assert not bool(torch.isfinite(mean[6])) and bool(torch.isnan(y[6]).all())
    assert abs(float(rstd[7]) * 1e-5 ** 0.5 - 1.0) <= 4 * U
    assert bool(((y[7] - b).abs() <= 2.0 ** -24 * b.abs() + 1e-20).all())
    assert float(_forward(x[7:8], w, b, eps=0.0)[2]) == float("inf")
    keep = [i for i in range(40) if i not in (5, 6, 7)]
    for got, ref in zip((y, mean, rstd), want):
        assert torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [7, 33, 64, 100, 513, 1024, 1001, 2049, 7168])
def test_bf16_weights_off_four_bytes(cols, dtype):
    gen = _gen(cols)
    w, b = (t[1:] for t in _weights(gen, cols + 1, BF16))
    x = _values(gen, 41, cols, dtype=dtype)
    _check_forward(x, w, b, 1e-5, True, *_forward(x, w, b))
    held = torch.full((2, cols + 2), 7.0, device=DEV, dtype=BF16)
    mean, rstd = (t.float() for t in _stats(x, 1e-5, True))
    dy = _values(gen, 41, cols, dtype=dtype)
    dw, db = held[0, 1:-1], held[1, 1:-1]
    _check_grad(x, dy, mean, rstd, w, True, *_grad(x, dy, mean, rstd, w, True, dw=dw, db=db))
    assert bool((held[:, 0] == 7).all()) and bool((held[:, -1] == 7).all())
