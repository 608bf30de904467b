"""Products grouped by expert against 64-bit products.

Whole numbers: with inputs of small integers every product and every partial
sum is a whole number below 2^24, exact in fp32 in any order, so the results
have to be the 64-bit ones rounded once to the output's type, bit for bit.

Other inputs: a sum of K products in fp32 is off by at most one step (2^-23
relative) of every partial sum, (K + 1) * 2^-23 * sum |a b| in all, and the
rounding to the output's type, 2^-8 for bf16 and 2^-24 for fp32."""

import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _ints(gen, shape, dtype, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen, device=DEV).to(dtype)


def _offsets(sizes, first=0):
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    return at, torch.tensor(at, dtype=torch.int32, device=DEV)


def _round(x, dtype):
    # whole numbers below 2^24 pass through fp32 unchanged
    return x.float().to(dtype)


class Layer:
    """Weights, tokens and gradients of one layer, leading dimensions padded."""

    def __init__(self, sizes, rows, cols, dtype, seed=0, spare=3, first=0, pad=0, grad_dtype=None,
                 shift=0, values=_ints):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.sizes, self.rows, self.cols, self.dtype = sizes, rows, cols, dtype
        self.at, self.offsets = _offsets(sizes, first)
        self.held = self.at[-1] + spare

        def tensor(n, width, dt):
            flat = values(gen, (n * (width + pad) + shift,), dt)
            return flat[shift:].view(n, width + pad)[:, :width]

        E = len(sizes)
        self.w = [tensor(rows, cols, dtype) for _ in range(E)]
        self.x = tensor(self.held, cols, dtype)
        self.dy = tensor(self.held, rows, dtype)
        self.y = tensor(self.held, rows, dtype)
        self.dx = tensor(self.held, cols, dtype)
        self.dw = [tensor(rows, cols, grad_dtype or dtype) for _ in range(E)]

    def groups(self):
        return [(e, a, b) for e, (a, b) in enumerate(zip(self.at, self.at[1:]))]

    def want_y(self):
        y = self.y.clone()
        for e, a, b in self.groups():
            y[a:b] = _round(self.x[a:b].double() @ self.w[e].double().t(), self.dtype)
        return y

    def want_dx(self):
        dx = self.dx.clone()
        for e, a, b in self.groups():
            dx[a:b] = _round(self.dy[a:b].double() @ self.w[e].double(), self.dtype)
        return dx

    def want_dw(self, accumulate):
        out = []
        for e, a, b in self.groups():
            g = self.dy[a:b].double().t() @ self.x[a:b].double()
            out.append(_round(self.dw[e].double() + g if accumulate else g, self.dw[e].dtype))
        return out

    def check(self, h=None, stream=None):
        """Every product, bit for bit; values around the outputs stay."""
        h = h or Handle.get()
        ex, gr = mu.muon_experts(self.w), mu.muon_experts(self.dw)
        want_y, want_dx = self.want_y(), self.want_dx()
        around = [_outside(t) for t in (self.y, self.dx)]
        mu.muon_expert_forward(h, ex, self.offsets, self.x, self.y, stream=stream)
        mu.muon_expert_grad_input(h, ex, self.offsets, self.dy, self.dx, stream=stream)
        torch.cuda.synchronize()
        _same(self.y, want_y, "forward")
        _same(self.dx, want_dx, "input gradient")
        for t, k in zip((self.y, self.dx), around):
            assert torch.equal(_outside(t), k)
        for accumulate in (True, False):
            want = self.want_dw(accumulate)
            around = [_outside(t) for t in self.dw]
            mu.muon_expert_grad_weight(h, gr, self.offsets, self.x, self.dy, accumulate=accumulate,
                                       stream=stream)
            torch.cuda.synchronize()
            for e, (g, k) in enumerate(zip(self.dw, want)):
                _same(g, k, "weight gradient %d, accumulate %s" % (e, accumulate))
                assert torch.equal(_outside(g), around[e])


def _outside(t):
    """What lies between and around the rows of a view: not to be written."""
    base = t._base if t._base is not None else t
    flat = base.reshape(-1).clone()
    mask = torch.ones_like(flat, dtype=torch.bool)
    if t.numel():
        torch.as_strided(mask, t.shape, t.stride(), t.storage_offset()).fill_(False)
    return flat[mask]


def _same(got, want, what):
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        raise AssertionError((what, len(bad), bad[:4].tolist(), got[tuple(bad[0])].item(),
                              want[tuple(bad[0])].item()))


SIZES = {
    "one token": [1],
    "one expert": [70],
    "some empty": [0, 5, 0, 0, 64, 1, 0],
    "all empty": [0, 0],
    "tile edges": [63, 64, 65, 127, 128, 129],
    "skewed": [3, 300, 1, 2, 17, 257],
}
# (rows, cols): the K of one product is the width of another
WIDTHS = [(64, 64), (128, 256), (8, 16), (1, 1), (7, 5), (33, 65), (200, 72), (264, 520)]


@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)],
                         ids=["bf16", "bf16 to fp32", "fp32"])
@pytest.mark.parametrize("widths", WIDTHS, ids=str)
@pytest.mark.parametrize("sizes", SIZES.values(), ids=list(SIZES))
def test_products(sizes, widths, dtype, grad_dtype):
    Layer(sizes, *widths, dtype, grad_dtype=grad_dtype).check()


@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, F32), (F32, F32)], ids=["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift,first", [(8, 0, 0), (3, 0, 2), (0, 1, 0), (5, 3, 9), (64, 8, 0)])
def test_strides_alignments_and_rows_before_the_first_group(pad, shift, first, dtype, grad_dtype):
    Layer([30, 0, 70, 4], 96, 136, dtype, grad_dtype=grad_dtype, pad=pad, shift=shift, first=first).check()


@pytest.mark.parametrize("experts", [63, 64, 65, 129, 300, 1024])
def test_many_experts(experts):
    r = torch.Generator().manual_seed(experts)
    sizes = torch.randint(0, 4, (experts,), generator=r).tolist()
    Layer(sizes, 24, 40, BF16, grad_dtype=F32, seed=experts).check()


@pytest.mark.parametrize("sizes,rows,cols", [
    ([256, 1000, 0, 513], 512, 768), ([700], 1000, 2056), ([40, 31, 33, 8, 0, 129, 16, 3], 640, 1152),
    ([2, 1, 1, 0, 0, 3, 1, 0, 8, 1], 1024, 2048)])
def test_larger_products(sizes, rows, cols):
    Layer(sizes, rows, cols, BF16, grad_dtype=F32).check()


def _close(got, want, bound, dtype, what):
    tol = bound + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * (want.abs() + bound)
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)],
                         ids=["bf16", "bf16 to fp32", "fp32"])
def test_products_of_other_values(dtype, grad_dtype):
    def normal(gen, shape, dt):
        return torch.randn(shape, generator=gen, device=DEV).to(dt)

    L = Layer([300, 0, 5, 129], 328, 712, dtype, grad_dtype=grad_dtype, values=normal)
    h, step = Handle.get(), 2.0 ** -23
    ex, gr = mu.muon_experts(L.w), mu.muon_experts(L.dw)
    old = [g.clone() for g in L.dw]
    mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y)
    mu.muon_expert_grad_input(h, ex, L.offsets, L.dy, L.dx)
    mu.muon_expert_grad_weight(h, gr, L.offsets, L.x, L.dy, accumulate=True)
    for e, a, b in L.groups():
        x, dy, w = L.x[a:b].double(), L.dy[a:b].double(), L.w[e].double()
        _close(L.y[a:b], x @ w.t(), (L.cols + 1) * step * (x.abs() @ w.abs().t()), dtype, "forward")
        _close(L.dx[a:b], dy @ w, (L.rows + 1) * step * (dy.abs() @ w.abs()), dtype, "input gradient")
        o = old[e].double()
        _close(L.dw[e], o + dy.t() @ x, (b - a + 2) * step * (dy.abs().t() @ x.abs() + o.abs()), grad_dtype,
               "weight gradient")


def test_gradients_are_those_of_the_forward():
    """<forward(x + t), dy> - <forward(x), dy> = <t, dx>, and the same for the
    weights: differences of a linear map, exact on whole numbers."""
    h = Handle.get()
    L = Layer([9, 0, 40, 17], 48, 56, F32, spare=0)
    gen = torch.Generator(device=DEV).manual_seed(5)
    t = _ints(gen, L.x.shape, F32)
    tw = [_ints(gen, w.shape, F32) for w in L.w]

    def loss(x, w):
        y = torch.zeros_like(L.y)
        mu.muon_expert_forward(h, mu.muon_experts(w), L.offsets, x, y)
        return float((y.double() * L.dy.double()).sum())

    mu.muon_expert_grad_input(h, mu.muon_experts(L.w), L.offsets, L.dy, L.dx)
    mu.muon_expert_grad_weight(h, mu.muon_experts(L.dw), L.offsets, L.x, L.dy)
    base = loss(L.x, L.w)
    assert loss(L.x + t, L.w) - base == float((t.double() * L.dx.double()).sum())
    assert loss(L.x, [a + b for a, b in zip(L.w, tw)]) - base == \
        sum(float((a.double() * g.double()).sum()) for a, g in zip(tw, L.dw))


def test_one_weight_for_two_experts():
    L = Layer([20, 30], 40, 48, BF16)
    L.w = [L.w[0], L.w[0]]
    want = L.want_y()
    mu.muon_expert_forward(Handle.get(), mu.muon_experts(L.w), L.offsets, L.x, L.y)
    _same(L.y, want, "forward")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_non_finite_values_stay_in_their_group(value, dtype):
    """Rows of another group, and rows behind the last one, never leak in."""
    sizes, rows, cols = [30, 50, 20], 72, 136
    a, b = Layer(sizes, rows, cols, dtype), Layer(sizes, rows, cols, dtype)
    for t in (b.x, b.dy):
        t[30:80] = value
        t[100:] = value
    b.w[1].fill_(value)
    h = Handle.get()
    for L in (a, b):
        ex, gr = mu.muon_experts(L.w), mu.muon_experts(L.dw)
        mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y)
        mu.muon_expert_grad_input(h, ex, L.offsets, L.dy, L.dx)
        mu.muon_expert_grad_weight(h, gr, L.offsets, L.x, L.dy)
    for got, want in ((b.y, a.y), (b.dx, a.dx)):
        assert torch.equal(got[:30], want[:30]) and torch.equal(got[80:], want[80:])
        assert not bool(torch.isfinite(got[30:80]).any())
    for e in (0, 2):
        assert torch.equal(a.dw[e], b.dw[e])
    assert not bool(torch.isfinite(b.dw[1]).any())


@pytest.mark.parametrize("bad", [[0, -5, 40, 50], [0, 60, 20, 50], [5, 100000, 2000000000, 7],
                                 [-2000000000, 10, 10, 2147483647], [50, 40, 30, 20]])
def test_offsets_that_make_no_sense_reach_no_memory(bad):
    """Clamped into [0, tokens] and to ascending order: rows beyond the tensors
    and values around them stay; what the rows get is not specified."""
    L = Layer([10, 20, 20], 72, 88, BF16, grad_dtype=F32, pad=8, spare=0)
    L.offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
    around = [_outside(t) for t in [L.y, L.dx] + L.dw]
    h = Handle.get()
    mu.muon_expert_forward(h, mu.muon_experts(L.w), L.offsets, L.x, L.y)
    mu.muon_expert_grad_input(h, mu.muon_experts(L.w), L.offsets, L.dy, L.dx)
    mu.muon_expert_grad_weight(h, mu.muon_experts(L.dw), L.offsets, L.x, L.dy)
    torch.cuda.synchronize()
    for t, k in zip([L.y, L.dx] + L.dw, around):
        assert torch.equal(_outside(t), k)


def test_no_tokens():
    L = Layer([0, 0], 16, 24, BF16, spare=0)
    h = Handle.get()
    mu.muon_expert_forward(h, mu.muon_experts(L.w), L.offsets, L.x, L.y)
    keep = [g.clone() for g in L.dw]
    mu.muon_expert_grad_weight(h, mu.muon_experts(L.dw), L.offsets, L.x, L.dy, accumulate=True)
    assert all(torch.equal(a, b) for a, b in zip(keep, L.dw))
    mu.muon_expert_grad_weight(h, mu.muon_experts(L.dw), L.offsets, L.x, L.dy)
    assert all(int(torch.count_nonzero(g)) == 0 for g in L.dw)


def test_another_stream_and_a_captured_graph():
    h = Handle.get()
    sizes = ([40, 0, 90, 7], [1, 70, 0, 66], [137, 0, 0, 0])
    s = torch.cuda.Stream()
    for n in sizes:
        L = Layer(n, 136, 72, BF16, grad_dtype=F32)
        torch.cuda.synchronize()
        L.check(h, stream=s)
    # the group sizes are read when the graph runs
    L = Layer(sizes[0], 136, 72, BF16, grad_dtype=F32, spare=0)
    ex, gr = mu.muon_experts(L.w), mu.muon_experts(L.dw)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y)
        mu.muon_expert_grad_input(h, ex, L.offsets, L.dy, L.dx)
        mu.muon_expert_grad_weight(h, gr, L.offsets, L.x, L.dy)
    for n in sizes + sizes:
        L.at, off = _offsets(n)
        L.offsets.copy_(off)
        L.x.mul_(-1)
        want = [L.want_y(), L.want_dx()] + L.want_dw(False)
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip([L.y, L.dx] + L.dw, want):
            _same(got, w, "replay")


def test_offsets_beyond_32_bits():
    # x and y hold more than 2^31 elements; the last group lies behind them
    K, N, T = 4096, 16, (1 << 19) + 300
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.zeros(T, K, dtype=BF16, device=DEV)
    x[-300:] = _ints(gen, (300, K), BF16)
    w = [_ints(gen, (N, K), BF16) for _ in range(2)]
    y = torch.zeros(T, N, dtype=BF16, device=DEV)
    off = torch.tensor([0, T - 300, T], dtype=torch.int32, device=DEV)
    h = Handle.get()
    mu.muon_expert_forward(h, mu.muon_experts(w), off, x, y)
    _same(y[-300:], _round(x[-300:].double() @ w[1].double().t(), BF16), "forward")
    assert int(torch.count_nonzero(y[:-300])) == 0
    dw = [torch.ones(N, K, device=DEV) for _ in range(2)]
    dy = torch.zeros(T, N, dtype=BF16, device=DEV)
    dy[-300:] = _ints(gen, (300, N), BF16)
    mu.muon_expert_grad_weight(h, mu.muon_experts(dw), off, x, dy)
    _same(dw[1], (dy[-300:].double().t() @ x[-300:].double()).float(), "weight gradient")
    assert int(torch.count_nonzero(dw[0])) == 0
    dx = x
    mu.muon_expert_grad_input(h, mu.muon_experts(w), off, dy, dx)
    _same(dx[-300:], _round(dy[-300:].double() @ w[1].double(), BF16), "input gradient")


def test_binding_refuses():
    L = Layer([4, 5], 16, 24, BF16)
    h, ex = Handle.get(), mu.muon_experts(L.w)
    with pytest.raises(ValueError):
        mu.muon_experts([L.w[0], L.w[1][:, :8]])
    with pytest.raises(ValueError):
        mu.muon_experts([L.w[0], L.w[1].float()])
    with pytest.raises(ValueError):
        mu.muon_expert_forward(h, ex, L.offsets[:2], L.x, L.y)
    with pytest.raises(ValueError):
        mu.muon_expert_forward(h, ex, L.offsets.long(), L.x, L.y)
    with pytest.raises(ValueError):
        mu.muon_expert_forward(h, ex, L.offsets, L.x[:, :8], L.y)
    with pytest.raises(ValueError):
        mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y[:-1])
    with pytest.raises(TypeError):
        mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y.float())
    with pytest.raises(ValueError):
        mu.muon_expert_forward(h, ex, L.offsets.cpu(), L.x, L.y)
    with pytest.raises(ValueError):
        mu.muon_expert_grad_weight(h, ex, L.offsets, L.dy, L.x)
    with pytest.raises(mu.MuonError) as e:
        mu.muon_expert_grad_input(h, ex, L.offsets, L.dy, L.w[0].as_strided(L.dx.shape, (24, 1), 0))
    assert e.value.status == 4


# Groups whose tiles end in each of the eight 32-row blocks of a 256-row tile,
# wide enough that 256-wide tiles are taken (forward, and the input gradient with
# the widths exchanged); K of one to thirteen slabs, whole and ragged, so that
# the loop over six slabs ends at each of them.
@pytest.mark.parametrize("k", [8, 64, 72, 128, 192, 264, 320, 384, 392, 456, 512, 640, 704, 768, 776])
def test_wide_tiles(k):
    sizes = [225, 193, 200, 161, 100, 33, 256, 1, 289]
    Layer(sizes, 4104, k, BF16, seed=k).check()
    Layer(sizes, k, 4104, BF16, seed=k + 1, pad=8).check()


# bf16 rows that do not start on 16 bytes, enough of them for the 128 x 128 tiles
# that go through registers: taken from 4096 tiles of 64 x 64 on.  Rows: 8000 / 64
# + 4 groups = 129 tiles by at least 32; weights: 4 experts by 32 x 33.
@pytest.mark.parametrize("grad_dtype", [BF16, F32], ids=["bf16", "bf16 to fp32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(2049, 2057, 0, 0), (2048, 2112, 1, 0), (2048, 2112, 8, 3)],
                         ids=["odd widths", "odd leading dimensions", "odd starts"])
def test_large_products_at_other_alignments(rows, cols, pad, shift, grad_dtype):
    Layer([3000, 0, 4097, 903], rows, cols, BF16, grad_dtype=grad_dtype, pad=pad, shift=shift, seed=rows + pad).check()


def test_large_products_at_other_alignments_read_no_other_group():
    """As the test of non-finite values above, for 128 x 128 tiles; rows of a
    group end inside a tile and inside a chunk of 8."""
    sizes, rows, cols = [3001, 4097, 902], 2049, 2057
    a, b = (Layer(sizes, rows, cols, BF16, grad_dtype=F32, seed=9) for _ in range(2))
    for t in (b.x, b.dy):
        t[3001:7098] = float("nan")
        t[8000:] = float("nan")
    b.w[1].fill_(float("nan"))
    h = Handle.get()
    for L in (a, b):
        ex, gr = mu.muon_experts(L.w), mu.muon_experts(L.dw)
        mu.muon_expert_forward(h, ex, L.offsets, L.x, L.y)
        mu.muon_expert_grad_input(h, ex, L.offsets, L.dy, L.dx)
        mu.muon_expert_grad_weight(h, gr, L.offsets, L.x, L.dy)
    for got, want in ((b.y, a.y), (b.dx, a.dx)):
        assert torch.equal(got[:3001], want[:3001]) and torch.equal(got[7098:], want[7098:])
    for e in (0, 2):
        assert torch.equal(a.dw[e], b.dw[e])


# Above 128 experts the kernels take longer lists of pointers, as variants of their
# own: 32 x 64, 128 x 128 and 256 x 256 tiles (by the rows of a group), tiles
# through registers of both sizes, and fp32.
@pytest.mark.parametrize("mean,rows,cols,dtype,grad_dtype", [
    (4, 256, 264, BF16, F32), (40, 264, 256, BF16, BF16), (200, 256, 256, BF16, F32), (20, 65, 63, BF16, BF16),
    (40, 1301, 383, BF16, F32), (20, 72, 100, F32, F32)],
    ids=["few rows", "128 x 128", "256 x 256", "registers", "registers, 128 x 128", "fp32"])
def test_more_than_128_experts(mean, rows, cols, dtype, grad_dtype):
    r = torch.Generator().manual_seed(mean)
    sizes = (torch.rand(130, generator=r) * 2 * mean).int().tolist()
    Layer(sizes, rows, cols, dtype, grad_dtype=grad_dtype, seed=rows).check()
