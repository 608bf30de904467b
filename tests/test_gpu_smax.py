"""The largest attention logit of every head against 64-bit logits.

Whole numbers: with q and k of small integers every logit is a whole number
that fp32 holds exactly, so the maximum times the scale has to come out as that
product rounded once.  Other values: a sum of D products in fp32 is off by at
most (D + 1) * 2^-23 * sum |q k| (one step per partial sum), then the scale's
product by 2^-24."""

import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NEG = -float("inf")


def _cu(sizes):
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return at, torch.tensor(at, dtype=torch.int32, device=DEV)


def _reference(q, k, at_q, at_k, scale, causal):
    """(largest logit, bound of its fp32 error) per query head, in 64 bits."""
    H, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    top = torch.full((H,), NEG, dtype=torch.float64, device=DEV)
    err = torch.zeros(H, dtype=torch.float64, device=DEV)
    for (a, b), (c, d) in zip(zip(at_q, at_q[1:]), zip(at_k, at_k[1:])):
        if a == b or c == d:
            continue
        mask = torch.ones(b - a, d - c, dtype=torch.bool, device=DEV)
        if causal:
            mask = mask.tril((d - c) - (b - a))
        if not bool(mask.any()):
            continue
        for h in range(H):
            x, y = q[a:b, h].double(), k[c:d, h // (H // Hk)].double().t().contiguous()
            z = (x @ y).masked_fill(~mask, NEG)
            top[h] = torch.maximum(top[h], z.max())
            err[h] = torch.maximum(err[h], ((x.abs() @ y.abs()) * mask).max() * (D + 1) * 2.0 ** -23)
    return top * scale, err * scale


def _call(q, k, cu_q, cu_k, scale, causal, **kw):
    h = Handle.get()
    sq = torch.full((q.shape[1],), 77.0, device=DEV)
    sk = torch.full((k.shape[1],), 77.0, device=DEV)
    ws = torch.full((mu.muon_qk_smax_workspace_size(h, q, k, cu_q),), 255, dtype=torch.uint8, device=DEV)
    mu.muon_qk_smax(h, q, k, cu_q, cu_k, sq, ws, smax_k=sk, scale=scale, causal=causal, **kw)
    return sq, sk


def _ints(seed, tokens, heads, dim, dtype, pad=0, shift=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    flat = torch.randint(-3, 4, (tokens * heads * (dim + pad) + shift,), generator=gen, device=DEV)
    return flat.to(dtype)[shift:].view(tokens, heads, dim + pad)[..., :dim]


def _check_whole(q, k, nq, nk, causal, scale=0.37):
    at_q, cu_q = _cu(nq)
    at_k, cu_k = _cu(nk)
    sq, sk = _call(q, k, cu_q, cu_k, scale, causal)
    want, _ = _reference(q, k, at_q, at_k, 1.0, causal)
    want = want.float() * torch.tensor(scale, device=DEV)
    assert torch.equal(sq, want), (sq, want)
    assert torch.equal(sk, want.view(k.shape[1], -1).amax(1))


LENGTHS = {
    "one token": ([1], [1]),
    "one query, many keys": ([1], [777]),
    "tile edges": ([63, 64, 65, 127, 128, 129], [63, 64, 65, 127, 128, 129]),
    "packed": ([5, 300, 1, 33, 257], [5, 300, 1, 33, 257]),
    "keys before the queries": ([5, 130, 1, 64], [9, 140, 400, 64]),
    "fewer keys than queries": ([70, 5], [9, 3]),
    "empty sequences": ([0, 4, 0, 66, 3, 0], [0, 4, 7, 66, 0, 0]),
}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", LENGTHS.values(), ids=list(LENGTHS))
def test_lengths_and_masks(lengths, causal, dtype):
    nq, nk = lengths
    q, k = _ints(1, sum(nq), 4, 64, dtype), _ints(2, sum(nk), 2, 64, dtype)
    _check_whole(q, k, nq, nk, causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [1, 3, 16, 32, 40, 63, 80, 96, 128, 129, 160, 192, 256, 264, 576])
def test_head_sizes(dim, dtype):
    n = [70, 200]
    _check_whole(_ints(3, 270, 4, dim, dtype), _ints(4, 270, 4, dim, dtype), n, n, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 2), (7, 7), (16, 1), (64, 8)])
def test_head_layouts(heads, kv, dtype):
    n = [3, 90, 65]
    _check_whole(_ints(5, 158, heads, 128, dtype), _ints(6, 158, kv, 128, dtype), n, n, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (5, 3), (64, 8)])
def test_strides_and_alignments(pad, shift, dtype):
    n = [100, 31]
    q, k = (_ints(s, 131, 4, 64, dtype, pad, shift) for s in (7, 8))
    _check_whole(q, k, n, n, True)
    # heads before tokens
    q, k = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
    _check_whole(q, k, n, n, True)
    # one key for every token: a stride of zero
    _check_whole(q, k[:1].expand(131, 4, 64), n, n, True)


@pytest.mark.parametrize("n", [1000, 2049])
def test_longer_sequences(n):
    _check_whole(_ints(9, n, 8, 128, BF16), _ints(10, n, 2, 128, BF16), [n], [n], True)
    _check_whole(_ints(9, n, 2, 192, BF16), _ints(10, n, 2, 192, BF16), [n], [n], False)


@pytest.mark.parametrize("where", [(0, 0), (5, 5), (140, 3), (140, 139), (299, 299), (299, 0), (63, 63),
                                   (64, 63), (128, 127)])
def test_the_one_largest_pair_is_found_and_masked_ones_are_not(where):
    i, j = where
    q, k = torch.zeros(300, 2, 64, device=DEV, dtype=BF16), torch.zeros(300, 2, 64, device=DEV, dtype=BF16)
    q[i, 1, 17], k[j, 1, 17] = 8.0, 16.0
    q[j, 0, 5], k[i, 0, 5] = 8.0, 16.0      # the mirrored pair: masked unless on the diagonal
    _, cu = _cu([300])
    sq, _ = _call(q, k, cu, cu, 0.5, True)
    assert sq.tolist() == [64.0 if i == j else 0.0, 64.0]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_other_values(dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    nq, nk = [100, 1, 513, 77], [100, 40, 513, 90]
    q = (torch.randn(sum(nq), 8, 128, generator=gen, device=DEV) * 3).to(dtype)
    k = torch.randn(sum(nk), 2, 128, generator=gen, device=DEV).to(dtype)
    at_q, cu_q = _cu(nq)
    at_k, cu_k = _cu(nk)
    for causal in (True, False):
        sq, sk = _call(q, k, cu_q, cu_k, None, causal)
        want, err = _reference(q, k, at_q, at_k, 128 ** -0.5, causal)
        # the scale itself is rounded to fp32 too
        assert bool(((sq.double() - want).abs() <= err + 2.0 ** -23 * want.abs()).all())
        assert torch.equal(sk, sq.view(2, 4).amax(1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), -3.3e38])
def test_masked_values_never_count(value, dtype):
    nq = [70, 200, 30]
    q, k = _ints(11, 300, 4, 128, dtype), _ints(12, 300, 4, 128, dtype)
    at, cu = _cu(nq)
    want = _call(q, k, cu, cu, 1.0, True)[0]
    # keys that no query of their sequence sees: none here but with fewer queries
    k2 = torch.cat([k, torch.full((64, 4, 128), value, dtype=dtype, device=DEV)])
    q2 = torch.cat([q, torch.full((64, 4, 128), value, dtype=dtype, device=DEV)])
    assert torch.equal(_call(q2, k2, cu, cu, 1.0, True)[0], want)       # rows behind the last sequence
    # the last query sees every key; the first of two sees all but the last
    q3, k3 = _ints(13, 2, 1, 64, dtype), _ints(14, 50, 1, 64, dtype)
    q3[1] = 0
    k3[49] = value
    _, cu_q = _cu([2])
    _, cu_k = _cu([50])
    got = float(_call(q3, k3, cu_q, cu_k, 1.0, True)[0])
    logits = (q3[0, 0].double() @ k3[:49, 0].double().t().contiguous()).max()
    if value == -3.3e38:
        assert got == max(float(logits), 0.0)
    else:
        assert got != got       # 0 * inf: an unmasked logit of the last query is NaN


def test_a_nan_logit_makes_its_head_nan():
    q, k = _ints(15, 200, 4, 128, BF16), _ints(16, 200, 2, 128, BF16)
    q[150, 2, 7] = float("nan")
    _, cu = _cu([200])
    sq, sk = _call(q, k, cu, cu, 1.0, True)
    assert torch.isnan(sq).tolist() == [False, False, True, False]
    assert torch.isnan(sk).tolist() == [False, True]


def test_heads_without_any_pair():
    q, k = _ints(17, 40, 4, 64, BF16), _ints(18, 40, 2, 64, BF16)
    _, none = _cu([0, 0])
    _, cu = _cu([40, 0])
    for a, b in ((none, none), (cu, none), (none, cu)):
        sq, sk = _call(q, k, a, b, 1.0, True)
        assert bool((sq == NEG).all()) and bool((sk == NEG).all())
    sq, sk = _call(q[:0], k, none, cu, 1.0, False)
    assert bool((sq == NEG).all()) and bool((sk == NEG).all())
    sq, sk = _call(q, k[:0], cu, none, 1.0, False)
    assert bool((sq == NEG).all())


def test_accumulate_over_micro_batches():
    h = Handle.get()
    _, cu = _cu([60, 40])
    parts = [(_ints(s, 100, 4, 64, BF16), _ints(s + 50, 100, 2, 64, BF16)) for s in range(3)]
    each = [_call(q, k, cu, cu, 1.0, True) for q, k in parts]
    sq, sk = torch.full((4,), NEG, device=DEV), torch.full((2,), NEG, device=DEV)
    ws = torch.empty(mu.muon_qk_smax_workspace_size(h, *parts[0], cu), dtype=torch.uint8, device=DEV)
    for q, k in parts:
        mu.muon_qk_smax(h, q, k, cu, cu, sq, ws, smax_k=sk, scale=1.0, accumulate=True)
    assert torch.equal(sq, torch.stack([a for a, _ in each]).amax(0))
    assert torch.equal(sk, torch.stack([b for _, b in each]).amax(0))
    only = torch.zeros(2, device=DEV)
    mu.muon_qk_smax(h, *parts[2], cu, cu, None, ws, smax_k=only, scale=1.0)
    assert torch.equal(only, each[2][1])


@pytest.mark.parametrize("bad", [[0, -5, 40], [0, 60, 20], [5, 100000, 2000000000], [-7, 10, 2147483647]])
def test_bounds_that_make_no_sense_reach_no_memory(bad):
    q, k = _ints(19, 50, 4, 64, BF16), _ints(20, 60, 2, 64, BF16)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    _call(q, k, cu, cu, 1.0, True)
    _call(q, k, cu, cu.flip(0).contiguous(), 1.0, False)
    torch.cuda.synchronize()


def test_another_stream_and_a_captured_graph():
    h = Handle.get()
    q, k = _ints(21, 400, 8, 128, BF16), _ints(22, 400, 4, 128, BF16)
    _, cu = _cu([100, 300, 0])
    sq = torch.zeros(8, device=DEV)
    ws = torch.empty(mu.muon_qk_smax_workspace_size(h, q, k, cu), dtype=torch.uint8, device=DEV)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        mu.muon_qk_smax(h, q, k, cu, cu, sq, ws, scale=1.0)
    for sizes in ([100, 300, 0], [1, 2, 3], [399, 0, 1], [200, 100, 100]):
        at, new = _cu(sizes)
        cu.copy_(new)
        q.mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(sq, _reference(q, k, at, at, 1.0, True)[0].float())
        with torch.cuda.stream(s):
            eager = _call(q, k, cu, cu, 1.0, True)[0]
        torch.cuda.synchronize()
        assert torch.equal(eager, sq)


def test_offsets_beyond_32_bits():
    # the last sequence of a k that holds more than 2^31 elements
    T, Hk, D = (1 << 20) + 50, 16, 128
    k = torch.zeros(T, Hk, D, dtype=BF16, device=DEV)
    k[-50:] = _ints(23, 50, Hk, D, BF16)
    q = _ints(24, 50, Hk, D, BF16)
    cu_q = torch.tensor([0, 0, 50], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, T - 50, T], dtype=torch.int32, device=DEV)
    sq, _ = _call(q, k, cu_q, cu_k, 1.0, True)
    want, _ = _reference(q, k[-50:], [0, 50], [0, 50], 1.0, True)
    assert torch.equal(sq, want.float())


def test_binding_refuses():
    h = Handle.get()
    q, k = _ints(25, 30, 4, 64, BF16), _ints(26, 30, 2, 64, BF16)
    _, cu = _cu([30])
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    out = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        mu.muon_qk_smax(h, q, k.float(), cu, cu, out, ws)
    with pytest.raises(ValueError):
        mu.muon_qk_smax(h, q, k[..., :32], cu, cu, out, ws)
    with pytest.raises(ValueError):
        mu.muon_qk_smax(h, q, k, cu, torch.cat([cu, cu]), out, ws)
    with pytest.raises(ValueError):
        mu.muon_qk_smax(h, q, k, cu.long(), cu.long(), out, ws)
    with pytest.raises(ValueError):
        mu.muon_qk_smax(h, q, k, cu, cu, out[:3], ws)
    with pytest.raises(ValueError):
        mu.muon_qk_smax(h, q, k, cu, cu, out, ws.cpu())
    with pytest.raises(mu.MuonError) as e:
        mu.muon_qk_smax(h, q[:, :3], k, cu, cu, out[:3], ws)
    assert e.value.status == 1


# Sequences of 512 queries and more on average take tiles of 256 queries, every
# head size its own kernel: ragged ends, more and fewer keys than queries, heads
# that divide by 8 (dealt to the XCDs) and heads that do not.
@pytest.mark.parametrize("heads,kv", [(4, 2), (8, 8)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [8, 64, 80, 96, 128, 160, 192, 200, 256])
def test_long_sequences_of_every_head_size(dim, causal, heads, kv):
    nq, nk = [700, 1, 1301, 613], [700, 40, 1400, 333]
    _check_whole(_ints(27, sum(nq), heads, dim, BF16), _ints(28, sum(nk), kv, dim, BF16), nq, nk, causal)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_sequences_read_no_masked_value(dim):
    """NaN in every key behind the last one a query sees, and behind the
    sequences: none may reach a maximum."""
    n, more = 600, 64
    q, k = _ints(29, n, 2, dim, BF16), _ints(30, n + more, 2, dim, BF16)
    at, cu = _cu([n])
    want = _call(q, k[:n], cu, cu, 1.0, True)[0]
    k[n:] = float("nan")
    assert torch.equal(_call(q, k, cu, cu, 1.0, True)[0], want)
    assert torch.equal(want, _reference(q, k[:n], at, at, 1.0, True)[0].float())
    # the last query alone sees the last key
    k[n - 1] = float("nan")
    assert bool(torch.isnan(_call(q, k, cu, cu, 1.0, True)[0]).all())
    q[n - 1:] = float("nan")
    cu_q = torch.tensor([0, n - 1], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, n - 1], dtype=torch.int32, device=DEV)
    got = _call(q, k, cu_q, cu_k, 1.0, True)[0]
    assert torch.equal(got, _reference(q, k, [0, n - 1], [0, n - 1], 1.0, True)[0].float())


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 63), (F32, 64)])
@pytest.mark.parametrize("nq,nk", [([1], [9000]), ([70, 1, 0, 3], [4000, 1, 5, 70]), ([129] * 5, [129] * 5),
                                   ([1500], [1500]), ([1] * 40, [2] * 40)])
def test_the_workspace_is_as_large_as_its_size_says(nq, nk, dtype, dim):
    """Nothing behind it is written: few queries, whose keys are split over
    workgroups, and many short sequences, each with a ragged tile."""
    h = Handle.get()
    q, k = _ints(31, sum(nq), 6, dim, dtype), _ints(32, sum(nk), 2, dim, dtype)
    at_q, cu_q = _cu(nq)
    at_k, cu_k = _cu(nk)
    need = mu.muon_qk_smax_workspace_size(h, q, k, cu_q)
    buf = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    sq = torch.zeros(6, device=DEV)
    mu.muon_qk_smax(h, q, k, cu_q, cu_k, sq, buf[:need], scale=1.0)
    assert torch.equal(sq, _reference(q, k, at_q, at_k, 1.0, True)[0].float())
    assert bool((buf[need:] == 0xA5).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sequences", [64, 65, 200])
def test_many_sequences(sequences, dtype):
    """More than a wave's lanes, some empty, a few of them long."""
    r = torch.Generator().manual_seed(sequences)
    nq = (torch.rand(sequences, generator=r) * 20 - 2).clamp(min=0).int().tolist()
    nq[3], nq[-2] = 300, 170
    nk = [n + i % 3 for i, n in enumerate(nq)]
    _check_whole(_ints(33, sum(nq), 4, 64, dtype), _ints(34, sum(nk), 2, 64, dtype), nq, nk, True)
