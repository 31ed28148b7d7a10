"""GPU parity of the embedding lookup and its gradient: token counts around the pieces of 8 to 32 and the sorting
workgroups, tables that take one to three sorting passes, frequent rows, padding, views, streams, graphs."""
import pytest
import torch

import dense_linear_algebra_alpha_amd as xt
import layer_oracle as L
from gpu_util import dev, note

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def words(count, rows, seed):
    """Indices of which the small ones are frequent, some negative, some beyond the table."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(count, generator=g, dtype=torch.float64) ** 4 * rows).long().clamp_max(rows - 1)
    odd = torch.rand(count, generator=g)
    return torch.where(odd < 0.05, -1, torch.where(odd > 0.98, rows + 3, ids)) if count > 2 else ids


def backward(G, ids, rows, scale, before=None):
    """(dtable, bound): sums of c tokens through at most c + 8 additions in fp32, rounded once."""
    there = (ids >= 0) & (ids < rows)
    k = G.shape[1]
    at = ids.long().clamp(0, max(rows - 1, 0))
    add = lambda v: torch.zeros(rows, k, dtype=torch.float64).index_add_(0, at[there], v[there])  # noqa: E731
    total, mag = add(G.double()) * scale, add(G.double().abs()) * abs(scale)
    count = torch.zeros(rows, dtype=torch.float64).index_add_(0, at[there], torch.ones(int(there.sum()), dtype=torch.float64))
    if before is not None:
        total, mag = total + before.double(), mag + before.double().abs()
    h, s = L.half_step(G.dtype), L.smallest(G.dtype)
    return total, (count[:, None] + 8) * 2.0 ** -24 * mag * (1 + h) + h * total.abs() + s


SIZES = [(1, 1, 1), (5, 3, 7), (31, 64, 10), (32, 8, 1), (33, 8, 1), (64, 128, 2), (65, 17, 3), (1000, 100, 37), (100, 1111, 5000),
         (4096, 260, 50001), (300, 2500, 511), (300, 24, 512), (16384, 64, 3), (16385, 64, 1000), (1024, 64, 1000), (1025, 64, 1000), (4096, 8, 100), (4097, 16, 70_000), (65537, 16, 3000), (40000, 72, 70001), (70000, 8, 300_000),
         (20000, 40, 300_000), (50000, 4, 1)]


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%dx%d" % s)
def test_forward_and_backward(size, dtype):
    count, k, rows = size
    dt = L.DTYPES[dtype]
    index = torch.int32 if (count + k) % 2 else torch.int64
    scale = 1.0 if k % 3 else 2.5
    ids, table, G = words(count, rows, count + k).to(index), rand((rows, k), 1, dt), rand((count, k), 2, dt)
    gi, gt, gG = ids.to(dev()), table.to(dev()), G.to(dev())
    note("embedding %s %s" % (size, dtype))
    out = xt.embedding(gi, gt, scale)
    torch.cuda.synchronize()
    want = (table.float()[ids.long().clamp(0, rows - 1)] * scale).to(dt)
    want[ids < 0] = 0.0
    want[ids >= rows] = float("nan")
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out.cpu().nan_to_num(1.0), want.nan_to_num(1.0))
    ref, bound = backward(G, ids, rows, scale)
    note("embedding_backward %s %s" % (size, dtype))
    got = xt.embedding_backward(gG, gi, rows, scale)
    again = xt.embedding_backward(gG, gi, rows, scale, dtable=torch.full_like(got, 9.0))
    torch.cuda.synchronize()
    L.check(got, ref, bound, "%s %s" % (size, dtype))
    assert torch.equal(got, again)
    before = rand((rows, k), 3, dt)
    ref, bound = backward(G, ids, rows, scale, before)
    gb = before.to(dev())
    got = xt.embedding_backward(gG, gi, rows, scale, dtable=gb, accumulate=True)
    torch.cuda.synchronize()
    assert got is gb
    L.check(got, ref, bound, "%s %s accumulated" % (size, dtype))
    unused = torch.ones(rows, dtype=torch.bool)
    unused[ids[(ids >= 0) & (ids < rows)].long()] = False
    assert torch.equal(got.cpu()[unused], before[unused])


def test_order_of_the_tokens():
    """The sum of a row's tokens is taken in their order: of three values that round differently, both orders."""
    big, one = 2.0 ** 24, 1.0
    for order, want in (((big, one, one), big), ((one, one, big), big + 2)):
        G = torch.tensor(order, device=dev())[:, None].expand(3, 8).contiguous()
        got = xt.embedding_backward(G, torch.full((3,), 4, device=dev()), 6)
        torch.cuda.synchronize()
        assert (got[4] == want).all() and got.count_nonzero() == 8


@pytest.mark.parametrize("count", [1, 40, 20000])
def test_padding_alone(count):
    """Nothing points anywhere: zeros, and NaN in the gradients of padding stays out."""
    d = dev()
    G = torch.full((count, 96), float("nan"), device=d)
    ids = torch.full((count,), -1, device=d)
    note("embedding padding %d" % count)
    got = xt.embedding_backward(G, ids, 100)
    before = torch.ones(100, 96, device=d)
    xt.embedding_backward(G, ids, 100, dtable=before, accumulate=True)
    torch.cuda.synchronize()
    assert not got.any() and (before == 1).all()
    ids[0] = 3
    got = xt.embedding_backward(G, ids, 100)
    torch.cuda.synchronize()
    assert torch.isnan(got[3]).all() and got.isnan().sum() == 96


def test_zero_sizes():
    d = dev()
    no = torch.empty(0, dtype=torch.int64, device=d)
    assert xt.embedding(no, torch.ones(3, 4, device=d)).shape == (0, 4)
    assert xt.embedding(torch.zeros(2, dtype=torch.int64, device=d), torch.ones(3, 0, device=d)).shape == (2, 0)
    out = xt.embedding(torch.tensor([-1, 0], device=d), torch.ones(0, 4, device=d))
    got = xt.embedding_backward(torch.empty(0, 5, device=d), no, 6)
    none = xt.embedding_backward(torch.ones(2, 5, device=d), torch.zeros(2, dtype=torch.int64, device=d), 0)
    torch.cuda.synchronize()
    assert not out[0].any() and out[1].isnan().all()
    assert got.shape == (6, 5) and not got.any() and none.shape == (0, 5)


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("k", [3, 100, 1111])
def test_views_of_wider_buffers(k, dtype):
    dt, count, rows = L.DTYPES[dtype], 200, 50
    ids, table, G, before = words(count, rows, 5), rand((rows, k), 6, dt), rand((count, k), 7, dt), rand((rows, k), 8, dt)

    def view(t, n):
        buf = torch.full((n, k + 12), 7.0, dtype=dt, device=dev())
        v = buf[:, 3:3 + k]
        if t is not None:
            v.copy_(t)
        return buf, v

    (_, vt), (ob, vo), (_, vG), (tb, vd), (ab, va) = view(table, rows), view(None, count), view(G, count), view(None, rows), view(before, rows)
    gi = ids.to(dev())
    note("embedding views %d %s" % (k, dtype))
    out = xt.embedding(gi, vt, out=vo)
    plain = xt.embedding(gi, table.to(dev()))
    xt.embedding_backward(vG, gi, rows, dtable=vd)
    xt.embedding_backward(vG, gi, rows, 0.5, dtable=va, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(1.0), plain.nan_to_num(1.0))
    L.check(vd, *backward(G, ids, rows, 1.0), what="dtable")
    L.check(va, *backward(G, ids, rows, 0.5, before), what="accumulated")
    for buf in (ob, tb, ab):
        assert (buf[:, :3] == 7.0).all() and (buf[:, 3 + k:] == 7.0).all()


def test_table_beyond_two_to_the_31_elements():
    rows, k = 530_000, 4100
    table = torch.zeros(rows, k, dtype=torch.float16, device=dev())
    table[-1] = 2.0
    ids = torch.tensor([rows - 1, 0, rows - 1], device=dev())
    note("embedding of 2^31 elements")
    out = xt.embedding(ids, table)
    G = rand((3, k), 9, torch.float16).to(dev())
    xt.embedding_backward(G, ids, rows, dtable=table)
    torch.cuda.synchronize()
    assert (out[::2] == 2.0).all() and not out[1].any()
    assert torch.equal(table[-1], (G[0].float() + G[2].float()).half()) and torch.equal(table[0], G[1])
    assert not table[1:-1:1000].any()


@pytest.mark.parametrize("count", [700, 20000])
def test_streams_and_graph(count):
    rows, k = 1000, 200
    ids, table, G = words(count, rows, 11).to(dev()), rand((rows, k), 12).to(dev()), rand((count, k), 13).to(dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    note("embedding on a stream %d" % count)
    out = xt.embedding(ids, table, 3.0, stream=side)
    got = xt.embedding_backward(G, ids, rows, 3.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.nan_to_num(1.0), xt.embedding(ids, table, 3.0).nan_to_num(1.0))
    assert torch.equal(got, xt.embedding_backward(G, ids, rows, 3.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = xt.embedding(ids, table)
        g = xt.embedding_backward(G, ids, rows)
    for seed in range(3):
        ids.copy_(words(count, rows, 20 + seed))
        note("embedding replay %d" % seed)
        graph.replay()
        torch.cuda.synchronize()
        eo, eg = xt.embedding(ids, table), xt.embedding_backward(G, ids, rows)
        torch.cuda.synchronize()
        assert torch.equal(o.nan_to_num(1.0), eo.nan_to_num(1.0)) and torch.equal(g, eg)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("size", [(40000, 1111, 37), (40001, 1111, 5000), (98400, 260, 300), (12000, 5003, 2)], ids=lambda s: "%dx%dx%d" % s)
def test_pieces_of_32_tokens(size, dtype, accumulate):
    """Rows of many slabs whose tokens go through many pieces of 32 (16 where the slabs are fewer). Whole numbers, whose sums in
    fp32 are exact: no token is lost or added twice. The oracle runs on the GPU."""
    count, k, rows = size
    dt = L.DTYPES[dtype]
    ids = words(count, rows, count).to(dev())
    g = torch.Generator(dev()).manual_seed(k)
    G = torch.randint(-4, 5, (count, k), generator=g, device=dev()).to(dt)
    before = torch.randint(-4, 5, (rows, k), generator=g, device=dev()).to(dt)
    note("embedding pieces of 32 %s %s" % (size, dtype))
    got = xt.embedding_backward(G, ids, rows, 0.5, dtable=before.clone(), accumulate=accumulate)
    torch.cuda.synchronize()
    there = (ids >= 0) & (ids < rows)
    want = torch.zeros(rows, k, dtype=torch.float64, device=dev()).index_add_(0, ids[there], G[there].double()) * 0.5
    if accumulate:
        want += before.double()
    assert want.abs().max() < 2.0 ** 15  # within fp16, and whole sums within fp32
    assert torch.equal(got, want.float().to(dt))


@pytest.mark.parametrize("dtype", list(L.DTYPES))
@pytest.mark.parametrize("lanes, chunks", [(16, 31.5), (64, 98.5), (256, 139)])
def test_lookups_beyond_the_caches(lanes, chunks, dtype):
    """Outputs of more than 32 MiB, which are stored past the L2s, by 16, 64 and 256 threads a row; widths that are no whole
    number of 16 bytes."""
    dt = L.DTYPES[dtype]
    es = torch.finfo(dt).bits // 8
    k = int(chunks * 16 / es) + 1
    count, rows = (36 << 20) // (k * es), 3001
    ids = words(count, rows, k).to(dev())
    table = rand((rows, k), 1, dt).to(dev())
    note("embedding beyond the caches %d %s" % (k, dtype))
    out = xt.embedding(ids, table, 2.5)
    torch.cuda.synchronize()
    assert out.numel() * es > 32 << 20
    want = (table.float()[ids.clamp(0, rows - 1)] * 2.5).to(dt)
    want[ids < 0] = 0.0
    want[ids >= rows] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(1.0), want.nan_to_num(1.0))
