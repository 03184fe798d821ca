"""Attention over the 8-bit cache on the GPU against softmax in 64 bits over the values that the cache stands for.

Tolerances. With A = sum_j p_j |v_j|: a probability enters the second product with eight bits, off by at most 2^-8 of
itself (and by 2^-19 of the row's reference, which its scores pass by at most 2^4 and their sum l, relative to the
largest, is no less than: N 2^-19 of the largest |v| over l); scores are float32 sums of Dk products of exact factors,
off by at most ds = (Dk + 8) 2^-23 of sum |q k| scale, which moves a probability by 2 ds of itself; float32 sums add
2^-12 of A; the result is rounded to bf16, 2^-8 of it."""
import math

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from test_gpu_cache import Case, decode

pytestmark = pytest.mark.gpu
bf16, f32, f64, i32, u8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


def reference(s, q, scale, host=None):
    """(out, lse, tolerance of out, tolerance of lse) for q [T, Hq, Dk] over the case's cache, in 64 bits."""
    k_all, v_all = decode(s.host[0], s.host[1], s.block), None
    v_all = k_all[..., :s.cache.Dv] if s.host[2] is None else decode(s.host[2], s.host[3], s.block)
    T, Hq, Dk = q.shape
    H = k_all.shape[1]
    g = Hq // H
    out, lse = torch.zeros((T, Hq, s.cache.Dv), dtype=f64), torch.full((T, Hq), -math.inf, dtype=f64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (start, n) in enumerate(zip(s.start, s.n)):
        length = start + n
        t = torch.arange(length)
        if n == 0 or length == 0:
            continue
        p = s.table[b, t // s.page].long()
        k, v = k_all[p, :, t % s.page], v_all[p, :, t % s.page]  # [L, H, D]
        for i in range(n):
            r = s.cu_list[b] + i
            seen = length - n + i + 1
            if seen <= 0:
                continue
            qq = q[r].to(f64).view(H, g, Dk)
            kk, vv = k[:seen], v[:seen]
            z = torch.einsum("hgd,thd->hgt", qq, kk) * scale
            size = torch.einsum("hgd,thd->hgt", qq.abs(), kk.abs()).amax(2) * abs(scale)
            ds = (Dk + 8) * 2.0 ** -23 * size
            w = torch.softmax(z, 2)
            o, a = torch.einsum("hgt,thd->hgd", w, vv), torch.einsum("hgt,thd->hgd", w, vv.abs())
            top = vv.abs().nan_to_num(0).amax((0, 2))[:, None, None]
            l = 1 / w.amax(2)
            out[r], lse[r] = o.reshape(Hq, -1), torch.logsumexp(z, 2).reshape(Hq)
            tol[r] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * ds[..., None]) * a + seen * 2.0 ** -19 * top / l[..., None]).reshape(Hq, -1)
            ltol[r] = (ds + 2.0 ** -20 + 2.0 ** -22 * lse[r].view(H, g).abs()).reshape(Hq)
    return out, lse, tol, ltol


def check(got, want, tol, what):
    got = got.cpu().to(f64)
    d = (got - want).abs()
    bad = ~(d <= tol) & ~(got == want) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def attend(dev, s, Hq, scale=None, seed=1, std=1.0, **kw):
    g = torch.Generator().manual_seed(seed)
    Dk = s.host[0].shape[3]
    q = (torch.randn((sum(s.n), Hq, Dk), generator=g) * std).to(bf16)
    # codes are random bytes: values up to 448 * 2^-4; a scale that brings scores to a few units
    scale = 0.3 / math.sqrt(Dk) / 8 if scale is None else scale
    st = torch.zeros(1, dtype=i32, device=dev)
    out, lse = mlaq.cache_attn(q.to(dev), s.cache, s.table_d, s.length_d, cu=kw.pop("cu", s.cu), scale=scale, lse=True, status=st, **kw)
    assert st.item() == 0
    return q, scale, out, lse


SMALL = [
    dict(Hq=1, c=dict(H=1, Dk=16, Dv=16, page=16, block=16, start=[0], n=[1])),
    dict(Hq=4, c=dict(H=1, Dk=128, Dv=128, page=16, block=16, start=[99], n=[1])),
    dict(Hq=8, c=dict(H=2, Dk=128, Dv=128, page=64, block=32, start=[127, 128, 129, 0, 1000], n=[1] * 5)),
    dict(Hq=3, c=dict(H=3, Dk=192, Dv=128, page=32, block=1, start=[511, 5], n=[1, 1])),
    dict(Hq=24, c=dict(H=2, Dk=80, Dv=112, page=128, block=64, start=[300, 7], n=[1, 1])),
    dict(Hq=32, c=dict(H=1, Dk=64, Dv=64, page=256, block=256, start=[700], n=[1])),
    dict(Hq=100, c=dict(H=2, Dk=256, Dv=256, page=16, block=8, start=[260, 31], n=[1, 1])),
    dict(Hq=128, c=dict(H=1, Dk=576, Dv=512, page=64, block=64, start=[400, 64], n=[1, 1], shared=True)),
    dict(Hq=8, c=dict(H=1, Dk=320, Dv=256, page=32, block=16, start=[200], n=[1], shared=True)),
    dict(Hq=5, c=dict(H=1, Dk=48, Dv=16, page=16, block=2, start=[33], n=[1], shared=True)),
]


@pytest.mark.parametrize("c", SMALL)
def test_tokens(cuda_device, c):
    s = Case(cuda_device, **c["c"])
    q, scale, out, lse = attend(cuda_device, s, c["Hq"])
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")
    # without cu: the same
    q2, _, out2, lse2 = attend(cuda_device, s, c["Hq"], cu=None)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


CHUNKS = [
    dict(Hq=4, c=dict(H=2, Dk=64, Dv=64, page=16, block=16, start=[0, 5, 130], n=[3, 1, 4])),
    dict(Hq=8, c=dict(H=2, Dk=128, Dv=128, page=64, block=32, start=[0, 250, 64], n=[200, 0, 129])),
    dict(Hq=2, c=dict(H=2, Dk=192, Dv=128, page=128, block=32, start=[100], n=[300])),
    dict(Hq=7, c=dict(H=1, Dk=96, Dv=96, page=32, block=8, start=[0, 90], n=[65, 66])),
    dict(Hq=64, c=dict(H=1, Dk=576, Dv=512, page=64, block=64, start=[100, 0], n=[3, 5], shared=True)),
    dict(Hq=2, c=dict(H=1, Dk=256, Dv=256, page=64, block=64, start=[10], n=[150])),
    dict(Hq=16, c=dict(H=1, Dk=128, Dv=128, page=16, block=4, start=[0] * 5, n=[1, 0, 0, 40, 0])),
]


@pytest.mark.parametrize("c", CHUNKS)
def test_several_tokens(cuda_device, c):
    s = Case(cuda_device, **c["c"])
    q, scale, out, lse = attend(cuda_device, s, c["Hq"])
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")


PAIRS = [  # latents with more query rows than a block takes: two blocks share their tiles
    dict(Hq=40, c=dict(H=1, Dk=576, Dv=512, page=16, block=16, start=[300, 0, 127], n=[1, 1, 1], shared=True)),
    dict(Hq=128, c=dict(H=1, Dk=320, Dv=256, page=128, block=32, start=[1000, 40], n=[1, 1], shared=True)),
    dict(Hq=200, c=dict(H=2, Dk=144, Dv=96, page=256, block=128, start=[600, 0, 0], n=[1, 0, 1], shared=True)),
    dict(Hq=33, c=dict(H=1, Dk=640, Dv=512, page=32, block=1, start=[5, 250], n=[9, 4], shared=True)),
    dict(Hq=3, c=dict(H=1, Dk=512, Dv=512, page=1024, block=64, start=[100, 0, 700], n=[60, 0, 33], shared=True)),
    dict(Hq=128, c=dict(H=1, Dk=576, Dv=512, page=64, block=64, start=[12000], n=[1], shared=True)),
]


@pytest.mark.parametrize("c", PAIRS)
def test_latents_of_many_rows(cuda_device, c):
    s = Case(cuda_device, **c["c"])
    q, scale, out, lse = attend(cuda_device, s, c["Hq"])
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")
    _, _, again, _ = attend(cuda_device, s, c["Hq"])
    assert torch.equal(out, again)


def test_nan_in_latents_of_many_rows(cuda_device):
    """A NaN in one channel of a cached row: the rows that see it, each in both blocks of a pair, and no others; a bad page."""
    s = Case(cuda_device, H=1, Dk=320, Dv=256, page=16, block=16, start=[150], n=[20], shared=True)
    at = 155
    p = int(s.table[0, at // 16])
    s.host[0][p, 0, at % 16, 300] = 0x7F  # behind the values: a score of NaN
    s.cache.k.copy_(s.host[0])
    q, scale, out, lse = attend(cuda_device, s, 8)
    ref = reference(s, q, scale)
    assert out[5:].isnan().all() and lse[5:].isnan().all()
    check(out[:5], ref[0][:5], ref[2][:5], "out")
    st = torch.zeros(1, dtype=i32, device=cuda_device)
    table = s.table_d.clone()
    table[0, 2] = 2 ** 30
    o = mlaq.cache_attn(q[:, :, :].to(cuda_device), s.cache, table, s.length_d, cu=s.cu, scale=scale, status=st)
    assert st.item() == mlaq.STATUS["MLA_ERR_POS_RANGE"] and o[:5].isfinite().all()


def test_one_long_sequence_over_every_sm(cuda_device):
    """More tiles than shares: parts that begin and end inside a pair, added in the second kernel."""
    s = Case(cuda_device, H=1, Dk=64, Dv=80, page=128, block=128, start=[40_000], n=[1])
    q, scale, out, lse = attend(cuda_device, s, 2)
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")


def test_many_sequences(cuda_device):
    """More than the lengths that shared memory holds, ragged, some of them empty."""
    g = torch.Generator().manual_seed(3)
    n = [int(v) for v in torch.randint(0, 3, (700,), generator=g)]
    start = [int(v) for v in torch.randint(0, 60, (700,), generator=g)]
    s = Case(cuda_device, H=2, Dk=32, Dv=32, page=16, block=16, start=start, n=n)
    q, scale, out, lse = attend(cuda_device, s, 4)
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")


def test_empty_rows(cuda_device):
    """A sequence without positions, and new tokens that the given length does not reach: zeros and -inf."""
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=16, block=16, start=[20, 0, 0], n=[1, 1, 4])
    s.length_d.copy_(torch.tensor([21, 0, 2], dtype=i32))
    q, scale, out, lse = attend(cuda_device, s, 4)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    assert (out[2:4] == 0).all() and (lse[2:4] == -math.inf).all() and lse[4:].isfinite().all()
    s.start[1], s.n[1] = -1, 1
    s.start[2] = -2
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")


def test_scores_that_grow_and_scales_that_differ(cuda_device):
    """Every tile raises the maximum and the largest scale of V, by far more than the reference may lag."""
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=128, block=128, start=[1200], n=[1])
    for i, p in enumerate(s.table[0, :10].tolist()):
        s.host[1][p], s.host[3][p] = 100 + 2 * i, 90 + 5 * i
    for a, b in ((s.cache.k_scales, s.host[1]), (s.cache.v_scales, s.host[3])):
        a.copy_(b)
    for scale in (0.02, 2.0, -1.0):
        q, _, out, lse = attend(cuda_device, s, 3, scale=scale)
        ref = reference(s, q, scale)
        check(lse, ref[1], ref[3], "lse")
        check(out, ref[0], ref[2], "out")


def test_a_sink_of_small_values(cuda_device):
    """Nearly all weight on a first token whose values are 2^-10 of the others'."""
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=64, block=1, start=[400], n=[1])
    p = int(s.table[0, 0])
    s.host[0][p, :, 0], s.host[1][p, :, 0] = 0x50, 127
    s.host[3][p, :, 0] = 108
    s.cache.k.copy_(s.host[0]), s.cache.k_scales.copy_(s.host[1]), s.cache.v_scales.copy_(s.host[3])
    q = torch.full((1, 2, 64), 0.5, dtype=bf16)
    out, lse = mlaq.cache_attn(q.to(cuda_device), s.cache, s.table_d, s.length_d, scale=0.01, lse=True)
    ref = reference(s, q, 0.01)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")


def test_nan_where_it_is_seen(cuda_device):
    """NaN behind the last position does not count; a NaN key or value reaches the rows that see it, in its channel; NaN and
    Inf in a query its own row."""
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=16, block=16, start=[150], n=[20])
    last = int(s.table[0, 10])
    s.host[0][last, :, 10:], s.host[2][last, :, 10:] = 0x7F, 0xFF
    at = 155
    p = int(s.table[0, at // 16])
    s.host[2][p, 0, at % 16, 5] = 0x7F
    s.cache.k.copy_(s.host[0]), s.cache.v.copy_(s.host[2])
    q, scale, out, lse = attend(cuda_device, s, 2)
    ref = reference(s, q, scale)
    assert ref[0][5:, :, 5].isnan().all() and not ref[0][:5].isnan().any() and int(ref[0].isnan().sum()) == 15 * 2
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")
    s.host[0][p, 0, at % 16, 7] = 0xFF
    s.cache.k.copy_(s.host[0])
    q, scale, out, lse = attend(cuda_device, s, 2)
    assert out[5:].isnan().all() and lse[5:].isnan().all()
    ref = reference(s, q, scale)
    check(out[:5], ref[0][:5], ref[2][:5], "out")
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=16, block=16, start=[150], n=[3])
    q = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(2)).to(bf16)
    q[1, 0, 3], q[2, 1, 60] = math.nan, math.inf
    out, lse = mlaq.cache_attn(q.to(cuda_device), s.cache, s.table_d, s.length_d, cu=s.cu, scale=0.005, lse=True)
    bad = torch.zeros((3, 2), dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(out.isnan().all(2).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    ref = reference(s, torch.where(bad[..., None], torch.zeros_like(q), q), 0.005)
    check(torch.where(bad[..., None], torch.zeros_like(out.cpu()), out.cpu()), torch.where(bad[..., None], torch.zeros_like(ref[0]), ref[0]), ref[2], "out")


def test_queries_of_any_size(cuda_device):
    """Zero rows, rows whose elements span the type, and far smaller rows beside large ones."""
    s = Case(cuda_device, H=1, Dk=128, Dv=64, page=16, block=16, start=[140], n=[1])
    g = torch.Generator().manual_seed(5)
    q = torch.randn((1, 6, 128), generator=g)
    q[0, 0] = 0
    q[0, 1] *= torch.exp2(-torch.arange(128) / 8.0)
    q[0, 2] *= 2.0 ** -60
    q[0, 3] *= 2.0 ** -130
    q[0, 4, 1:] = 0
    q = q.to(bf16)
    for scale in (0.004, 2.0 ** 50):
        if scale > 1:
            q[0, [1, 4, 5]] = 0
        out, lse = mlaq.cache_attn(q.to(cuda_device), s.cache, s.table_d, s.length_d, scale=scale, lse=True)
        ref = reference(s, q, scale)
        check(lse, ref[1], ref[3], "lse")
        check(out, ref[0], ref[2], "out")


def test_strides_and_rows_behind(cuda_device):
    s = Case(cuda_device, H=2, Dk=64, Dv=48, page=16, block=16, start=[30, 0], n=[5, 9])
    q, scale, out, lse = attend(cuda_device, s, 6)
    T = sum(s.n)
    for view in (q.transpose(0, 1).contiguous().transpose(0, 1), torch.cat([q, q], 2)[..., :64],
                 torch.zeros(q.numel() + 1, dtype=bf16)[1:].view_as(q).copy_(q)):
        d = torch.empty_strided(view.shape, view.stride(), dtype=bf16, device=cuda_device)
        d.copy_(view)
        if view.storage_offset() % 8:
            d = torch.zeros(q.numel() + 1, dtype=bf16, device=cuda_device)[1:].view_as(q).copy_(q)
        assert torch.equal(mlaq.cache_attn(d, s.cache, s.table_d, s.length_d, cu=s.cu, scale=scale), out)
    wide = torch.full((T + 4, 6, 64), math.nan, dtype=bf16, device=cuda_device)
    wide[:T] = q.to(cuda_device)
    o = torch.full((T + 4, 6, 48), 3.0, dtype=bf16, device=cuda_device)
    ls = torch.full((T + 4, 6), 3.0, device=cuda_device)
    mlaq.cache_attn(wide, s.cache, s.table_d, s.length_d, cu=s.cu, scale=scale, out=o, lse=ls)
    assert torch.equal(o[:T], out) and torch.equal(ls[:T], lse) and (o[T:] == 3).all() and (ls[T:] == 3).all()


def test_bad_pages_and_bounds(cuda_device):
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=16, block=16, start=[100, 40], n=[2, 2])
    q, scale, out, lse = attend(cuda_device, s, 2)
    R, I = mlaq.STATUS["MLA_ERR_POS_RANGE"], mlaq.STATUS["MLA_ERR_INVALID_ARG"]
    d = q.to(cuda_device)

    def run(table=None, length=None, cu=None):
        st = torch.zeros(1, dtype=i32, device=cuda_device)
        o = mlaq.cache_attn(d, s.cache, s.table_d if table is None else table,
                            s.length_d if length is None else torch.tensor(length, dtype=i32, device=cuda_device),
                            cu=s.cu if cu is None else torch.tensor(cu, dtype=i32, device=cuda_device), scale=scale, status=st)
        return o, st.item()

    for bad in (-1, 1000, 2 ** 31 - 1, -2 ** 31):
        t = s.table_d.clone()
        t[1, 1] = bad
        o, st = run(table=t)
        assert st == R and torch.equal(o[:2], out[:2]) and o[2:].isfinite().all()
    for length in ([102, 1000], [102, 2 ** 31 - 1], [102, -5]):
        o, st = run(length=length)
        assert st == R and torch.equal(o[:2], out[:2])
    for cu in ([0, 2, 5], [0, -3, 4], [0, 2 ** 31 - 1, 4], [-2 ** 31, 2, 4]):
        assert run(cu=cu)[1] == I
    assert torch.equal(run()[0], out)


def test_no_rows(cuda_device):
    s = Case(cuda_device, H=1, Dk=64, Dv=64, page=16, block=16, start=[10, 5], n=[0, 0])
    out, lse = mlaq.cache_attn(torch.zeros((0, 2, 64), dtype=bf16, device=cuda_device), s.cache, s.table_d, s.length_d, cu=s.cu, lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    o = torch.full((3, 2, 64), 5.0, dtype=bf16, device=cuda_device)  # rows, but of no sequence
    mlaq.cache_attn(torch.zeros((3, 2, 64), dtype=bf16, device=cuda_device), s.cache, s.table_d, s.length_d, cu=s.cu, out=o)
    assert (o == 5).all()


def test_the_same_bytes_again(cuda_device):
    s = Case(cuda_device, H=4, Dk=128, Dv=128, page=64, block=32, start=[3000, 17, 900], n=[1, 1, 1])
    _, _, out, lse = attend(cuda_device, s, 32)
    for _ in range(5):
        _, _, o, l = attend(cuda_device, s, 32)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_captured_with_lengths_that_change(cuda_device):
    """A graph of a write and the attention behind it, replayed as the sequences grow; another graph beside it."""
    s = Case(cuda_device, H=2, Dk=64, Dv=64, page=16, block=8, start=[6, 29], n=[1, 1])
    g = torch.Generator().manual_seed(9)
    wide = torch.cat([s.table[:, :1], torch.arange(20, 28).view(2, 4).to(i32)], 1)
    cache = mlaq.KvCache.empty(40, 16, 2, 64, 64, block=8, device=cuda_device)
    for t in (cache.k, cache.v):
        t.fill_(0x7F)
    table = wide.to(cuda_device)
    table[:, 0] = torch.tensor([1, 2], dtype=i32)
    start = torch.zeros(2, dtype=i32, device=cuda_device)
    k, v = (torch.zeros((2, 2, 64), dtype=bf16, device=cuda_device) for _ in range(2))
    q = torch.zeros((2, 8, 64), dtype=bf16, device=cuda_device)

    def step(c):
        mlaq.kv_cache_write(c, k, v, table, start)
        start.add_(1)
        return mlaq.cache_attn(q, c, table, start)

    step(cache)  # warm
    start.zero_()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    with torch.cuda.graph(other):
        mlaq.cache_attn(q, cache, table, start)
    eager = mlaq.KvCache.empty(40, 16, 2, 64, 64, block=8, device=cuda_device)
    at = torch.zeros_like(start)
    for i in range(70):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).to(bf16))
        graph.replay()
        got = out.clone()
        other.replay()
        mlaq.kv_cache_write(eager, k, v, table, at)
        at.add_(1)
        assert torch.equal(got, mlaq.cache_attn(q, eager, table, at)), i


def test_far_pages(cuda_device):
    """Codes behind 2^32 bytes."""
    c = mlaq.KvCache.empty(2 ** 32 // (64 * 256) + 8, 64, 1, 256, 16, block=16, device=cuda_device)
    pages = c.k.shape[0]
    small = mlaq.KvCache.empty(4, 64, 1, 256, 16, block=16, device=cuda_device)
    table = torch.tensor([[pages - 1, 3]], dtype=i32, device=cuda_device)
    near = torch.tensor([[2, 3]], dtype=i32, device=cuda_device)
    k, v = (torch.randn((100, 1, D), device=cuda_device).to(bf16) for D in (256, 16))
    zero, cu = torch.zeros(1, dtype=i32, device=cuda_device), torch.tensor([0, 100], dtype=i32, device=cuda_device)
    length = torch.tensor([100], dtype=i32, device=cuda_device)
    q = torch.randn((1, 4, 256), device=cuda_device).to(bf16)
    got = []
    for cache, t in ((c, table), (small, near)):
        mlaq.kv_cache_write(cache, k, v, t, zero, cu=cu)
        got.append(mlaq.cache_attn(q, cache, t, length))
    assert torch.equal(*got)
