"""Attention over a cache whose blocks of values differ in scale: a row keeps its result whatever the values are that it gives
no weight, or does not see.

Tolerances. A weight p 2^e (e the exponent of the value's block) enters the second product as two E4M3 numbers by way of
f16: off by at most 2^-8 + 2^-11 of itself, and by half of their smallest step. The row's largest weight so far stands at
2^4 or up to 2^8, the smallest step is 2^-9 / 32 = 2^-14, so half of it is at most 2^-19 of the row's largest weight W, for
each code: 2^-19 W sum_j |code_j|. Scores and float32 sums as in test_gpu_cache_attn: (2^-12 + 2 ds) A with
A = sum_j p_j |v_j|, ds = (Dk + 8) 2^-23 of sum |q k| scale; the result is rounded to bf16, 2^-8 of it. A row's reference
may lie up to 94 below its scores (in powers of two): their difference, below 128, is a float32 number off by 2^-18 at most,
which a probability and the log-sum-exp are then off by as well."""
import math

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from test_gpu_cache import Case, decode
from test_gpu_cache_attn import check

pytestmark = pytest.mark.gpu
bf16, f32, f64, i32, u8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


def e4m3(v):
    return int(torch.tensor(v).to(torch.float8_e4m3fn).view(u8))


def scene(dev, seed=0, **c):
    """A cache of codes of magnitude 0.5 to 1 without zeros, keys of 2^-8 (scores near 0), values of 1."""
    s = Case(dev, seed=seed, **c)
    g = torch.Generator().manual_seed(seed + 100)
    for i in (0, 2):
        if s.host[i] is not None:
            shape = s.host[i].shape
            s.host[i] = torch.randint(0x30, 0x38, shape, generator=g, dtype=u8) | (torch.randint(0, 2, shape, generator=g, dtype=u8) << 7)
            s.host[i + 1].fill_(127)
    s.shared = s.host[2] is None
    if not s.shared:
        s.host[1].fill_(119)
    return s


def place(s, b, t):
    return int(s.table[b, t // s.page]), t % s.page


def block_of(s, b, t, score, e):
    """The block of sequence b's position t: values of 2^e, and keys of one score (for a query with 1 in the first channel
    that the scores use)."""
    p, at = place(s, b, t)
    first = at // s.block * s.block
    if s.shared:
        s.host[1][p, :, at // s.block] = 127 + e
        rows = s.host[0][p, :, first:first + s.block, s.cache.Dv:]
        rows[:] = 0
        rows[..., 0] = e4m3(score * 2.0 ** -e) or 0x81  # the least below 0
    else:
        s.host[3][p, :, at // s.block] = 127 + e
        s.host[1][p, :, at // s.block] = 127
        rows = s.host[0][p, :, first:first + s.block]
        rows[:] = 0
        rows[..., 0] = e4m3(score)


def attend(dev, s, Hq, seed=1, score=1.0):
    """Its outputs and the definition's in 64 bits with their tolerances."""
    for t, h in zip((s.cache.k, s.cache.k_scales, s.cache.v, s.cache.v_scales), s.host):
        if h is not None:
            t.copy_(h)
    T, Dk = sum(s.n), s.host[0].shape[3]
    H = s.host[0].shape[1]
    q = torch.randn((T, Hq, Dk), generator=torch.Generator().manual_seed(seed))
    if s.shared:
        q[..., :s.cache.Dv] = 0
        q *= 2.0 ** -8
    at = s.cache.Dv if s.shared else 0
    q[..., at] = score
    q = q.to(bf16)
    st = torch.zeros(1, dtype=i32, device=dev)
    out, lse = mlaq.cache_attn(q.to(dev), s.cache, s.table_d, s.length_d, cu=s.cu, scale=1.0, lse=True, status=st)
    assert st.item() == 0
    kk = decode(s.host[0], s.host[1], s.block)
    marks = s.host[1] if s.shared else s.host[3]
    codes = s.host[0][..., :s.cache.Dv] if s.shared else s.host[2]
    codes = codes.contiguous().view(torch.float8_e4m3fn).to(f64)
    want, wlse = torch.zeros((T, Hq, s.cache.Dv), dtype=f64), torch.zeros((T, Hq), dtype=f64)
    tol, ltol = torch.zeros_like(want), torch.zeros_like(wlse)
    for b, (start, n) in enumerate(zip(s.start, s.n)):
        t = torch.arange(start + n)
        p = s.table[b, t // s.page].long()
        k, c = kk[p, :, t % s.page], codes[p, :, t % s.page]  # [L, H, D]
        e = marks[p, :, t % s.page // s.block].to(f64) - 127
        for i in range(n):
            r, seen = s.cu_list[b] + i, start + i + 1
            qq = q[r].to(f64).view(H, Hq // H, Dk)
            z = torch.einsum("hgd,thd->hgt", qq, k[:seen])
            ds = (Dk + 8) * 2.0 ** -23 * torch.einsum("hgd,thd->hgt", qq.abs(), k[:seen].abs()).amax(2)
            w = torch.softmax(z, 2) * torch.exp2(e[:seen]).t()[:, None]
            o, a = torch.einsum("hgt,thd->hgd", w, c[:seen]), torch.einsum("hgt,thd->hgd", w, c[:seen].abs())
            least = 2.0 ** -19 * w.amax(2)[..., None] * c[:seen].abs().sum(0)[:, None]
            want[r], wlse[r] = o.flatten(0, 1), torch.logsumexp(z, 2).flatten()
            tol[r] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + 2 * ds[..., None]) * a + least).flatten(0, 1)
            ltol[r] = (ds + 2.0 ** -18 + 2.0 ** -20 + 2.0 ** -22 * wlse[r].view(H, -1).abs()).flatten()
    check(lse, wlse, ltol, "lse")
    check(out, want, tol, "out")
    return out, lse


# query rows for each of the kernel's tiles: 8, 16, 32 and 64; then latents
HEADS = [dict(Hq=4, c=dict(H=1, Dk=64, Dv=64)), dict(Hq=32, c=dict(H=2, Dk=128, Dv=80)), dict(Hq=32, c=dict(H=1, Dk=64, Dv=64)),
         dict(Hq=64, c=dict(H=1, Dk=64, Dv=128)), dict(Hq=8, c=dict(H=1, Dk=192, Dv=128, shared=True)),
         dict(Hq=72, c=dict(H=1, Dk=576, Dv=512, shared=True))]


@pytest.mark.parametrize("gap", [10, 14, 20, 40, 80])
@pytest.mark.parametrize("c", HEADS)
def test_a_block_of_larger_values_without_weight(cuda_device, c, gap):
    """In the first tile, in the middle and in the last."""
    s = scene(cuda_device, page=64, block=32, start=[1000, 700, 900], n=[1, 1, 1], **c["c"])
    for b, t in ((0, 40), (1, 400), (2, 899)):
        block_of(s, b, t, -0.15625 * 2.0 ** gap if s.shared and gap < 14 else -40.0, gap)
    if not s.shared:  # the row's own token, whose block is the last one's, has a weight
        p, at = place(s, 2, 900)
        s.host[0][p, :, at], s.host[2][p, :, at] = 0, 0
        s.host[0][p, :, at, 0] = e4m3(-40.0)
    attend(cuda_device, s, c["Hq"])


@pytest.mark.parametrize("gap", [20, 40])
@pytest.mark.parametrize("c", HEADS[:4])
def test_two_sinks_of_small_values(cuda_device, c, gap):
    """Nearly all weight, in two unequal parts, on tokens whose values are 2^-gap of the others', in tiles apart."""
    s = scene(cuda_device, page=64, block=1, start=[600], n=[1], **c["c"])
    for t, more in ((3, 0.75), (300, 0.0)):
        block_of(s, 0, t, 44.0, -gap)
        p, at = place(s, 0, t)
        s.host[0][p, :, at, 1] = e4m3(more)
    attend(cuda_device, s, c["Hq"])


@pytest.mark.parametrize("gap", [20, 60, 90])
@pytest.mark.parametrize("c", HEADS)
def test_a_later_token_of_larger_values(cuda_device, c, gap):
    """Each new token's values are far larger than those before: rows that do not see it keep their result."""
    s = scene(cuda_device, page=128, block=1, start=[130, 0], n=[20, 3], **c["c"])
    for b, t in ((0, 140), (0, 145), (1, 2)):
        block_of(s, b, t, 0.0, gap)
    attend(cuda_device, s, c["Hq"])


@pytest.mark.parametrize("c", HEADS[:4])
def test_scales_all_over(cuda_device, c):
    """Blocks of 2^-40 to 2^40 in any order."""
    s = scene(cuda_device, page=64, block=16, start=[1500, 77], n=[2, 1], **c["c"])
    s.host[3].copy_(torch.randint(87, 168, s.host[3].shape, generator=torch.Generator().manual_seed(4), dtype=u8))
    attend(cuda_device, s, c["Hq"])


@pytest.mark.parametrize("c", HEADS[:4])
def test_weights_that_balance_scales(cuda_device, c):
    """Scores that fall as the values grow, so that every block has a share in the result; and the other way round."""
    for sign in (-1, 1):
        s = scene(cuda_device, page=64, block=64, start=[1000], n=[1], **c["c"])
        for i, t in enumerate(range(0, 1000, 64)):
            block_of(s, 0, t, -2.75 * i, sign * 4 * i)  # 2.75 in powers of two: 3.97
        attend(cuda_device, s, c["Hq"])


@pytest.mark.parametrize("c", HEADS[:4])
def test_a_sink_of_zeros(cuda_device, c):
    """Nearly all weight on a token whose values are 0, at the least scale; then nothing but such values."""
    s = scene(cuda_device, page=64, block=1, start=[600], n=[1], **c["c"])
    block_of(s, 0, 0, 12.0, -127)
    p, at = place(s, 0, 0)
    s.host[2][p, :, at] = 0
    attend(cuda_device, s, c["Hq"])
    s.host[2].zero_(), s.host[3].zero_()
    out, _ = attend(cuda_device, s, c["Hq"])
    assert (out == 0).all()


@pytest.mark.parametrize("gap", [20, 80])
def test_parts_of_one_sequence(cuda_device, gap):
    """A sequence over every SM, one of whose parts holds larger values without weight, another the smaller ones with all."""
    s = scene(cuda_device, H=1, Dk=64, Dv=64, page=128, block=128, start=[40_000], n=[1])
    block_of(s, 0, 20_000, -40.0, gap)
    block_of(s, 0, 30_000, 12.0, -gap // 2)
    attend(cuda_device, s, 2)


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128, 256])
def test_scale_bytes_by_the_tile(cuda_device, block):
    """Every block has scales of its own, for keys and values, over more tiles than shared memory holds bytes for: a tile that
    got another's, or an older one's, is off by a power of two."""
    s = scene(cuda_device, H=2, Dk=64, Dv=64, page=256, block=block, start=[5000, 200, 2500], n=[1, 2, 1])
    g = torch.Generator().manual_seed(block)
    s.host[1].copy_(torch.randint(112, 121, s.host[1].shape, generator=g, dtype=u8))
    s.host[3].copy_(torch.randint(123, 132, s.host[3].shape, generator=g, dtype=u8))
    attend(cuda_device, s, 8)


@pytest.mark.parametrize("Hq", [2, 64])
def test_the_largest_values(cuda_device, Hq):
    """Values of 2^126 to 2^127, all of one sign, in parts: their sums are beyond float32, their mean is not."""
    s = scene(cuda_device, H=1, Dk=64, Dv=64, page=128, block=128, start=[40_000], n=[1])
    s.host[2] &= 0x7F
    s.host[3].fill_(254)
    out, _ = attend(cuda_device, s, Hq)
    assert out.isfinite().all()
