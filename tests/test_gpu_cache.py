"""The 8-bit cache of keys and values on the GPU: writes bit for bit against the rule in 64 bits, block by block, and
reads bit for bit against codes times scales."""
import math

import pytest
import torch

import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16, f32, f64, i32, u8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


def decode(codes, scales, block):
    """[pages, H, page, D] in 64 bits."""
    e = scales.to(i32).repeat_interleave(block, 2) - 127
    v = torch.ldexp(codes.view(torch.float8_e4m3fn).to(f64), e[..., None])
    return torch.where((e == 128)[..., None], torch.full_like(v, math.nan), v)


def code(v):
    """E4M3 codes (uint8) of v in 64 bits, |v| <= 448: nearest, ties to even; NaN and Inf keep their sign as NaN."""
    a = v.abs().clamp(max=448)
    _, k = torch.frexp(a.clamp(min=2.0 ** -6))
    n = torch.round(torch.ldexp(a, 4 - k))  # in steps of 2^(k - 4); torch rounds ties to even
    c = torch.ldexp(n, k - 4).to(f32).to(torch.float8_e4m3fn).view(u8)
    c = torch.where(v.isfinite(), c, torch.full_like(c, 0x7F))
    return c | (torch.signbit(v).to(u8) << 7)


def exponent(amax):
    """The smallest e in -127..127 with amax <= 448 2^e."""
    e = torch.full(amax.shape, -127, dtype=i32)
    for _ in range(255):
        e = torch.where((amax > torch.ldexp(torch.full_like(amax, 448.0), e)) & (e < 127), e + 1, e)
    return e


class Case:
    """A cache of pages in shuffled order with known contents, sequences with known lengths and new tokens."""

    def __init__(self, dev, H, Dk, Dv, page, block, start, n, shared=False, seed=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.start, self.n, self.block, self.page = start, n, block, page
        per = [-(-(a + b) // page) for a, b in zip(start, n)]
        pages = sum(per) + spare
        order = torch.randperm(pages, generator=g)
        width = max(per) + 1
        table, at = [], 0
        for k in per:
            table.append(torch.cat([order[at:at + k], torch.full((width - k,), -7)]))
            at += k
        self.table = torch.stack(table).to(i32)

        def codes(D):
            return torch.randint(0, 256, (pages, H, page, D), generator=g, dtype=u8)  # NaN codes among them

        def scales():
            return torch.randint(118, 124, (pages, H, page // block), generator=g, dtype=u8)

        self.host = [codes(Dk), scales()] + ([None, None] if shared else [codes(Dv), scales()])
        for b in range(len(n)):  # no NaN up to the last new token, whatever lies behind it
            t = torch.arange(start[b] + n[b])
            p, place = self.table[b, t // page].long(), t % page
            for c in (self.host[0], self.host[2]):
                if c is not None:
                    w = c[p, :, place]
                    c[p, :, place] = torch.where((w & 0x7F) == 0x7F, torch.full_like(w, 0x70), w)
        self.cache = mlaq.KvCache(*[None if t is None else t.to(dev) for t in self.host], Dv=Dv)
        cu = [0]
        for k in n:
            cu.append(cu[-1] + k)
        self.cu_list = cu
        self.cu = torch.tensor(cu, dtype=i32, device=dev)
        self.table_d, self.start_d = self.table.to(dev), torch.tensor(start, dtype=i32, device=dev)
        self.length_d = torch.tensor([a + b for a, b in zip(start, n)], dtype=i32, device=dev)
        T = cu[-1]
        spread = torch.exp(1.5 * torch.randn((T, H, 1), generator=g))
        self.k = (torch.randn((T, H, Dk), generator=g) * spread).to(bf16)
        self.v = None if shared else (torch.randn((T, H, Dv), generator=g) / spread).to(bf16)

    def written(self):
        """What the cache holds after the write, by the rule."""
        out = []
        for codes, scales, new in ((*self.host[:2], self.k), (*self.host[2:], self.v)):
            if codes is None:
                out += [None, None]
                continue
            codes, scales = codes.clone(), scales.clone()
            for b, (s, n) in enumerate(zip(self.start, self.n)):
                lo = self.cu_list[b]
                for first in range(s // self.block * self.block, s + n, self.block) if n else ():
                    p, place = int(self.table[b, first // self.page]), first % self.page
                    a, e = max(first, s), min(first + self.block, s + n)
                    v = new[lo + a - s:lo + e - s].to(f64).transpose(0, 1)  # [H, tokens, D]
                    amax = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)).amax((1, 2))
                    ex = exponent(amax)
                    j = place // self.block
                    if a > first:
                        old = scales[p, :, j].to(i32) - 127
                        ex = torch.maximum(ex, old)
                        held = codes[p, :, place:place + a - first]
                        w = torch.ldexp(held.view(torch.float8_e4m3fn).to(f64), (old - ex)[:, None, None])
                        codes[p, :, place:place + a - first] = torch.where((held & 0x7F) == 0x7F, held, code(w))
                    codes[p, :, place + a - first:place + e - first] = code(torch.ldexp(v, -ex[:, None, None]))
                    scales[p, :, j] = (ex + 127).to(u8)
            out += [codes, scales]
        return out

    def write(self, k=None, v=None, **kw):
        cu = kw.pop("cu", self.cu)
        dev = self.table_d.device
        mlaq.kv_cache_write(self.cache, self.k.to(dev) if k is None else k, (None if self.v is None else self.v.to(dev)) if v is None else v,
                            self.table_d, self.start_d, cu=cu, **kw)

    def now(self):
        return [None if t is None else t.cpu() for t in (self.cache.k, self.cache.k_scales, self.cache.v, self.cache.v_scales)]

    def check(self, want=None):
        for name, got, ref in zip(("k", "k_scales", "v", "v_scales"), self.now(), self.written() if want is None else want):
            assert (got is None) == (ref is None)
            if ref is not None:
                bad = (got != ref).nonzero()
                assert not len(bad), (name, len(bad), bad[:5].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


CASES = [
    dict(H=1, Dk=16, Dv=16, page=16, block=16, start=[0], n=[1]),
    dict(H=2, Dk=64, Dv=32, page=16, block=4, start=[0, 3, 17], n=[5, 1, 30]),
    dict(H=3, Dk=48, Dv=112, page=32, block=32, start=[31, 0, 40, 9], n=[2, 0, 70, 33]),
    dict(H=2, Dk=192, Dv=128, page=64, block=16, start=[5, 64, 63], n=[100, 1, 1]),
    dict(H=1, Dk=576, Dv=512, page=64, block=64, start=[0, 33, 100], n=[200, 64, 7], shared=True),
    dict(H=4, Dk=128, Dv=128, page=128, block=128, start=[1, 127], n=[300, 129]),
    dict(H=1, Dk=256, Dv=256, page=1024, block=512, start=[700, 0], n=[900, 1025]),  # more than a block's registers hold
    dict(H=5, Dk=80, Dv=96, page=16, block=1, start=[0, 15, 2], n=[1, 18, 3]),
]


@pytest.mark.parametrize("c", CASES)
def test_write(cuda_device, c):
    s = Case(cuda_device, **c)
    st = torch.zeros(1, dtype=i32, device=cuda_device)
    s.write(status=st)
    s.check()
    want = s.now()
    s.write()  # again, over itself: nothing changes
    s.check(want)
    assert st.item() == 0


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_read(cuda_device, c, dtype):
    s = Case(cuda_device, **c)
    for starts in (s.start, [0] * len(s.start)):  # the new rows, and as many from the first
        at = torch.tensor(starts, dtype=i32, device=cuda_device)
        k, v = mlaq.kv_cache_read(s.cache, s.table_d, at, sum(s.n) + 1, cu=s.cu, dtype=dtype)
        assert (v is None) == (s.host[2] is None)
        for got, codes, scales in ((k, s.host[0], s.host[1]), (v, s.host[2], s.host[3])):
            if got is None:
                continue
            full = decode(codes, scales, s.block)
            for b, n in enumerate(s.n):
                t = torch.arange(starts[b], starts[b] + n)
                want = full[s.table[b, t // s.page].long(), :, t % s.page].to(dtype)
                assert torch.equal(got[s.cu_list[b]:s.cu_list[b] + n].cpu().nan_to_num(99), want.nan_to_num(99))


def test_appending_token_by_token_holds_what_a_prompt_does_within_a_step(cuda_device):
    """A block whose scale was raised has been rounded twice: half a step of the smaller and half of the larger scale."""
    c = dict(H=2, Dk=64, Dv=64, page=32, block=16)
    s = Case(cuda_device, start=[0], n=[50], **c)
    for i in range(50):
        mlaq.kv_cache_write(s.cache, s.k[i:i + 1].to(cuda_device), s.v[i:i + 1].to(cuda_device), s.table_d,
                            torch.tensor([i], dtype=i32, device=cuda_device))
    k, _ = mlaq.kv_cache_read(s.cache, s.table_d, s.start_d, 50, cu=s.cu, dtype=f32)
    whole = Case(cuda_device, start=[0], n=[50], **c)
    whole.write()
    assert all(torch.equal(a, b) for a, b in zip((s.cache.k_scales, s.cache.v_scales), (whole.cache.k_scales, whole.cache.v_scales)))
    want = s.k.to(f64)
    scale = torch.stack([torch.ldexp(torch.ones(2, dtype=f64), whole.cache.k_scales.cpu().to(i32)[int(s.table[0, t // 32]), :, t % 32 // 16] - 127)
                         for t in range(50)])[..., None]
    # each of at most 15 roundings moves a value by half a step at its scale; scales double, so all before the last
    # sum to less than one more
    assert ((k.cpu().to(f64) - want).abs() <= 2 * (2.0 ** -4 * want.abs() + 2.0 ** -10 * scale) * (1 + 2.0 ** -4)).all()


def test_strides(cuda_device):
    """Keys and values as slices of one projection, heads before tokens, off 16 bytes, one row for all heads."""
    base = dict(H=2, Dk=64, Dv=32, page=16, block=8, start=[3, 20], n=[9, 30])
    s = Case(cuda_device, **base)
    k, v = s.k.to(cuda_device), s.v.to(cuda_device)
    joint = torch.cat([k, v], 2)
    s.write(joint[..., :64], joint[..., 64:])
    s.check()
    s = Case(cuda_device, **base)
    s.write(k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1))
    s.check()
    s = Case(cuda_device, **base)
    off = torch.zeros(k.numel() + 3, dtype=bf16, device=cuda_device)[3:].view_as(k).copy_(k)
    s.write(off, v)
    s.check()
    s = Case(cuda_device, **base)
    s.k = s.k[:, :1].expand(-1, 2, -1)
    s.write(k[:, :1].expand(-1, 2, -1), v)
    s.check()


def test_special_values(cuda_device):
    """NaN, Inf, zeros, the largest and the smallest bf16, in blocks with others."""
    s = Case(cuda_device, H=1, Dk=32, Dv=16, page=16, block=4, start=[0, 2], n=[16, 9])
    s.k[1, 0, 3], s.k[2, 0, 5], s.k[2, 0, 6] = math.nan, math.inf, -math.inf
    s.k[4:8] = 0
    s.k[8, 0, 0] = torch.finfo(bf16).max
    s.k[12:16] = s.k[12:16] * 0 + 2.0 ** -133
    s.k[13, 0, 1] = -2.0 ** -126
    s.v[:4] = math.nan
    s.k[20, 0, 0] = math.nan
    s.write()
    s.check()
    k, v = mlaq.kv_cache_read(s.cache, s.table_d, s.start_d, 25, cu=s.cu, dtype=f32)
    assert k.isnan().sum() == 4 and v.isnan().sum() == 4 * 16


def test_rows_behind_the_last_sequence(cuda_device):
    s = Case(cuda_device, H=2, Dk=32, Dv=32, page=16, block=16, start=[4, 0], n=[20, 0])
    k, v = (torch.full((25, 2, 32), math.nan, dtype=bf16, device=cuda_device) for _ in range(2))
    k[:20], v[:20] = s.k.to(cuda_device), s.v.to(cuda_device)
    s.write(k, v)
    s.check()
    out = torch.full((25, 2, 32), 7.0, dtype=bf16, device=cuda_device)
    mlaq.kv_cache_read(s.cache, s.table_d, s.start_d, 25, cu=s.cu, k=out)
    assert (out[20:] == 7).all() and not (out[:20] == 7).all()


def test_bad_pages_and_bounds(cuda_device):
    """Pages outside the cache, positions outside the table and rows outside the call are skipped and reported."""
    good = dict(H=1, Dk=32, Dv=32, page=16, block=16, start=[0, 0], n=[32, 32])
    R, I = mlaq.STATUS["MLA_ERR_POS_RANGE"], mlaq.STATUS["MLA_ERR_INVALID_ARG"]
    for bad in (-1, 1000, 2 ** 31 - 1, -2 ** 31):
        s = Case(cuda_device, **good)
        want = s.written()
        p = int(s.table[1, 1])
        for i in range(4):
            want[i][p] = s.host[i][p]
        s.table_d[1, 1] = bad
        st = torch.zeros(1, dtype=i32, device=cuda_device)
        s.write(status=st)
        s.check(want)
        assert st.item() == R
        st.zero_()
        mlaq.kv_cache_read(s.cache, s.table_d, s.start_d, 64, cu=s.cu, status=st)
        assert st.item() == R
    for starts, cu, code_ in (([0, -3], None, R), ([0, 2 ** 31 - 8], None, R), ([0, 40], None, R), ([0, 0], [0, 32, 65], I),
                              ([0, 0], [0, -5, 64], I), ([0, 0], [0, 2 ** 31 - 1, 64], I)):
        s = Case(cuda_device, **good)
        st = torch.zeros(1, dtype=i32, device=cuda_device)
        s.start_d.copy_(torch.tensor(starts, dtype=i32))
        cu = s.cu if cu is None else torch.tensor(cu, dtype=i32, device=cuda_device)
        s.write(cu=cu, status=st)
        assert st.item() == code_, (starts, cu)
        st.zero_()
        mlaq.kv_cache_read(s.cache, s.table_d, s.start_d, 64, cu=cu, status=st)
        assert st.item() == code_


def test_far_pages(cuda_device):
    """Codes behind 2^32 bytes."""
    c = mlaq.KvCache.empty(2 ** 32 // (64 * 256) + 8, 64, 1, 256, 16, block=16, device=cuda_device)
    pages = c.k.shape[0]
    table = torch.tensor([[pages - 1, 3]], dtype=i32, device=cuda_device)
    k = torch.randn((100, 1, 256), device=cuda_device).to(bf16)
    v = torch.randn((100, 1, 16), device=cuda_device).to(bf16)
    zero, cu = torch.zeros(1, dtype=i32, device=cuda_device), torch.tensor([0, 100], dtype=i32, device=cuda_device)
    mlaq.kv_cache_write(c, k, v, table, zero, cu=cu)
    small = mlaq.KvCache.empty(4, 64, 1, 256, 16, block=16, device=cuda_device)
    near = torch.tensor([[2, 3]], dtype=i32, device=cuda_device)
    mlaq.kv_cache_write(small, k, v, near, zero, cu=cu)
    assert torch.equal(c.k[pages - 1], small.k[2]) and torch.equal(c.k_scales[pages - 1], small.k_scales[2])
    for a, b in zip(mlaq.kv_cache_read(c, table, zero, 100, cu=cu), mlaq.kv_cache_read(small, near, zero, 100, cu=cu)):
        assert torch.equal(a, b)
