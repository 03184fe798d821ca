"""The norm, the projections, the 8-bit cache and the attention over it as a decoder's attention block runs them: a
prompt, then single tokens; on other streams, in captured graphs side by side.

Tolerance of the attention against exact keys and values. Writing a block's scale 2^e, amax <= 448 2^e: a code is off by at
most 2^-4 of its value, or by 2^-10 2^e where it is subnormal; once more by the same where a later token raised the scale
(each raise rounds again, half a step of a coarser grid, so that all raises together are off by at most twice the last: 3
times in all is taken). The errors dk move a score by at most ds = scale sum |q dk|, a weight by the factor exp(2 max ds);
with A = sum p |v| and B = sum p dv the result is off by (A + B) (exp(2 ds) - 1) + B, and by what the kernel itself may
be (2^-7 A with room, the scores being of a few units)."""
import math

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import autograd

pytestmark = pytest.mark.gpu
bf16, f32, f64, i32, u8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
H, Dn, Dr, Dv, K, KL, PAGE, BLOCK = 2, 64, 64, 64, 256, 128, 16, 8


class Block:
    """One attention block's weights, cache and pages for sequences of up to 96 positions."""

    def __init__(self, dev, B, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rand(*s, std=1.0, dtype=bf16):
            return (torch.randn(s, generator=g) * std).to(dtype).to(dev)

        self.dev, self.B, self.rand = dev, B, rand
        self.wx, self.wl = 1 + rand(K, std=0.1, dtype=f32), 1 + rand(KL, std=0.1)
        self.W, self.Ws = mlaq.mxfp8_quantize_rows(rand(H * (Dn + Dr), K, std=K ** -0.5))
        self.Wkv = rand(H * (Dn + Dv), KL, std=KL ** -0.5)
        t = torch.arange(96)[:, None] * torch.exp2(-torch.arange(Dr // 2) / 4)
        self.cos, self.sin = (torch.cat([f(t)] * 2, 1).to(dev) for f in (torch.cos, torch.sin))
        self.cache = mlaq.KvCache.empty(B * 6 + 3, PAGE, H, Dn + Dr, Dv, block=BLOCK, device=dev)
        for c in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales):
            c.fill_(0xFF)  # NaN wherever nothing is written
        self.table = torch.randperm(B * 6 + 3, generator=g)[:B * 6].view(B, 6).to(i32).to(dev)

    def inputs(self, T):
        return self.rand(T, K), self.rand(T, K), self.rand(T, KL), self.rand(T, Dr)

    def step(self, ins, start, length, pos, cu=None, each=lambda: None):
        """(out, lse, h, q, k, v); each() is called behind every operator."""
        x, r, latent, k_pe = ins
        codes, scales, h = mlaq.rms_norm_fwd(x, self.wx, residual=r, out="mxfp8")
        each()
        q = mlaq.fwd(codes, self.W, self.cos, self.sin, H, Dn, Dr, pos=pos, weight_mode="mxfp8", x_scales=scales,
                     w_scales=self.Ws, out_mode="bf16")
        each()
        c = mlaq.rms_norm_fwd(latent, self.wl)
        each()
        k, v = mlaq.kv_fwd(c, self.Wkv, k_pe, self.cos, self.sin, H, Dn, Dv, Dr, pos=pos)
        each()
        mlaq.kv_cache_write(self.cache, k, v, self.table, start, cu=cu)
        each()
        out, lse = mlaq.cache_attn(q, self.cache, self.table, length, cu=cu, lse=True)
        each()
        return out, lse, h, q, k, v


def ints(dev, v):
    return torch.tensor(v, dtype=i32, device=dev)


def quantum(x):
    """What a cached x may be off by, from the largest of its block's neighbours: [tokens, H, D], blocks of BLOCK tokens."""
    amax = x.abs().amax(2)
    top = torch.stack([amax[t // BLOCK * BLOCK:(t // BLOCK + 1) * BLOCK].amax(0) for t in range(len(x))])
    e = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-30) / 448)))
    return 3 * torch.maximum(2.0 ** -4 * x.abs(), (2.0 ** -10 * e)[..., None].expand_as(x))


def check_attention(q, k, v, first, out, lse):
    """Rows of one sequence: row i sees first + i + 1 of the exact keys and values."""
    if not len(q):
        return
    q, k, v = (t.cpu().to(f64) for t in (q, k, v))
    scale = (Dn + Dr) ** -0.5
    dk, dv = quantum(k), quantum(v)
    for i in range(len(q)):
        n = first + i + 1
        z = torch.einsum("hd,thd->ht", q[i], k[:n]) * scale
        w = torch.softmax(z, 1)
        ds = (torch.einsum("hd,thd->ht", q[i].abs(), dk[:n]) * scale).amax(1)[:, None]
        want = torch.einsum("ht,thd->hd", w, v[:n])
        a, b = (torch.einsum("ht,thd->hd", w, t) for t in (v[:n].abs(), dv[:n]))
        tol = (a + b) * torch.expm1(2 * ds) + b + 2.0 ** -7 * a
        assert ((out[i].cpu().to(f64) - want).abs() <= tol).all(), (i, (out[i].cpu().to(f64) - want).abs().max(), tol.min())
        assert ((lse[i].cpu().to(f64) - torch.logsumexp(z, 1)).abs() <= ds[:, 0] + 1e-4).all()


def test_a_prompt_and_the_tokens_behind_it(cuda_device):
    """Without a wait between the operators, and with one behind each: the same bytes; the attention within its bound of the
    exact keys and values; the norm's sum h; the single tokens on another stream."""
    n = [40, 1, 0, 67]
    got = []
    for wait in (False, True):
        each = torch.cuda.synchronize if wait else lambda: None
        s = Block(cuda_device, len(n))
        cu = [0, 40, 41, 41, 108]
        pos = ints(cuda_device, [i for m in n for i in range(m)])
        prompt = s.inputs(108)
        r = s.step(prompt, ints(cuda_device, [0] * 4), ints(cuda_device, n), pos, ints(cuda_device, cu), each)
        torch.cuda.synchronize()
        assert torch.equal(r[2], (prompt[0].float() + prompt[1].float()).to(bf16))
        results, kv = [r], [[t[a:b] for t in r[4:]] for a, b in zip(cu, cu[1:])]
        side = torch.cuda.Stream(cuda_device)
        for i in range(5):
            ins = s.inputs(4)
            start = ints(cuda_device, [m + i for m in n])
            length = start + 1
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                r = s.step(ins, start, length, start, None, each)
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            results.append(r)
            for b in range(4):
                kv[b] = [torch.cat([old, t[b:b + 1]]) for old, t in zip(kv[b], r[4:])]
        got.append(results)
        if not wait:
            for b in range(4):
                k, v = kv[b]
                check_attention(results[0][3][cu[b]:cu[b + 1]], k[:n[b]], v[:n[b]], 0, *[t[cu[b]:cu[b + 1]] for t in results[0][:2]])
                for i, r in enumerate(results[1:]):
                    m = n[b] + i
                    check_attention(r[3][b:b + 1], k[:m + 1], v[:m + 1], m, r[0][b:b + 1], r[1][b:b + 1])
    for a, b in zip(*got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_side_by_side(cuda_device):
    """Two captured blocks replayed on two streams at once, and an eager one beside them, each as it is alone."""
    blocks, alone, graphs, outs = [Block(cuda_device, 3, seed) for seed in (1, 2, 3)], [], [], []
    args = [(b.inputs(3), ints(cuda_device, [0] * 3), ints(cuda_device, [1] * 3), ints(cuda_device, [0] * 3)) for b in blocks]
    for b, a in zip(blocks, args):
        alone.append([t.clone() for t in b.step(*a)])
    torch.cuda.synchronize()
    for b, a in zip(blocks[:2], args):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(b.step(*a))
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    for _ in range(20):
        for g, st, o in zip(graphs, streams, outs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                for t in o:
                    t.zero_()
                g.replay()
        eager = blocks[2].step(*args[2])
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        for got, want in zip([*outs, eager], alone):
            assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_stream_that_is_passed(cuda_device):
    """stream= another one than the current: the same bytes."""
    s = Block(cuda_device, 2)
    ins = s.inputs(2)
    zero, one = ints(cuda_device, [0, 0]), ints(cuda_device, [1, 1])
    out, lse, h, q, k, v = s.step(ins, zero, one, zero)
    rstd = mlaq.rms_norm_fwd(h, s.wx, save=True)[1]
    dx, dw = mlaq.rms_norm_bwd(ins[0], h, s.wx, rstd)
    a, b = mlaq.kv_cache_read(s.cache, s.table, zero, 2)
    side = torch.cuda.Stream(cuda_device)
    other = mlaq.KvCache.empty(*s.cache.k.shape[:1], PAGE, H, Dn + Dr, Dv, block=BLOCK, device=cuda_device)
    torch.cuda.synchronize()
    h2 = mlaq.rms_norm_fwd(ins[0], s.wx, residual=ins[1], stream=side)[1]
    grads = mlaq.rms_norm_bwd(ins[0], h2, s.wx, rstd, stream=side)
    mlaq.kv_cache_write(other, k, v, s.table, zero, stream=side)
    dense = mlaq.kv_cache_read(other, s.table, zero, 2, stream=side)
    o, l = mlaq.cache_attn(q, other, s.table, one, lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((h, dx, dw, a, b, out, lse), (h2, *grads, *dense, o, l)):
        assert torch.equal(x, y)


def test_the_norms_gradient_in_a_graph(cuda_device):
    g = torch.Generator().manual_seed(4)
    x, r, dy, dh = (torch.randn((300, 136), generator=g).to(bf16).to(cuda_device) for _ in range(4))
    w = torch.ones(136, dtype=f32, device=cuda_device)

    def gradients():
        leaves = [t.detach().requires_grad_() for t in (x, w, r)]
        return torch.autograd.grad(autograd.rms_norm(leaves[0], leaves[1], residual=leaves[2]), leaves, (dy, dh))

    side = torch.cuda.Stream(cuda_device)
    with torch.cuda.stream(side):
        gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gradients()
    for _ in range(3):
        for t in (x, r, dy, dh):
            t.copy_(torch.randn(t.shape, generator=g).to(bf16))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, gradients()))


def test_lse_alone_and_scales_that_are_refused(cuda_device):
    s = Block(cuda_device, 2)
    zero, one = ints(cuda_device, [0, 0]), ints(cuda_device, [1, 1])
    out, lse, _, q, _, _ = s.step(s.inputs(2), zero, one, zero)
    mine = torch.zeros_like(lse)
    o, l = mlaq.cache_attn(q, s.cache, s.table, one, lse=mine)
    assert l is mine and torch.equal(l, lse) and torch.equal(o, out)
    for scale in (math.nan, math.inf, -math.inf):
        with pytest.raises(ValueError):
            mlaq.cache_attn(q, s.cache, s.table, one, scale=scale)


def test_bounds_that_fall(cuda_device):
    """cu has to rise; one that falls ends the call, touches no other row and leaves the next call alone."""
    s = Block(cuda_device, 6)
    n = [9, 30, 0, 5, 17, 3]
    cu = [0, 9, 39, 39, 44, 61, 64]
    pos = ints(cuda_device, [i for m in n for i in range(m)])
    zero, length = ints(cuda_device, [0] * 6), ints(cuda_device, n)
    out, lse, _, q, _, _ = s.step(s.inputs(64), zero, length, pos, ints(cuda_device, cu))
    wide = torch.full((70, H, Dv), 3.0, dtype=bf16, device=cuda_device)
    many = torch.cat([q, q[:6]])
    for bad in ([0, 39, 9, 39, 44, 61, 64], [0, 64, 0, 64, 0, 64, 0], [64, 61, 44, 39, 39, 9, 0], [0, 9, 39, 0, 44, 2, 64],
                [5, 4, 3, 2, 1, 0, 64], [0, 0, 0, 64, 0, 0, 0]):
        mlaq.cache_attn(many, s.cache, s.table, length, cu=ints(cuda_device, bad), out=wide)
        torch.cuda.synchronize()
        assert (wide[64:] == 3).all()
    assert torch.equal(mlaq.cache_attn(q, s.cache, s.table, length, cu=ints(cuda_device, cu)), out)
