"""Rotary positions with several axes against the definition in 64 bits.

Bounds: an output is a sum of two products of float32 values, each rounded
once, so it is off by at most 2^-22 of the products' magnitudes; a sum of H
heads adds H * 2^-24 of the sum of magnitudes. A bf16 result is the rounding
of some value inside that bound: rounding is monotone, so it lies between the
roundings of the bound's two ends.
"""
import pytest
import torch

import synth
import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import autograd as mlaq_grad

pytestmark = pytest.mark.gpu
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def make(T, H, Dn, Dr, A, dtype, seed=0, pad=0, rows=97, dev="cuda:0"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, Dn + Dr + pad), generator=g).to(dtype).to(dev)[:, :, pad:]
    cos = torch.randn((rows, Dr + 4), generator=g).to(dev)  # any table: not only unit rotations
    sin = torch.randn((rows, Dr + 4), generator=g).to(dev)
    pos = torch.randint(0, rows, (A, T), generator=g).to(torch.int32).to(dev)
    axes = [int(a) for a in torch.randint(0, A, (Dr // 2,), generator=g)]
    return x, cos, sin, pos, axes


def reference(x, cos, sin, pos, axes, Dr, mode):
    """(result, bound before the rounding of the output) in 64 bits."""
    H, D = x.shape[1:]
    Dn, h = D - Dr, Dr // 2
    x = x.to(f64)
    mag = x.abs()
    steps = 4.0
    if mode == "sum":
        x, mag, steps = x.sum(1, keepdim=True), mag.sum(1, keepdim=True), 4.0 + H
    y, e = x.clone(), mag * (steps if mode == "sum" else 0.0)
    for i, a in enumerate(axes):
        row = pos[a].long()
        c0, c1 = cos[row, i].to(f64)[:, None], cos[row, i + h].to(f64)[:, None]
        s0, s1 = sin[row, i].to(f64)[:, None], sin[row, i + h].to(f64)[:, None]
        u, w, mu, mw = x[..., Dn + i], x[..., Dn + h + i], mag[..., Dn + i], mag[..., Dn + h + i]
        if mode != "apply":
            s0, s1 = -s1, -s0
        y[..., Dn + i], y[..., Dn + h + i] = u * c0 - w * s0, w * c1 + u * s1
        e[..., Dn + i] = steps * (mu * c0.abs() + mw * s0.abs())
        e[..., Dn + h + i] = steps * (mw * c1.abs() + mu * s1.abs())
    return y, e * 2.0 ** -24


def check(out, ref, bound):
    bf = out.dtype == bf16
    out = out.to(f64)
    if bf:
        bound = bound + ref.abs() * 2.0 ** -24  # 64 bits are rounded to bf16 by way of float32
        bad = (out < (ref - bound).to(bf16).to(f64)) | (out > (ref + bound).to(bf16).to(f64))
    else:
        bad = (out - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside their bounds"


SHAPES = [
    # T, H, Dn, Dr, A, pad: single token and head, odd counts, scalar and 16-byte paths, wide rows, many slots
    (1, 1, 0, 2, 1, 0), (1, 128, 128, 64, 3, 0), (3, 5, 7, 6, 2, 1), (33, 3, 16, 32, 3, 0), (130, 2, 128, 64, 3, 64),
    (17, 9, 40, 48, 4, 0), (64, 1, 0, 256, 3, 0), (5, 2, 1024, 128, 2, 0), (9, 2, 600, 250, 3, 3), (1000, 7, 8, 16, 3, 8),
]


@pytest.mark.parametrize("T,H,Dn,Dr,A,pad", SHAPES)
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("mode", ["apply", "inverse", "sum"])
def test_matches_definition(cuda_device, T, H, Dn, Dr, A, pad, dtype, mode):
    x, cos, sin, pos, axes = make(T, H, Dn, Dr, A, dtype, seed=T + H, pad=pad)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = mlaq.rope_axes(x, cos, sin, pos, axes, Dr, inverse=mode != "apply", sum_heads=mode == "sum", status=status)
    mlaq.check_status(status)
    assert out.shape == (T, 1 if mode == "sum" else H, Dn + Dr) and out.dtype == dtype
    check(out, *reference(x, cos, sin, pos, axes, Dr, mode))


def test_no_tokens(cuda_device):
    x, cos, sin, pos, axes = make(0, 4, 8, 16, 3, bf16)
    assert mlaq.rope_axes(x, cos, sin, pos, axes, 16).shape == (0, 4, 24)
    c, s = mlaq.rope_axes_table(cos, sin, pos, axes, 16)
    assert c.shape == s.shape == (0, 16)


def test_strided_output_and_head_major(cuda_device):
    """The key's rope part written in place of its slice; a head-major result; the rest of the buffers untouched."""
    x, cos, sin, pos, axes = make(37, 6, 0, 64, 3, bf16)
    ref, e = reference(x, cos, sin, pos, axes, 64, "apply")
    key = torch.full((37, 6, 192), 7.0, dtype=bf16, device=cuda_device)
    mlaq.rope_axes(x, cos, sin, pos, axes, 64, out=key[:, :, 128:])
    check(key[:, :, 128:], ref, e)
    assert (key[:, :, :128] == 7.0).all()
    heads = torch.empty((6, 37, 64), dtype=bf16, device=cuda_device)
    mlaq.rope_axes(x, cos, sin, pos, axes, 64, out=heads.transpose(0, 1))
    check(heads.transpose(0, 1), ref, e)


def test_one_axis_equals_the_projection_rope(cuda_device):
    """One axis is the framework's rotation: the same bits as kv_fwd's rotated key."""
    T, H, Dr = 70, 2, 64
    g = torch.Generator().manual_seed(3)
    c_kv = torch.randn((T, 64), generator=g).to(bf16).to(cuda_device)
    W = torch.randn((H * 64, 64), generator=g).to(bf16).to(cuda_device)
    k_pe = torch.randn((T, Dr), generator=g).to(bf16).to(cuda_device)
    cos, sin = (t.to(cuda_device) for t in synth.rope_table_standard(200, Dr))
    pos = torch.randint(0, 200, (1, T), generator=g).to(torch.int32).to(cuda_device)
    key, _ = mlaq.kv_fwd(c_kv, W, k_pe, cos, sin, H, 32, 32, Dr, pos=pos[0].contiguous())
    out = mlaq.rope_axes(k_pe.view(T, 1, Dr).expand(T, H, Dr), cos, sin, pos, [0] * (Dr // 2), Dr)
    ref, e = reference(k_pe.view(T, 1, Dr).expand(T, H, Dr), cos, sin, pos, [0] * (Dr // 2), Dr, "apply")
    check(out, ref, e)
    check(key[:, :, 32:], ref, e)


@pytest.mark.parametrize("Dr", [2, 16, 62, 64, 256])
@pytest.mark.parametrize("T", [1, 129])
def test_table_is_an_exact_gather(cuda_device, Dr, T):
    _, cos, sin, pos, axes = make(T, 1, 0, Dr, 3, f32)
    c, s = mlaq.rope_axes_table(cos, sin, pos, axes, Dr)
    rows = pos.long()[torch.tensor(axes * 2, device=cuda_device)].t()
    cols = torch.arange(Dr, device=cuda_device)[None]
    assert torch.equal(c, cos[rows, cols]) and torch.equal(s, sin[rows, cols])


def test_fused_projection_with_several_axes(cuda_device):
    """The per-token table turns the fused projection's query like rope_axes turns the plain one."""
    T, K, H, Dn, Dr = 130, 64, 4, 32, 16
    g = torch.Generator().manual_seed(5)
    x = torch.randn((T, K), generator=g).to(bf16).to(cuda_device)
    W = (torch.randn((H * (Dn + Dr), K), generator=g) / 8).to(bf16).to(cuda_device)
    _, cos, sin, pos, axes = make(T, H, Dn, Dr, 3, bf16)
    c, s = mlaq.rope_axes_table(cos, sin, pos, axes, Dr)
    q = mlaq.fwd(x, W, c, s, H, Dn, Dr, out_mode="bf16")
    plain = (x.to(f64) @ W.to(f64).t()).view(T, H, Dn + Dr)
    ref, _ = reference(plain, cos, sin, pos, axes, Dr, "apply")
    rms = ref.square().mean().sqrt()
    assert ((q.to(f64) - ref).abs() <= 8e-3 * ref.abs() + 2e-3 * rms).all()


def test_position_outside_the_table_is_reported(cuda_device):
    for bad in (-1, 97):
        x, cos, sin, pos, axes = make(33, 2, 8, 16, 2, bf16)
        axes = [0, 1] * 4
        pos[1, 20] = bad
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        out = mlaq.rope_axes(x, cos, sin, pos, axes, 16, status=status)
        assert int(status) == mlaq.STATUS["MLA_ERR_POS_RANGE"]
        ok = torch.arange(33, device=cuda_device) != 20
        pos[1, 20] = 0
        ref, e = reference(x, cos, sin, pos, axes, 16, "apply")
        check(out[ok], ref[ok], e[ok])  # the other tokens are right
        check(out[20, :, :8], ref[20, :, :8], e[20, :, :8])
        pos[1, 20] = bad
        status.zero_()
        mlaq.rope_axes_table(cos, sin, pos, axes, 16, status=status)
        assert int(status) == mlaq.STATUS["MLA_ERR_POS_RANGE"]


def test_infinities_and_nans_stay_in_their_pairs(cuda_device):
    x, cos, sin, pos, axes = make(20, 2, 8, 16, 2, f32)
    x = x.clone()
    x[3, 1, 9], x[4, 0, 2] = float("inf"), float("nan")
    out = mlaq.rope_axes(x, cos, sin, pos, axes, 16)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[3, 1, 9] = want[3, 1, 17] = want[4, 0, 2] = True
    assert torch.equal(bad, want)


def test_another_stream(cuda_device):
    x, cos, sin, pos, axes = make(513, 4, 64, 64, 3, bf16)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty((513, 4, 128), dtype=bf16, device=cuda_device)
    mlaq.rope_axes(x, cos, sin, pos, axes, 64, out=out, stream=s)
    s.synchronize()
    check(out, *reference(x, cos, sin, pos, axes, 64, "apply"))


def test_gradients(cuda_device):
    """The autograd faces against differences in 64 bits: the map is linear, so a difference quotient of the
    definition at any step is its derivative."""
    x, cos, sin, pos, axes = make(11, 3, 4, 8, 3, f32)
    g = torch.randn((11, 3, 12), generator=torch.Generator().manual_seed(9)).to(cuda_device)
    leaf = x.clone().requires_grad_()
    mlaq_grad.rope_axes(leaf, cos, sin, pos, axes, 8).backward(g)
    shared = x[:, :1].clone().requires_grad_()
    mlaq_grad.rope_axes(shared, cos, sin, pos, axes, 8, heads=3).backward(g)

    def loss(v):
        return (reference(v, cos, sin, pos, axes, 8, "apply")[0] * g.to(f64)).sum()

    for t, h, c in [(0, 0, 0), (3, 1, 4), (5, 2, 8), (10, 0, 11), (7, 1, 7)]:
        d = torch.zeros_like(x, dtype=f64)
        d[t, h, c] = 0.5
        diff = float(loss(x.to(f64) + d) - loss(x.to(f64) - d))
        # at most 2 products of magnitude below 100 in float32
        assert abs(float(leaf.grad[t, h, c]) - diff) <= 4 * 2.0 ** -24 * 100
        d = torch.zeros_like(x, dtype=f64)
        d[t, :, c] = 0.5
        diff = float(loss(x[:, :1].expand(-1, 3, -1).to(f64) + d) - loss(x[:, :1].expand(-1, 3, -1).to(f64) - d))
        assert abs(float(shared.grad[t, 0, c]) - diff) <= 8 * 2.0 ** -24 * 100


# more heads and rows than are resident at once: the path that gathers a block's table entries, its scalar and its wide
# form, runs of many tokens, and runs cut short by the table's room
ROWS = [(2100, 64, 16, 32, 3, 0), (1700, 33, 7, 6, 2, 1), (300, 20, 600, 250, 3, 3), (200, 130, 128, 256, 3, 0),
        (12000, 17, 0, 32, 4, 0), (1111, 50, 40, 48, 3, 8)]


@pytest.mark.parametrize("T,H,Dn,Dr,A,pad", ROWS)
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("mode", ["apply", "inverse", "sum"])
def test_many_rows(cuda_device, T, H, Dn, Dr, A, pad, dtype, mode):
    x, cos, sin, pos, axes = make(T, H, Dn, Dr, A, dtype, seed=T, pad=pad)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = mlaq.rope_axes(x, cos, sin, pos, axes, Dr, inverse=mode != "apply", sum_heads=mode == "sum", status=status)
    mlaq.check_status(status)
    check(out, *reference(x, cos, sin, pos, axes, Dr, mode))


def test_many_rows_report_a_bad_position(cuda_device):
    x, cos, sin, pos, axes = make(2100, 64, 16, 32, 2, bf16)
    axes = [0, 1] * 8
    ref, e = reference(x, cos, sin, pos, axes, 32, "apply")
    pos[1, 1500] = 97
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = mlaq.rope_axes(x, cos, sin, pos, axes, 32, status=status)
    assert int(status) == mlaq.STATUS["MLA_ERR_POS_RANGE"]
    ok = torch.arange(2100, device=cuda_device) != 1500
    check(out[ok], ref[ok], e[ok])


@pytest.mark.parametrize("T,Dr", [(16387, 64), (25001, 256), (5003, 30), (50001, 30), (90001, 64)])
@pytest.mark.parametrize("mixed", [False, True])
def test_table_of_many_tokens(cuda_device, T, Dr, mixed):
    """Several tokens per thread, axes in runs or mixed inside four columns; positions outside the table give zero."""
    _, cos, sin, pos, axes = make(T, 1, 0, Dr, 3, f32, rows=301)
    if not mixed:
        axes = sorted(axes)
    pos[1, 7], pos[2, T - 1] = -1, 301
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    c, s = mlaq.rope_axes_table(cos, sin, pos, axes, Dr, status=status)
    assert int(status) == mlaq.STATUS["MLA_ERR_POS_RANGE"]
    rows = pos.long()[torch.tensor(axes * 2, device=cuda_device)].t()
    inside = (rows >= 0) & (rows < 301)
    rows, cols = rows.clamp(0, 300), torch.arange(Dr, device=cuda_device)[None]
    assert torch.equal(c, cos[rows, cols] * inside) and torch.equal(s, sin[rows, cols] * inside)
