"""AdamW over many tensors against the formula in 64 bits and, for the 8-bit
moments, against the framework's MXFP8 rule on the exact neighbours.

Bounds (float32): m' and v' are sums of two products of rounded factors, off
by at most 4 * 2^-24 of the products' magnitudes; p' adds the step, whose
quotient has 2 ulp, a root and a product: 16 * 2^-24 of the step and 3 * 2^-24
of p. A bf16 parameter is the rounding of some value inside that bound, so it
lies between the roundings of the bound's two ends (rounded at random: within
one bf16 step, 2^-7 of the value, of it).
"""
import math

import numpy as np
import pytest
import torch

import oracle
import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16, f32, f64, u8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
HP = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [1, 31, 32, 33, 255, 4096, 8192, 8193, 20000, 0, 7]
E4M3 = np.array([oracle.e4m3_decode(c) for c in range(256)])


def flat(sizes, gen, std, dtype, offset):
    """Contiguous tensors inside one buffer, `offset` elements off a 256-byte start each."""
    out = []
    for n in sizes:
        t = torch.zeros(n + offset, dtype=f32)
        t[offset:] = torch.randn(n, generator=gen) * std
        out.append(t.to(dtype).to("cuda:0")[offset:])
    return out


def make(pdtype, gdtype, master, offset=0, seed=0, sizes=SIZES):
    g = torch.Generator().manual_seed(seed)
    masters = flat(sizes, g, 0.5, f32, offset)
    return dict(p=[t.to(pdtype) if offset == 0 else flat_like(t, pdtype, offset) for t in masters],
                g=flat(sizes, g, 0.1, gdtype, offset), m=flat(sizes, g, 0.03, f32, offset),
                v=[t.square_() for t in flat(sizes, g, 0.08, f32, offset)], ma=masters if master else None)


def flat_like(t, dtype, offset):
    b = torch.zeros(t.numel() + offset, dtype=dtype, device=t.device)
    b[offset:] = t.to(dtype)
    return b[offset:]


def formula(p, g, m, v, t, gs=1.0):
    b1, b2 = HP["betas"]
    g = g.to(f64) * gs
    m, v = b1 * m.to(f64) + (1 - b1) * g, b2 * v.to(f64) + (1 - b2) * g * g
    step = HP["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HP["eps"])
    return p.to(f64) * (1 - HP["lr"] * HP["weight_decay"]) - step, m, v, step


U = 2.0 ** -24


def near(p, ref, e, at_random):
    """A parameter tensor within e of ref, but for its own rounding."""
    got = p.to(f64)
    if p.dtype != bf16:
        return (got - ref).abs() <= e
    if at_random:
        return (got - ref).abs() <= e + ref.abs() * 2.0 ** -7
    e = e + ref.abs() * U  # 64 bits are rounded to bf16 by way of float32
    return (got >= (ref - e).to(bf16).to(f64)) & (got <= (ref + e).to(bf16).to(f64))


@pytest.mark.parametrize("pdtype,gdtype,master", [(bf16, bf16, True), (bf16, bf16, False), (f32, f32, False),
                                                  (f32, bf16, False), (bf16, f32, True)])
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("seed", [None, 1234])
def test_float32_moments(cuda_device, pdtype, gdtype, master, offset, seed):
    s = make(pdtype, gdtype, master, offset)
    gs = torch.full((1,), 0.375, device=cuda_device)
    old = {k: [t.clone() for t in v] for k, v in s.items() if v is not None}
    plan = mlaq.adamw_plan(s["p"], s["g"], s["m"], s["v"], masters=s["ma"])
    mlaq.adamw_step(plan, 7, grad_scale=gs, seed=seed, **HP)
    for i in range(len(SIZES)):
        p0 = (old["ma"] if master else old["p"])[i]
        p, m, v, step = formula(p0, old["g"][i], old["m"][i], old["v"][i], 7, 0.375)
        gm = (old["g"][i].to(f64) * 0.375).abs()
        assert ((s["m"][i].to(f64) - m).abs() <= 4 * U * (old["m"][i].to(f64).abs() + 0.1 * gm)).all()
        assert ((s["v"][i].to(f64) - v).abs() <= 5 * U * v).all()
        # the step's own moments are off as above, and m may cancel: carry its absolute error through the quotient
        rel_m = 4 * U * (old["m"][i].to(f64).abs() + 0.1 * gm) / m.abs().clamp(min=1e-300)
        e = 3 * U * (p0.to(f64).abs() + step.abs()) + step.abs() * (16 * U + rel_m)
        if master:
            assert ((s["ma"][i].to(f64) - p).abs() <= e).all()
            assert torch.equal(s["p"][i], s["ma"][i].to(bf16))
        else:
            assert near(s["p"][i], p, e, seed is not None).all()
        assert torch.equal(s["g"][i], old["g"][i])


def quantized(values, root=False):
    """(codes, scales) of flat float32 tensors by the framework's quantizer, as one block row each 32."""
    codes, scales = [], []
    for t in values:
        n = t.numel()
        if n == 0:
            codes.append(torch.zeros(0, dtype=u8, device=t.device))
            scales.append(torch.zeros(0, dtype=u8, device=t.device))
            continue
        pad = torch.zeros(-(-n // 32) * 32, device=t.device)
        pad[:n] = t.sqrt() if root else t
        c, s = mlaq.mxfp8_quantize_rows(pad.view(-1, 32))
        codes.append(c.reshape(-1)[:n].contiguous())
        scales.append(s.reshape(-1).contiguous())
    return codes, scales


def decoded(c, s):
    e = np.repeat(s.cpu().numpy().astype(np.int64) - 127, 32)[:c.numel()]
    return E4M3[c.cpu().numpy()] * np.exp2(e.astype(np.float64))


def moments32(m, v, g, t, gs):
    """m' and the root of v' in float32, each operation rounded once in the documented order."""
    b1, b2 = (np.float32(b) for b in HP["betas"])
    o1, o2 = (np.float32(1.0 - b) for b in HP["betas"])
    g = (g.astype(np.float32) * np.float32(gs)).astype(np.float32)
    m = m.astype(np.float32) * b1 + g * o1
    r = v.astype(np.float32)
    v = r * r * b2 + (g * o2) * g
    return m, np.sqrt(v)


def check_codes(c, s, want, stochastic, keep):
    """Scales follow the rule; every code is a nearest neighbour, or one of the two neighbours when random."""
    n = want.size
    pad = np.zeros(-(-n // 32) * 32)
    pad[:n] = want
    ref_c, ref_s = oracle.mxfp8_quantize(pad.reshape(-1, 32))
    assert np.array_equal(s.cpu().numpy(), ref_s.reshape(-1))
    c = c.cpu().numpy()
    if not stochastic:
        ref = ref_c.reshape(-1)[:n].copy()
        if keep:
            ref[(want > 0) & (ref == 0)] = 1
        assert np.array_equal(c, ref)
        return
    e = np.repeat(ref_s.reshape(-1).astype(np.int64) - 127, 32)[:n].astype(np.float64)
    scaled = np.abs(want) * np.exp2(-e)
    one = np.exp2(np.maximum(np.floor(np.log2(np.maximum(scaled, 1e-300))), -6.0) - 3)
    got = np.abs(E4M3[c])
    assert (np.abs(got - scaled) < one).all()
    assert ((c >> 7) == (np.signbit(want))).all()
    if keep:
        assert (got[want > 0] > 0).all()


@pytest.mark.parametrize("pdtype,gdtype,master", [(bf16, bf16, False), (bf16, bf16, True), (f32, f32, False),
                                                  (f32, bf16, False), (bf16, f32, False)])
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("seed", [None, 99])
def test_mxfp8_moments(cuda_device, pdtype, gdtype, master, offset, seed):
    s = make(pdtype, gdtype, master, offset, seed=4)
    s["m"][3][5], s["v"][3][5], s["g"][3][5] = 0.0, 0.0, 0.0  # a vanished element
    s["v"][5][:32] = 1e-12
    s["v"][5][3] = 1.0  # roots far below their block's largest
    cm, sm = quantized(s["m"])
    cv, sv = quantized(s["v"], root=True)
    if offset:
        cm, cv = ([flat_like(t, u8, offset) for t in c] for c in (cm, cv))
    old = [[decoded(a, b) for a, b in zip(c, k)] for c, k in ((cm, sm), (cv, sv))]
    p_old = [t.clone() for t in (s["ma"] if master else s["p"])]
    plan = mlaq.adamw_plan(s["p"], s["g"], cm, cv, masters=s["ma"], exp_avg_scales=sm, exp_avg_sq_scales=sv)
    mlaq.adamw_step(plan, 3, seed=seed, **HP)
    for i, n in enumerate(SIZES):
        if n == 0:
            continue
        g = s["g"][i].float().cpu().numpy()
        m, r = moments32(old[0][i], old[1][i], g, 3, 1.0)
        check_codes(cm[i], sm[i], m.astype(np.float64), seed is not None, False)
        check_codes(cv[i], sv[i], r.astype(np.float64), seed is not None, True)
        dev = [torch.from_numpy(old[0][i]).to(cuda_device), torch.from_numpy(old[1][i]).to(cuda_device).square()]
        p, m64, _, step = formula(p_old[i], s["g"][i], dev[0], dev[1], 3)
        rel_m = 4 * U * (dev[0].abs() + 0.1 * s["g"][i].to(f64).abs()) / m64.abs().clamp(min=1e-300)
        e = 3 * U * (p_old[i].to(f64).abs() + step.abs()) + step.abs() * (16 * U + rel_m)
        step0 = torch.isfinite(step) & (m64 != 0)
        assert near((s["ma"] if master else s["p"])[i], p, e, seed is not None)[step0].all()
        if master:
            assert torch.equal(s["p"][i], s["ma"][i].to(bf16))


def test_random_rounding_is_unbiased_and_reproducible(cuda_device):
    """A million equal values between two codes: the mean lies within 6 standard errors, the same seed gives the same
    codes and another seed others; places repeat for a tensor listed at the same place."""
    n = 1 << 20
    def run(seed):
        p = torch.zeros(n, device=cuda_device)
        g = torch.zeros(n, device=cuda_device)
        c, s = quantized([torch.full((n,), 0.875, device=cuda_device)])
        cv, sv = quantized([torch.full((n,), 1.0, device=cuda_device)])
        plan = mlaq.adamw_plan([p], [g], c, cv, exp_avg_scales=s, exp_avg_sq_scales=sv)
        mlaq.adamw_step(plan, 1, seed=seed, **HP)
        return c[0], s[0], p

    c, s, _ = run(5)
    want = 0.875 * float(np.float32(0.9))
    e = float(s[0]) - 127
    scaled = want * 2.0 ** -e
    one = 2.0 ** (math.floor(math.log2(scaled)) - 3)
    frac = scaled / one - math.floor(scaled / one)
    got = E4M3[c.cpu().numpy()] * 2.0 ** e
    assert abs(got.mean() - want) <= 6 * one * 2.0 ** e * math.sqrt(frac * (1 - frac) / n) + one * 2.0 ** (e - 16)
    assert torch.equal(run(5)[0], c) and not torch.equal(run(6)[0], c)
    # neighbouring places and the two moments' bits are not correlated: the up-roundings' autocorrelation vanishes
    up = (got > want).astype(np.float64)
    up -= up.mean()
    for lag in (1, 2, 8, 32, 64):
        assert abs((up[:-lag] * up[lag:]).mean()) <= 6 * up.var() / math.sqrt(n)


def test_non_finite_gradient_marks_its_block_only(cuda_device):
    n = 96
    s = make(f32, f32, False, sizes=[n])
    s["g"][0][40] = float("nan")
    cm, sm = quantized(s["m"])
    cv, sv = quantized(s["v"], root=True)
    plan = mlaq.adamw_plan(s["p"], s["g"], cm, cv, exp_avg_scales=sm, exp_avg_sq_scales=sv)
    for seed in (None, 3):
        mlaq.adamw_step(plan, 2, seed=seed, **HP)
        assert sm[0].tolist()[1] == 255 and sv[0].tolist()[1] == 255
        assert 255 not in (sm[0].tolist()[0], sm[0].tolist()[2], sv[0].tolist()[0], sv[0].tolist()[2])
    ok = torch.isfinite(s["p"][0])
    assert not ok[40] and ok[:32].all() and ok[64:].all()


@pytest.mark.parametrize("bits", [32, 8])
def test_many_small_tensors(cuda_device, bits):
    """Every tensor of a long list is stepped once, none twice."""
    sizes = [(i * 37) % 200 + 1 for i in range(700)]
    ps = [torch.ones(n, device=cuda_device) for n in sizes]
    opt = mlaq.AdamW(ps, lr=0.01, weight_decay=0.0, state_bits=bits)
    opt.step([torch.ones_like(p) for p in ps])
    for p in ps:
        # the first step of a fresh state is lr * g / (|g| + eps): 16 ulp of it as above
        assert ((p.double() - 0.99).abs() <= 20 * U).all()


def test_optimizer_follows_new_gradient_buffers_and_streams(cuda_device):
    p = torch.nn.Parameter(torch.ones(1000, device=cuda_device, dtype=bf16))
    q = p.detach().float().clone()
    opt = mlaq.AdamW([p], lr=0.125, betas=(0.9, 0.95), weight_decay=0.0, masters=True)
    m = v = torch.zeros(1000, dtype=f64, device=cuda_device)
    ref = q.to(f64)
    for t in range(1, 4):
        g = torch.full((1000,), float(t), dtype=bf16, device=cuda_device)
        p.grad = g
        side = torch.cuda.Stream(cuda_device)
        side.wait_stream(torch.cuda.current_stream())
        version = p._version
        opt.step(stream=side)
        assert p._version > version
        side.synchronize()
        m, v = 0.9 * m + 0.1 * t, 0.95 * v + 0.05 * t * t
        ref = ref - 0.125 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.95 ** t)).sqrt() + 1e-8)
    assert ((opt.masters[0].to(f64) - ref).abs() <= 100 * U).all()
    assert torch.equal(p.detach(), opt.masters[0].to(bf16))


def test_graph_replay(cuda_device):
    """A captured step replays: the launch holds no host state."""
    s = make(f32, f32, False, sizes=[5000])
    plan = mlaq.adamw_plan(s["p"], s["g"], s["m"], s["v"])
    start = [s[k][0].clone() for k in "pmv"]
    mlaq.adamw_step(plan, 1, **HP)
    want = [s[k][0].clone() for k in "pmv"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlaq.adamw_step(plan, 1, **HP)
    for k, t in zip("pmv", start):
        s[k][0].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s[k][0], w) for k, w in zip("pmv", want))


def test_random_rounding_keeps_nans_and_infinities(cuda_device):
    """A NaN or an infinite parameter stays one when it is rounded at random, whatever its bits and neighbours."""
    p = torch.ones(64, dtype=bf16, device=cuda_device)
    p[3], p[17], p[40] = float("nan"), float("inf"), -float("inf")
    p.view(torch.int16)[50] = -1  # a NaN with every bit set
    s = [torch.zeros(64, device=cuda_device) for _ in range(2)]
    plan = mlaq.adamw_plan([p], [torch.ones(64, dtype=bf16, device=cuda_device)], [s[0]], [s[1]])
    mlaq.adamw_step(plan, 1, seed=7, lr=1e-3, weight_decay=0.0)
    bad = torch.zeros(64, dtype=torch.bool, device=cuda_device)
    bad[[3, 50]] = True
    assert torch.equal(torch.isnan(p), bad) and p[17] == float("inf") and p[40] == -float("inf")
    rest = torch.ones(64, dtype=torch.bool, device=cuda_device)
    rest[[3, 17, 40, 50]] = False
    assert ((p[rest].double() - 0.999).abs() <= 2.0 ** -8).all()


def test_gradients_beyond_the_range_of_their_square(cuda_device):
    """v' overflows: it counts as the largest float32, and the parameters stay finite."""
    p, m, v = torch.ones(8, device=cuda_device), torch.zeros(8, device=cuda_device), torch.zeros(8, device=cuda_device)
    g = torch.full((8,), 1e30, device=cuda_device)
    g[1] = 1.0
    mlaq.adamw_step(mlaq.adamw_plan([p], [g], [m], [v]), 1, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0)
    assert torch.isfinite(p).all() and torch.isinf(v[0]) and torch.isfinite(v[1])



@pytest.mark.parametrize("bits", [32, 8])
def test_many_elements(cuda_device, bits):
    """Above 100 million elements a block may take more of them: the same results as in steps over fewer at a time."""
    sizes = [60_000_000, 40_000_000, 8191, 8193, 16383, 16384, 16385, 24577, 5]

    def run(some):
        p = [torch.linspace(-1, 1, n, device=cuda_device) for n in some]
        g = [t * 0.5 for t in p]
        kind, at, scales = (f32, 0.0, {}) if bits == 32 else (u8, 0, dict(
            zip(("exp_avg_scales", "exp_avg_sq_scales"),
                ([torch.zeros(-(-n // 32), dtype=u8, device=cuda_device) for n in some] for _ in range(2)))))
        m, v = ([torch.full((n,), at, dtype=kind, device=cuda_device) for n in some] for _ in range(2))
        plan = mlaq.adamw_plan(p, g, m, v, **scales)
        for step in (1, 2):
            mlaq.adamw_step(plan, step, lr=0.25, betas=(0.5, 0.75), weight_decay=0.0)
        return [p, m, v] + list(scales.values())

    whole, parts = run(sizes), [run(sizes[:1]), run(sizes[1:2]), run(sizes[2:])]
    for k, got in enumerate(whole):
        assert all(torch.equal(a, b) for a, b in zip(got, parts[0][k] + parts[1][k] + parts[2][k]))
    moved = whole[0][0] - torch.linspace(-1, 1, sizes[0], device=cuda_device)
    assert (moved[:29_000_000] > 0.2).all() and (moved[31_000_000:] < -0.2).all()
