"""Workloads of the training-step operators around the query up-projection:
the gated feed-forward block, rotary positions with several axes and AdamW
over many tensors, each with its plain form in elementary torch operations.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` their
inputs, ``run(state)`` one pass: the plain form, or (``own = True``) the
package's calls. ``exact(case, seed)`` is the same result from the definition
in 64 bits and ``work(case)`` the bytes and operations a pass cannot avoid.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token through the feed-forward block: the weights are read once
        dict(name="ffn_fwd_token", op="ffn_fwd", T=1, K=2048, F=5632, act="silu", save=False, pitch=0),
        # a decode batch (a few sequences) through a wide block
        dict(name="ffn_fwd_decode24", op="ffn_fwd", T=24, K=4096, F=11008, act="silu", save=False, pitch=0),
        # a ragged micro-batch of a training step, activations kept, x a slice of a wider buffer
        dict(name="ffn_fwd_ragged", op="ffn_fwd", T=1001, K=1536, F=4104, act="gelu_tanh", save=True, pitch=64),
        # a full training micro-batch, activations kept
        dict(name="ffn_fwd_train", op="ffn_fwd", T=8192, K=4096, F=14336, act="silu", save=True, pitch=0),
        # the gradient of a small ragged micro-batch
        dict(name="ffn_bwd_ragged", op="ffn_bwd", T=777, K=1536, F=4096, act="gelu", pitch=0),
        # the gradient of a training micro-batch
        dict(name="ffn_bwd_train", op="ffn_bwd", T=4096, K=4096, F=14336, act="silu", pitch=0),
        # one generated token's query: 128 heads of 128 + 64 channels, three axes
        dict(name="rope_token", op="rope", mode="apply", T=1, H=128, Dn=128, Dr=64, A=3, dtype="bf16", pad=0),
        # the per-token table of a video clip's positions for the fused projection
        dict(name="rope_table_video", op="rope", mode="table", T=16384, H=1, Dn=0, Dr=64, A=3, dtype="fp32", pad=0),
        # a video micro-batch's query heads
        dict(name="rope_video", op="rope", mode="apply", T=8190, H=128, Dn=128, Dr=64, A=3, dtype="bf16", pad=0),
        # the gradient of the rope key that all heads share, read from the key gradient's slices
        dict(name="rope_shared_grad", op="rope", mode="sum", T=4096, H=128, Dn=0, Dr=64, A=3, dtype="bf16", pad=128),
        # a layer's small tensors and matrices: fp32 moments, bf16 weights with fp32 masters
        dict(name="adamw_layer32", op="adamw", bits=32, tensors=40, total=3_000_000, sizes=1, param="bf16",
             master=True, stochastic=False, align=64),
        # a model's worth of tensors, MXFP8 moments, stochastic rounding of moments and bf16 weights
        dict(name="adamw_model8", op="adamw", bits=8, tensors=290, total=300_000_000, sizes=2, param="bf16",
             master=False, stochastic=True, align=64),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_bwd", "rope", "adamw"])
    if op.startswith("ffn"):
        cap = 8192 * 4096 * 14336 // (1 if op == "ffn_fwd" else 2)
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 8192), K=_log_int(rng, 256, 4096, 8), F=_log_int(rng, 256, 14336, 8),
                     act=rng.choice(["silu", "gelu", "gelu_tanh"]), pitch=rng.choice([0, 0, 8, 136]))
            if c["T"] * c["K"] * c["F"] <= cap:
                break
        if op == "ffn_fwd":
            c["save"] = rng.random() < 0.5
        return c
    if op == "rope":
        mode = rng.choice(["apply", "inverse", "sum", "table"])
        Dr = rng.choice([16, 32, 48, 64, 96, 128])
        if mode == "table":
            return dict(op=op, mode=mode, T=_log_int(rng, 1, 32768), H=1, Dn=0, Dr=Dr, A=rng.randint(1, 4),
                        dtype="fp32", pad=0)
        H = _log_int(rng, 1, 128)
        return dict(op=op, mode=mode, T=_log_int(rng, 1, 8190), H=H, Dn=rng.choice([0, 0, 32, 40, 64, 128]), Dr=Dr,
                    A=rng.randint(1, 4), dtype=rng.choice(["bf16", "bf16", "fp32"]), pad=rng.choice([0, 0, 8, 13, 64]))
    bits = rng.choice([32, 8])
    stochastic = rng.random() < 0.5
    param = rng.choice(["bf16", "bf16", "fp32"])
    return dict(op=op, bits=bits, tensors=_log_int(rng, 1, 300), total=_log_int(rng, 20_000, 100_000_000),
                sizes=rng.randrange(1 << 20), param=param, master=param == "bf16" and rng.random() < 0.5,
                stochastic=stochastic, align=64 if bits == 8 or stochastic else rng.choice([64, 1]))


def _sizes(case):
    """The tensors' sizes: log-uniform weights shared out over about `total` elements, odd ones among them, and their
    places in the flat buffers (each place a multiple of `align`)."""
    rng = random.Random(case["sizes"])
    w = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    n = [max(1, int(case["total"] * v / sum(w))) for v in w]
    places, at = [], 0
    for v in n:
        places.append(at)
        at += -(-v // case["align"]) * case["align"]
    return n, places, at


def work(case):
    if case["op"] == "ffn_fwd":
        T, K, F = case["T"], case["K"], case["F"]
        return {"bytes": 2 * (2 * T * K + 3 * F * K + (3 * T * F if case["save"] else 0)), "flops": 6 * T * K * F}
    if case["op"] == "ffn_bwd":
        T, K, F = case["T"], case["K"], case["F"]
        return {"bytes": 2 * (3 * T * K + 6 * F * K + 3 * T * F), "flops": 12 * T * K * F}
    if case["op"] == "rope":
        T, H, D, Dr, A = case["T"], case["H"], case["Dn"] + case["Dr"], case["Dr"], case["A"]
        size = 2 if case["dtype"] == "bf16" else 4
        if case["mode"] == "table":
            return {"bytes": 4 * A * T + 16 * T * Dr, "flops": T * Dr}
        outs = T * D if case["mode"] == "sum" else T * H * D
        rows = min(A * T, _rows(case))
        return {"bytes": size * (T * H * D + outs) + 4 * A * T + 8 * rows * Dr,
                "flops": 3 * T * Dr * (1 if case["mode"] == "sum" else H) + (T * H * D if case["mode"] == "sum" else 0)}
    n = sum(_sizes(case)[0])
    p = 2 if case["param"] == "bf16" else 4
    state = 8 if case["bits"] == 32 else 2 + 2 / 32
    m = 4 if case["master"] else 0
    # gradient read, parameter written (and read where it has no master), master and moments read and written
    return {"bytes": n * (p + p + (0 if m else p) + 2 * m + 2 * state), "flops": 16 * n}


# ------------------------------------------------------------------ inputs
def _rows(case):
    return 4096 if case["T"] <= 4096 else 16384


def _positions(case, g):
    """Positions of a clip of frames of patches: axis 0 the frame, axis 1 the row, axis 2 the column, axis 3 a text
    position; a clip starts at an offset drawn from the seed."""
    T, A = case["T"], case["A"]
    t = torch.arange(T, device=DEV, dtype=torch.int64)
    w = max(1, min(64, int(math.isqrt(T))))
    off = int(torch.randint(0, 64, (1,), generator=g, device=DEV))
    if A == 1:
        return ((t + off) % _rows(case)).to(torch.int32)[None]
    axes = [t // (w * w) + off, (t // w) % w + off, t % w + off, t + off]
    return (torch.stack(axes[:A]) % _rows(case)).to(torch.int32).contiguous()


def _axes(case):
    """Which axis each of the Dr/2 pairs follows: contiguous sections, the first the widest."""
    h, A = case["Dr"] // 2, case["A"]
    s = [h // A + (1 if i < h % A else 0) for i in range(A)]
    return [a for a in range(A) for _ in range(s[a])]


def _tables(case):
    Dr, rows = case["Dr"], _rows(case)
    f = 10000.0 ** (-torch.arange(0, Dr, 2, device=DEV, dtype=torch.float64) / Dr)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * torch.cat([f, f])[None]
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case=case)
    op = case["op"]
    if op.startswith("ffn"):
        T, K, F = case["T"], case["K"], case["F"]
        s["x"] = normal(T, K + case["pitch"])[:, :K]
        s["w_gate_up"] = normal(2 * F, K, std=K ** -0.5)
        s["w_down"] = normal(K, F, std=F ** -0.5)
        if op == "ffn_bwd":
            s["dy"] = normal(T, K, std=0.01)
            s["gate_up"] = normal(T, 2 * F)  # gates and up products of unit variance, as the fwd gives them
            a = _act(s["gate_up"][:, :F].float(), case["act"])[0]
            s["h"] = (a * s["gate_up"][:, F:].float()).to(torch.bfloat16)
    elif op == "rope":
        s["cos"], s["sin"] = _tables(case)
        s["pos"] = _positions(case, g)
        s["axes"] = _axes(case)
        s["axis_of_channel"] = torch.tensor(s["axes"] * 2, device=DEV)
        D = case["Dn"] + case["Dr"]
        if case["mode"] != "table":
            dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
            s["x"] = normal(case["T"], case["H"], D + case["pad"], dtype=dt)[:, :, case["pad"]:]
        else:
            # a clip's positions do not hold random numbers: another seed is another table scale
            a = 1.0 + 0.25 * torch.rand(1, generator=g, device=DEV)
            s["cos"], s["sin"] = s["cos"] * a, s["sin"] * a
    else:
        n, places, total = _sizes(case)
        pd = torch.bfloat16 if case["param"] == "bf16" else torch.float32
        used = torch.zeros(total, dtype=torch.bool, device=DEV)
        for v, at in zip(n, places):
            used[at:at + v] = True

        def flat(std, dtype=torch.float32):
            return torch.where(used, normal(total, std=std, dtype=torch.float32), torch.zeros((), device=DEV)).to(dtype)

        p32 = flat(0.02)
        s["p"] = p32.to(pd)
        s["master"] = p32 if case["master"] else None
        s["g"] = flat(0.01, pd)
        m, v = flat(0.003), flat(0.008).square()
        s["grad_scale"] = 0.5 + torch.rand(1, generator=g, device=DEV)
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["ms"] = _encode(m, None)
            s["v"], s["vs"] = _encode(v.sqrt(), None, keep=True)
        s["step"], s["lr"], s["betas"], s["eps"], s["wd"] = 100, 3e-4, (0.9, 0.95), 1e-8, 0.1
        s["seed"] = (int(seed) * 2654435761) % (1 << 31) if case["stochastic"] else None
        if own:
            import up_proj_gemm_gb300 as mlaq

            def views(t, per=1):
                return None if t is None else [t[at // per:at // per + -(-k // per)] for k, at in zip(n, places)]

            s["plan"] = mlaq.adamw_plan(views(s["p"]), views(s["g"]), views(s["m"]), views(s["v"]),
                                        masters=views(s["master"]), exp_avg_scales=views(s.get("ms"), 32),
                                        exp_avg_sq_scales=views(s.get("vs"), 32))
    return s


# ------------------------------------------------------------- plain forms
def _act(g, act):
    """(act(g), act'(g))"""
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e * (1.0 + g * (1.0 - e))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    k = (2.0 / math.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _ffn_fwd(s, wide, out):
    c = s["case"]
    gu = s["x"].to(wide) @ s["w_gate_up"].to(wide).t()
    h = _act(gu[:, :c["F"]], c["act"])[0] * gu[:, c["F"]:]
    y = h @ s["w_down"].to(wide).t()
    return dict(y=y.to(out), gate_up=gu.to(out), h=h.to(out)) if c["save"] else dict(y=y.to(out))


def _ffn_bwd(s, wide, out):
    c = s["case"]
    F = c["F"]
    dy, gu = s["dy"].to(wide), s["gate_up"].to(wide)
    dh = dy @ s["w_down"].to(wide)
    a, da = _act(gu[:, :F], c["act"])
    dgu = torch.cat([dh * gu[:, F:] * da, dh * a], 1)
    return dict(dx=(dgu @ s["w_gate_up"].to(wide)).to(out), dw_gate_up=(dgu.t() @ s["x"].to(wide)).to(out),
                dw_down=(dy.t() @ s["h"].to(wide)).to(out))


def _rope(s):
    c = s["case"]
    Dr = c["Dr"]
    rows = s["pos"].long()[s["axis_of_channel"]].t()  # [T, Dr]
    cos, sin = s["cos"].gather(0, rows), s["sin"].gather(0, rows)
    if c["mode"] == "table":
        return dict(cos=cos, sin=sin)
    x = s["x"].float()
    if c["mode"] == "sum":
        x = x.sum(1, keepdim=True)
    cos, sin = cos[:, None], sin[:, None]
    h = Dr // 2
    lo, hi = x[..., c["Dn"]:c["Dn"] + h], x[..., c["Dn"] + h:]
    if c["mode"] == "apply":
        a, b = lo * cos[..., :h] - hi * sin[..., :h], hi * cos[..., h:] + lo * sin[..., h:]
    else:
        a, b = lo * cos[..., :h] + hi * sin[..., h:], hi * cos[..., h:] - lo * sin[..., :h]
    return dict(x=torch.cat([x[..., :c["Dn"]], a, b], -1).to(s["x"].dtype))


def _random16(total, seed, which):
    """16 random bits for each place of the flat buffers: a multiplicative mix of the place and the seed in 32 bits;
    which 0, 1: the two halves of the first mix, 2: the upper half of a second."""
    M = 0xFFFFFFFF
    x = (torch.arange(total, device=DEV, dtype=torch.int64) * 0x9E3779B1 + seed) & M
    x = ((x ^ (x >> 15)) * 0x6A09E667) & M
    x = ((x ^ (x >> 13)) * 0xBB67AE85) & M
    x = x ^ (x >> 16)
    if which == 2:
        x = (x * 0x3C6EF373) & M
    return x & 0xFFFF if which == 1 else x >> 16


def _encode(v, rnd, keep=False):
    """E4M3 codes and one E8M0 scale for each 32 values: the smallest exponent e with amax <= 448 * 2^e; a code is v *
    2^-e rounded to nearest even, or (rnd: 16 random bits a value) up where its fraction is above rnd / 65536. keep: a
    value above zero never gets code 0."""
    b = v.reshape(-1, 32)
    amax = b.abs().amax(1)
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = (ex - 9 + (mant > 0.875)).clamp(-127, 127)
    e = torch.where(amax < 2.0 ** -126, torch.full_like(e, -127), e)
    s = torch.ldexp(b, -e[:, None])
    _, k = torch.frexp(s)
    one = torch.ldexp(torch.ones_like(s), (k - 1).clamp(min=-6) - 3)  # the E4M3 step at s
    a = s.abs() / one
    if rnd is None:
        n = torch.round(a)
    else:
        n = torch.floor(a)
        n = n + (a - n > rnd.reshape(-1, 32).to(a.dtype) * 2.0 ** -16)
    if keep:
        n = torch.where((a > 0) & (n == 0), torch.ones_like(n), n)
    q = torch.copysign(n * one, s).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(-1), (e + 127).to(torch.uint8)


def _decode(codes, scales, wide):
    e = scales.to(torch.int32) - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).to(wide).reshape(-1, 32), e[:, None]).reshape(-1)


def _f32(v):
    """A host number as the kernels get it: rounded to 32 bits."""
    return float(torch.tensor(v, dtype=torch.float64).float())


def _adamw(s, wide):
    """New (master, p, m, v, ms, vs) of one step; the moments in 8 bits are m and the root of v."""
    c = s["case"]
    b1, b2 = s["betas"]
    lr, wd, t = s["lr"], s["wd"], s["step"]
    size, root = _f32(lr / (1 - b1 ** t)), _f32((1 - b2 ** t) ** -0.5)
    total = s["p"].numel()
    g = s["g"].to(wide) * s["grad_scale"].to(wide)
    p = (s["master"] if c["master"] else s["p"]).to(wide)
    if c["bits"] == 32:
        m, v = s["m"].to(wide), s["v"].to(wide)
    else:
        m, r = _decode(s["m"], s["ms"], wide), _decode(s["v"], s["vs"], wide)
        v = r * r
    p = p * _f32(1 - lr * wd)
    m = m * _f32(b1) + g * _f32(1 - b1)
    v = v * _f32(b2) + (g * _f32(1 - b2)) * g
    r = torch.sqrt(v)
    p = p - (m / (r * root + _f32(s["eps"]))) * size
    master = p if c["master"] else None
    if s["seed"] is not None and c["param"] == "bf16" and not c["master"]:
        bits = p.float().view(torch.int32)
        bits = bits + _random16(total, s["seed"], 2).to(torch.int32)
        p = torch.where(torch.isfinite(p), (bits & -65536).view(torch.float32), p.float())
    if c["bits"] == 32:
        return master, p, m, v, None, None
    rnd = (lambda k: None if s["seed"] is None else _random16(total, s["seed"], k))
    m, ms = _encode(m, rnd(0))
    v, vs = _encode(r, rnd(1), keep=True)
    return master, p, m, v, ms, vs


def _adamw_out(s):
    names = ["p", "master", "m", "v"]
    if s["case"]["bits"] == 32:
        return {k: s[k] for k in names if s[k] is not None}
    out = {k: s[k] for k in names[:2] if s[k] is not None}
    # the moments are E4M3 values and E8M0 scales: returned as those types
    out.update({k: s[k].view(torch.float8_e4m3fn) for k in ("m", "v")})
    out.update({k: s[k].view(torch.float8_e8m0fnu) for k in ("ms", "vs")})
    return out


# ------------------------------------------------------------------- passes
def _run_own(s):
    import up_proj_gemm_gb300 as mlaq

    c = s["case"]
    op = c["op"]
    if op == "ffn_fwd":
        r = mlaq.gated_ffn_fwd(s["x"], s["w_gate_up"], s["w_down"], act=c["act"], save=c["save"])
        return dict(y=r[0], gate_up=r[1], h=r[2]) if c["save"] else dict(y=r)
    if op == "ffn_bwd":
        dx, dwgu, dwd = mlaq.gated_ffn_bwd(s["dy"], s["x"], s["w_gate_up"], s["w_down"], s["gate_up"], s["h"],
                                           act=c["act"])
        return dict(dx=dx, dw_gate_up=dwgu, dw_down=dwd)
    if op == "rope":
        if c["mode"] == "table":
            cos, sin = mlaq.rope_axes_table(s["cos"], s["sin"], s["pos"], s["axes"], c["Dr"])
            return dict(cos=cos, sin=sin)
        return dict(x=mlaq.rope_axes(s["x"], s["cos"], s["sin"], s["pos"], s["axes"], c["Dr"],
                                     inverse=c["mode"] != "apply", sum_heads=c["mode"] == "sum"))
    mlaq.adamw_step(s["plan"], s["step"], lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=s["wd"],
                    grad_scale=s["grad_scale"], seed=s["seed"])
    return _adamw_out(s)


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "ffn_fwd":
        return _ffn_fwd(state, torch.float32, torch.bfloat16)
    if c["op"] == "ffn_bwd":
        return _ffn_bwd(state, torch.float32, torch.bfloat16)
    if c["op"] == "rope":
        return _rope(state)
    master, p, m, v, ms, vs = _adamw(state, torch.float32)
    state["p"].copy_(p)
    if master is not None:
        state["master"].copy_(master)
    state["m"].copy_(m)
    state["v"].copy_(v)
    if ms is not None:
        state["ms"].copy_(ms)
        state["vs"].copy_(vs)
    return _adamw_out(state)


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"].startswith("ffn"):
        F = case["F"]
        if work(case)["flops"] > 4e12:
            return None
        W, Wd, x = s["w_gate_up"].to(f64), s["w_down"].to(f64), s["x"].to(f64)

        def act(z):
            if case["act"] == "silu":
                return z * torch.sigmoid(z)
            return torch.nn.functional.gelu(z, approximate="none" if case["act"] == "gelu" else "tanh")

        if case["op"] == "ffn_fwd":
            g, u = x @ W[:F].t(), x @ W[F:].t()
            h = act(g).mul_(u)
            y = h @ Wd.t()
            return dict(y=y, gate_up=torch.cat([g, u], 1), h=h) if case["save"] else dict(y=y)
        dy = s["dy"].to(f64)
        dh = dy @ Wd
        g, u = s["gate_up"].to(f64).split(F, 1)
        leaf = g.clone().requires_grad_()
        with torch.enable_grad():
            (dact,) = torch.autograd.grad(act(leaf).sum(), leaf)
        dg, du = dh * u * dact, dh * act(g)
        return dict(dx=dg @ W[:F] + du @ W[F:], dw_gate_up=torch.cat([dg.t() @ x, du.t() @ x]),
                    dw_down=dy.t() @ s["h"].to(f64))
    if case["op"] == "rope":
        if case["mode"] == "table":
            return None  # a copy of table entries
        T, Dn, Dr = case["T"], case["Dn"], case["Dr"]
        h = Dr // 2
        x = s["x"].to(f64)
        if case["mode"] == "sum":
            x = x.sum(1, keepdim=True)
        y = x.clone()
        for i, a in enumerate(s["axes"]):
            p = s["pos"][a].long()
            c0, s0, c1, s1 = (t[p, j].to(f64)[:, None] for j in (i, i + h) for t in (s["cos"], s["sin"]))
            u, w = x[..., Dn + i], x[..., Dn + h + i]
            if case["mode"] == "apply":
                y[..., Dn + i], y[..., Dn + h + i] = u * c0 - w * s0, w * c1 + u * s1
            else:
                y[..., Dn + i], y[..., Dn + h + i] = u * c0 + w * s1, w * c1 - u * s0
        return dict(x=y)
    if sum(_sizes(case)[0]) > 150_000_000:
        return None
    b1, b2 = s["betas"]
    g = s["g"].to(f64) * s["grad_scale"].to(f64)
    p = (s["master"] if case["master"] else s["p"]).to(f64)
    if case["bits"] == 32:
        m, v = s["m"].to(f64), s["v"].to(f64)
    else:
        m, v = _decode(s["m"], s["ms"], f64), _decode(s["v"], s["vs"], f64).square()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    mhat, vhat = m / (1 - b1 ** s["step"]), v / (1 - b2 ** s["step"])
    p = p - s["lr"] * s["wd"] * p - s["lr"] * mhat / (vhat.sqrt() + s["eps"])
    # moments in 8 bits have no value in 64 bits to be near to: their rounding is a choice between two neighbours
    out = dict(m=m, v=v) if case["bits"] == 32 else dict(m=None, v=None, ms=None, vs=None)
    if case["master"]:
        out["master"] = p
    # and so for a parameter rounded up or down at random
    out["p"] = None if s["seed"] is not None and case["param"] == "bf16" and not case["master"] else p
    return out
