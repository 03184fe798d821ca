"""Workloads of the operators around a cached attention layer: the RMS norm in
front of the projections (with the residual's addition, an MXFP8 output and
its gradient), the 8-bit cache of keys and values (written as it grows, read
back) and the attention over that cache, each with its plain form in
elementary torch operations.

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
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the norm of one generated token's query latent, quantized for the MXFP8 up-projection
        dict(name="norm_token", op="norm", T=1, K=1536, x="bf16", w="bf16", residual=False, out="mxfp8", pitch=576,
             save=False),
        # a ragged prompt's query latents, a slice of the joint down-projection, as the up-projection's tiled operands
        dict(name="norm_mxfp8_ragged", op="norm", T=4099, K=1536, x="bf16", w="bf16", residual=False, out="tiled",
             pitch=576, save=True),
        # the residual stream of a training micro-batch
        dict(name="norm_residual_train", op="norm", T=8192, K=7168, x="bf16", w="fp32", residual=True, out="same",
             pitch=0, save=True),
        # the gradient at a short odd width in 32 bits
        dict(name="norm_grad_ragged", op="norm_grad", T=777, K=1001, x="fp32", w="fp32", residual=False, pitch=3),
        # the gradient of a training micro-batch's residual stream
        dict(name="norm_grad_train", op="norm_grad", T=8192, K=7168, x="bf16", w="fp32", residual=True, pitch=0),
        # a decode batch appends a token to every sequence
        dict(name="write_decode", op="write", B=64, new=1, ctx=2048, H=8, Dk=128, Dv=128, shared=False, page=64,
             block=32, sizes=1),
        # ragged prompts of 128 heads, the projection's keys and values, from empty
        dict(name="write_prompt", op="write", B=5, new=1000, ctx=0, H=128, Dk=192, Dv=128, shared=False, page=64,
             block=16, sizes=2),
        # latents and rotary keys read back for a prompt's expanded form
        dict(name="read_latent", op="read", B=7, new=4096, ctx=300, H=1, Dk=576, Dv=512, shared=True, page=64, block=64,
             sizes=3),
        # one generated token of one sequence
        dict(name="attn_token", op="attn", B=1, new=1, ctx=1100, Hq=32, H=8, Dk=128, Dv=128, shared=False, page=16,
             block=16, sizes=4),
        # a ragged decode batch of grouped heads
        dict(name="attn_decode", op="attn", B=64, new=1, ctx=8192, Hq=64, H=8, Dk=128, Dv=128, shared=False, page=64,
             block=32, sizes=5),
        # a decode batch over latents: 128 query heads share one cached row, whose first channels are the values
        dict(name="attn_latent", op="attn", B=48, new=1, ctx=4096, Hq=128, H=1, Dk=576, Dv=512, shared=True, page=64,
             block=64, sizes=6),
        # a prompt's chunk of 128 heads over what is cached of it
        dict(name="attn_chunk", op="attn", B=1, new=2048, ctx=4096, Hq=128, H=128, Dk=192, Dv=128, shared=False,
             page=128, block=32, sizes=7),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "write", "read", "attn", "attn"])
    if op.startswith("norm"):
        c = dict(op=op, x=rng.choice(["bf16", "bf16", "fp32"]), w=rng.choice(["bf16", "fp32"]),
                 residual=rng.random() < 0.5, pitch=rng.choice([0, 0, 8, 576, 5]))
        if op == "norm":
            c["out"] = rng.choice(["same", "same", "mxfp8", "tiled"])
            c["save"] = rng.random() < 0.5
        step = 32 if c.get("out", "same") != "same" else rng.choice([1, 8, 128])
        while True:
            c["T"], c["K"] = _log_int(rng, 1, 32768), _log_int(rng, 64, 16384, step)
            if c["T"] * c["K"] * (2 if c["x"] == "fp32" else 1) <= 8192 * 7168:
                return c
    while True:
        c = dict(op=op, sizes=rng.randrange(1 << 20), page=rng.choice([16, 32, 64, 128, 256]))
        c["block"] = rng.choice([b for b in (1, 8, 16, 32, 64, 128) if b <= c["page"]])
        c["shared"] = rng.random() < 0.25
        if c["shared"]:
            c["H"], (c["Dk"], c["Dv"]) = 1, rng.choice([(576, 512), (320, 256), (288, 256)])
        else:
            c["H"] = _log_int(rng, 1, 128)
            c["Dk"], c["Dv"] = rng.choice([(64, 64), (80, 80), (96, 96), (128, 128), (192, 128), (256, 256), (48, 112)])
        if op == "attn":
            c["Hq"] = c["H"] * (_log_int(rng, 8, 128) if c["shared"] else rng.choice([1, 2, 3, 4, 5, 7, 8, 16]))
            kind = rng.choice(["token", "token", "draft", "chunk"])
            c["new"] = {"token": 1, "draft": rng.randint(2, 8), "chunk": _log_int(rng, 16, 2048)}[kind]
            c["B"] = _log_int(rng, 1, 4 if kind == "chunk" else 128)
            c["ctx"] = _log_int(rng, 1, 32768)
            n, start = _sizes(c)
            far = max(a + b for a, b in zip(n, start))
            if (c["Hq"] <= 128 and work(c)["flops"] <= 8e11 and work(c)["bytes"] <= 6e8
                    and c["B"] * far * c["H"] * (c["Dk"] + c["Dv"]) <= 1.5e9 and c["B"] * c["Hq"] * max(n) * far <= 1.4e9):
                return c
        else:
            c["new"] = rng.choice([1, 1, _log_int(rng, 2, 8), _log_int(rng, 16, 8192)])
            c["B"] = _log_int(rng, 1, 256 if c["new"] < 16 else 16)
            c["ctx"] = rng.choice([0, _log_int(rng, 1, 8192)])
            row = c["H"] * (c["Dk"] + (0 if c["shared"] else c["Dv"]))
            if sum(map(sum, _sizes(c))) * row <= 6e8 and sum(_sizes(c)[0]) * row <= 1.4e8:
                return c


def _sizes(case):
    """(new tokens, tokens already cached) of every sequence: a batch's first sequence has the most, the others are
    spread below it; a longer batch has one that brings nothing."""
    rng = random.Random(case["sizes"])
    B, new, ctx = case["B"], case["new"], case["ctx"]
    n = [new if new == 1 or b == 0 else rng.randint(max(1, new // 4), new) for b in range(B)]
    start = [ctx if b == 0 else rng.randint(ctx // 8, ctx) for b in range(B)]
    if B > 4 and new > 1:
        n[B // 2] = 0
    return n, start


def _bytes(kind):
    return 4 if kind == "fp32" else 2


def work(case):
    op = case["op"]
    if op == "norm":
        T, K, e = case["T"], case["K"], _bytes(case["x"])
        out = T * K * e if case["out"] == "same" else T * K + T * K // 32
        return {"bytes": T * K * e * (3 if case["residual"] else 1) + out + K * _bytes(case["w"]) + (4 * T if case["save"] else 0),
                "flops": (5 if case["residual"] else 4) * T * K}
    if op == "norm_grad":
        T, K, e = case["T"], case["K"], _bytes(case["x"])
        return {"bytes": T * K * e * (4 if case["residual"] else 3) + 2 * K * _bytes(case["w"]) + 4 * T, "flops": 9 * T * K}
    n, start = _sizes(case)
    row = case["H"] * (case["Dk"] + (0 if case["shared"] else case["Dv"]))
    marks = case["H"] * (1 if case["shared"] else 2)
    block = case["block"]
    if op in ("write", "read"):
        blocks = sum((s + k - 1) // block - s // block + 1 for k, s in zip(n, start) if k)
        return {"bytes": 3 * sum(n) * row + blocks * marks, "flops": 2 * sum(n) * row}
    cached = [s + k for k, s in zip(n, start) if k]
    pairs = sum(k * s + k * (k + 1) // 2 for k, s in zip(n, start))
    return {"bytes": sum(cached) * row + sum(-(-t // block) for t in cached) * marks
            + 2 * sum(n) * case["Hq"] * (case["Dk"] + case["Dv"]) + 4 * sum(n) * case["Hq"],
            "flops": 2 * pairs * case["Hq"] * (case["Dk"] + case["Dv"])}


# ------------------------------------------------------------------ inputs
def _pages(case):
    """Pages of every sequence and of the cache (a few of which nobody has)."""
    per = [-(-(a + b) // case["page"]) for a, b in zip(*_sizes(case))]
    return per, sum(per) + 3


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case=case)
    types = {"bf16": torch.bfloat16, "fp32": torch.float32}
    if case["op"].startswith("norm"):
        T, K, x = case["T"], case["K"], types[case["x"]]
        s["w"] = (1.0 + normal(K, std=0.1, dtype=torch.float32)).to(types[case["w"]])
        spread = torch.exp(normal(T, 1, std=0.5, dtype=torch.float32))  # tokens of different size
        first = normal(T, K + case["pitch"], dtype=torch.float32) * spread
        if case["op"] == "norm":
            s["x"] = first.to(x)[:, :K]
            s["residual"] = normal(T, K, std=2.0, dtype=x) if case["residual"] else None
        else:
            s["h"] = first[:, :K].to(x).contiguous()
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dy"] = normal(T, K + case["pitch"], std=0.01, dtype=x)[:, :K]
            s["dres"] = normal(T, K, std=0.01, dtype=x) if case["residual"] else None
        return s
    n, start = _sizes(case)
    B, H, Dk, Dv, page, block = (case[k] for k in ("B", "H", "Dk", "Dv", "page", "block"))
    per, pages = _pages(case)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at, rows = 0, []
    for k in per:  # a sequence's pages lie anywhere; the table's rows end in entries that nothing reads
        rows.append(torch.cat([order[at:at + k], torch.full((max(per) + 1 - k,), -1, dtype=torch.int32, device=DEV)]))
        at += k
    s["table"] = torch.stack(rows).contiguous()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s["n"], s["start"], s["tokens"] = n, start, sum(n)
    s["start_d"], s["length_d"] = ints(start), ints([a + b for a, b in zip(n, start)])
    s["cu"] = None if all(k == 1 for k in n) else ints([sum(n[:b]) for b in range(B + 1)])
    s["row_seq"] = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(n, device=DEV), output_size=sum(n))
    s["row_new"] = torch.arange(sum(n), device=DEV) - torch.tensor([sum(n[:b]) for b in range(B)], device=DEV)[s["row_seq"]]

    if case["op"] == "write":  # older tokens in the block that a sequence's first new token falls into
        part = [(b, t) for b in range(B) if n[b] for t in range(start[b] // block * block, start[b])]
        s["old_seq"], s["old_at"] = (torch.tensor([x[i] for x in part], dtype=torch.int64, device=DEV) for i in (0, 1))

    def codes(D):  # what normal values are held as: scales one below or above the usual one
        c = torch.empty((pages, H, page, D), dtype=torch.uint8, device=DEV)
        for p in range(0, pages, 256):
            v = torch.randn((min(256, pages - p), H, page, D), generator=g, device=DEV) * 96.0
            c[p:p + 256] = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return c, torch.randint(120, 122, (pages, H, page // block), generator=g, device=DEV, dtype=torch.uint8)

    s["k"], s["ks"] = codes(Dk)
    s["v"], s["vs"] = (None, None) if case["shared"] else codes(Dv)
    if case["op"] == "attn":
        s["q"] = normal(sum(n), case["Hq"], Dk)
        s["scale"] = Dk ** -0.5
    elif case["op"] == "write":
        s["new_k"] = normal(sum(n), H, Dk)
        s["new_v"] = None if case["shared"] else normal(sum(n), H, Dv, std=0.7)
    if own:
        import up_proj_gemm_gb300 as mlaq

        s["cache"] = mlaq.KvCache(s["k"], s["ks"], s["v"], s["vs"], Dv=Dv)
    return s


# ------------------------------------------------------------- plain forms
def _held(codes, marks):
    """Codes and scale bytes as torch's types of 8 bits: the values that they stand for."""
    return codes.view(torch.float8_e4m3fn), marks.view(torch.float8_e8m0fnu)


def _e4m3(v):
    """E4M3 codes of values within its range, to nearest even."""
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def _exponent(amax):
    """The smallest e in -127..127 with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    mant, ex = torch.frexp(amax)
    e = (ex - 9 + (mant > 0.875)).clamp(-127, 127)
    return torch.where(amax < 2.0 ** -126, torch.full_like(e, -127), e)


def _tile(marks):
    """Scales [T, C] as 128 x 4 tiles, each in the block-scaled product's order, padded with zeros."""
    T, C = marks.shape
    t, c = -(-T // 128), -(-C // 4)
    full = torch.zeros((t * 128, c * 4), dtype=torch.uint8, device=marks.device)
    full[:T, :C] = marks
    return full.view(t, 4, 32, c, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _norm(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    wide = h.double() if c["out"] != "same" else h  # a value beside a border of its code
    rstd = torch.rsqrt(wide.square().mean(1, keepdim=True) + EPS)
    y = wide * rstd * s["w"].to(wide.dtype)
    r = {}
    if c["out"] == "same":
        r["y"] = y.to(s["x"].dtype)
    else:
        b = y.view(T, K // 32, 32)
        e = _exponent(b.abs().amax(2).float())
        marks = (e + 127).to(torch.uint8)
        r["y"], r["scales"] = _held(_e4m3(torch.ldexp(b, -e[..., None]).float()).view(T, K),
                                    marks if c["out"] == "mxfp8" else _tile(marks))
    if s["residual"] is not None:
        r["h"] = h.to(s["x"].dtype)
    if c["save"]:
        r["rstd"] = rstd[:, 0].float()
    return r


def _norm_grad(s):
    hhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - hhat * (g * hhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["h"].dtype), dw=(dy.double() * hhat.double()).sum(0).to(s["w"].dtype))


def _places(s, seq, t):
    """Page of the cache and place in it of the sequences' positions t."""
    page = s["case"]["page"]
    return s["table"].long()[seq, t // page], t % page


def _write_plain(s, codes, marks, new):
    P, H, page, D = codes.shape
    block, per = s["case"]["block"], marks.shape[2]
    where, place = _places(s, s["row_seq"], s["start_d"].long()[s["row_seq"]] + s["row_new"])
    v = new.float()
    amax = torch.zeros((P * per, H), device=DEV).index_reduce_(0, where * per + place // block, v.abs().amax(2), "amax")
    e = _exponent(amax)
    # older tokens of a block that grows: its exponent never falls, and they follow it
    w0, p0 = _places(s, s["old_seq"], s["old_at"])
    e0 = marks[w0, :, p0 // block].to(torch.int32) - 127
    floor = torch.full_like(e, -127)
    floor[w0 * per + p0 // block] = e0
    e = torch.maximum(e, floor)
    held = torch.ldexp(codes[w0, :, p0].view(torch.float8_e4m3fn).float(), (e0 - e[w0 * per + p0 // block])[..., None])
    codes[w0, :, p0] = _e4m3(held)
    codes[where, :, place] = _e4m3(torch.ldexp(v, -e[where * per + place // block][..., None]))
    marks[where, :, place // block] = (e[where * per + place // block] + 127).to(torch.uint8)


def _read_plain(s, codes, marks, seq, t, wide=torch.float32):
    where, place = _places(s, seq, t)
    e = marks[where, :, place // s["case"]["block"]].to(torch.int32) - 127
    return torch.ldexp(codes[where, :, place].view(torch.float8_e4m3fn).to(wide), e[..., None])


def _padded(s):
    """Every sequence's positions up to the furthest [B, L], and which of them it has."""
    far = max(a + b for a, b in zip(s["n"], s["start"]))
    t = torch.arange(far, device=DEV)[None].expand(s["case"]["B"], -1)
    have = t < s["length_d"][:, None]
    seq = torch.arange(s["case"]["B"], device=DEV)[:, None]
    return seq, torch.where(have, t, torch.zeros_like(t)), t


def _attn_plain(s):
    c = s["case"]
    B, Hq, H, Dk, Dv, most = c["B"], c["Hq"], c["H"], c["Dk"], c["Dv"], max(s["n"])
    seq, at, t = _padded(s)
    k = _read_plain(s, s["k"], s["ks"], seq, at).permute(0, 2, 1, 3)  # [B, H, L, Dk]
    v = k[..., :Dv] if c["shared"] else _read_plain(s, s["v"], s["vs"], seq, at).permute(0, 2, 1, 3)
    q = torch.zeros((B, most, Hq, Dk), device=DEV)
    q[s["row_seq"], s["row_new"]] = s["q"].float()
    q = q.view(B, most, H, Hq // H, Dk).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * most, Dk)
    p = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, H, Hq // H, most, -1)
    last = s["start_d"][:, None] + torch.arange(most, device=DEV)  # the last position that a new token sees
    p.masked_fill_((t[:, None] > last[..., None])[:, None, None], -math.inf)
    top = p.amax(4, keepdim=True)
    p = p.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    o = (p.view(B, H, Hq // H * most, -1) @ v).view(B, H, Hq // H, most, Dv) / total
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, Dv)[s["row_seq"], s["row_new"]]
    lse = lse.permute(0, 3, 1, 2).reshape(B, most, Hq)[s["row_seq"], s["row_new"]]
    return dict(out=o.to(torch.bfloat16), lse=lse)


def _written(s):
    r = dict(zip(("k", "k_scales"), _held(s["k"], s["ks"])))
    if s["v"] is not None:
        r.update(zip(("v", "v_scales"), _held(s["v"], s["vs"])))
    return r


# ------------------------------------------------------------------- passes
def _run_own(s):
    import up_proj_gemm_gb300 as mlaq

    c = s["case"]
    if c["op"] == "norm":
        got = mlaq.rms_norm_fwd(s["x"], s["w"], eps=EPS, residual=s["residual"], out=c["out"], save=c["save"])
        names = ["y"] if c["out"] == "same" else ["y", "scales"]
        names += (["h"] if c["residual"] else []) + (["rstd"] if c["save"] else [])
        r = dict(zip(names, got if len(names) > 1 else (got,)))
        if c["out"] != "same":
            r["y"], r["scales"] = _held(r["y"], r["scales"])
        return r
    if c["op"] == "norm_grad":
        return dict(zip(("dx", "dw"), mlaq.rms_norm_bwd(s["dy"], s["h"], s["w"], s["rstd"], dres=s["dres"])))
    if c["op"] == "write":
        mlaq.kv_cache_write(s["cache"], s["new_k"], s["new_v"], s["table"], s["start_d"], cu=s["cu"])
        return _written(s)
    if c["op"] == "read":
        k, v = mlaq.kv_cache_read(s["cache"], s["table"], s["start_d"], s["tokens"], cu=s["cu"])
        return dict(k=k) if v is None else dict(k=k, v=v)
    out, lse = mlaq.cache_attn(s["q"], s["cache"], s["table"], s["length_d"], cu=s["cu"], scale=s["scale"], lse=True)
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["case"]["op"]
    if op == "norm":
        return _norm(s)
    if op == "norm_grad":
        return _norm_grad(s)
    if op == "write":
        _write_plain(s, s["k"], s["ks"], s["new_k"])
        if s["v"] is not None:
            _write_plain(s, s["v"], s["vs"], s["new_v"])
        return _written(s)
    if op == "read":
        t = s["start_d"].long()[s["row_seq"]] + s["row_new"]
        r = dict(k=_read_plain(s, s["k"], s["ks"], s["row_seq"], t).to(torch.bfloat16))
        if s["v"] is not None:
            r["v"] = _read_plain(s, s["v"], s["vs"], s["row_seq"], t).to(torch.bfloat16)
        return r
    return _attn_plain(s)


# ------------------------------------------------- the definitions in 64 bits
def _two(e):
    """2^e of whole numbers e, exactly."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e.to(torch.int32))


def _low(a):
    """The exponent of the largest power of two that is not above a > 0."""
    e = torch.floor(torch.log2(a))
    e = torch.where(_two(e) > a, e - 1, e)
    return torch.where(_two(e + 1) <= a, e + 1, e)


def _steps(v):
    """v rounded to the E4M3 grid: steps of 2^-3 of the value's power of two, of 2^-9 below 2^-6."""
    one = _two(_low(v.abs().clamp(min=2.0 ** -6)) - 3)
    return torch.round(v / one) * one


def _power(amax):
    """log2 of a block's scale: the smallest with amax within 448 of them."""
    e = _low(amax.clamp(min=2.0 ** -127)) - 8
    return torch.where(amax > 448 * _two(e), e + 1, e).clamp(min=-127)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "norm":
        T, K = case["T"], case["K"]
        h = s["x"].to(f64) + (0 if s["residual"] is None else s["residual"].to(f64))
        var = torch.linalg.vector_norm(h, dim=1) ** 2 / K + EPS
        y = h / var.sqrt()[:, None] * s["w"].to(f64)
        r = dict(y=y)
        if case["out"] != "same":
            b = y.view(T, -1, 32)
            e = _power(b.abs().max(2).values)
            r["y"] = (_steps(b / _two(e)[..., None])).view(T, K)
            r["scales"] = _two(e)
            if case["out"] == "tiled":
                C = K // 32
                full = torch.full((-(-T // 128) * -(-C // 4) * 512,), 2.0 ** -127, dtype=f64, device=DEV)
                i, j = torch.arange(T, device=DEV)[:, None], torch.arange(C, device=DEV)[None]
                at = ((i // 128) * -(-C // 4) + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4
                full[at.reshape(-1)] = r["scales"].reshape(-1)
                r["scales"] = full
        if s["residual"] is not None:
            r["h"] = h
        if case["save"]:
            r["rstd"] = var.rsqrt()
        return r
    if op == "norm_grad":
        leaf = s["h"].to(f64).requires_grad_()
        w = s["w"].to(f64).requires_grad_()
        # rstd is given: its gradient is the formula's, at the value that the forward kept
        r = s["rstd"].to(f64)[:, None]
        with torch.enable_grad():
            mean = (leaf * leaf).mean(1, keepdim=True)
            y = leaf * (r - 0.5 * r ** 3 * (mean - mean.detach())) * w
            dx, dw = torch.autograd.grad(y, (leaf, w), s["dy"].to(f64))
        return dict(dx=dx if s["dres"] is None else dx + s["dres"].to(f64), dw=dw)
    if op == "read":
        return None  # codes times powers of two: nothing is rounded
    if op == "write":
        if s["k"].numel() > 1_200_000_000 // (1 if s["v"] is None else 2):
            return None
        r = {}
        for name, codes, marks, new in (("k", s["k"], s["ks"], s["new_k"]), ("v", s["v"], s["vs"], s["new_v"])):
            if codes is None:
                continue
            block = case["block"]
            out, scale = codes.view(torch.float8_e4m3fn).to(f64), _two(marks.to(torch.int32) - 127)
            seen = 0
            for b in range(case["B"]):
                lo, hi = s["start"][b], s["start"][b] + s["n"][b]
                if hi == lo:
                    continue
                t = torch.arange(lo // block * block, hi, device=DEV)
                page, place = s["table"][b].long()[t // case["page"]], t % case["page"]
                old = t < lo
                value = torch.zeros((len(t), case["H"], codes.shape[3]), dtype=f64, device=DEV)
                value[lo - lo // block * block:] = new[seen:seen + hi - lo].to(f64)
                seen += hi - lo
                amax = torch.zeros((-(-len(t) // block) * block, case["H"]), dtype=f64, device=DEV)
                amax[:len(t)] = value.abs().amax(2)
                e = _power(amax.view(-1, block, case["H"]).amax(1))
                before = scale[page, :, place // block]
                value = torch.where(old[:, None, None], out[page, :, place] * before[..., None], value)
                if lo % block:
                    e[0] = torch.maximum(e[0], _low(before[0]))
                each = _two(e).repeat_interleave(block, 0)[:len(t)]
                out[page, :, place] = _steps(value / each[..., None])
                scale[page, :, place // block] = each
            r[name], r[name + "_scales"] = out, scale
        return r
    if work(case)["flops"] > 1.5e12 or work(case)["bytes"] > 4e9:
        return None
    o = torch.empty((s["tokens"], case["Hq"], case["Dv"]), dtype=f64, device=DEV)
    lse = torch.empty((s["tokens"], case["Hq"]), dtype=f64, device=DEV)
    group, seen = case["Hq"] // case["H"], 0
    for b in range(case["B"]):
        n, start = s["n"][b], s["start"][b]
        if n == 0:
            continue
        t = torch.arange(start + n, device=DEV)
        page, place = s["table"][b].long()[t // case["page"]], t % case["page"]

        def values(codes, marks):
            return codes[page, :, place].view(torch.float8_e4m3fn).to(f64) * _two(marks[page, :, place // case["block"]].to(torch.int32) - 127)[..., None]

        k = values(s["k"], s["ks"])
        v = k[..., :case["Dv"]] if case["shared"] else values(s["v"], s["vs"])
        hidden = t[None] > start + torch.arange(n, device=DEV)[:, None]
        step = max(1, 250_000_000 // (group * n * len(t)))  # heads of keys at once
        for h in range(0, case["H"], step):
            part = slice(h * group, min(case["H"], h + step) * group)
            q = s["q"][seen:seen + n, part].to(f64).unflatten(1, (-1, group))
            z = torch.einsum("nhgd,thd->hgnt", q, k[:, h:h + step]) * s["scale"]
            z = z.masked_fill(hidden, -math.inf)
            lse[seen:seen + n, part] = torch.logsumexp(z, 3).permute(2, 0, 1).flatten(1)
            o[seen:seen + n, part] = torch.einsum("hgnt,thd->nhgd", torch.softmax(z, 3), v[:, h:h + step]).flatten(1, 2)
        seen += n
    return dict(out=o, lse=lse)
