"""Measured cases of the layer's feed-forward companions: the gated feed-forward block (forward,
backward, few-token calls), 8-bit activation checkpoints and products with 4-bit weights.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where ``own`` is true, through the calls a user makes of
``product_key_memory_pkm_b200.pkm``.  ``exact`` gives the same outputs from the definition in
64 bits.
"""
import torch

own = False

CKPT = 32  # columns that share one scale in an 8-bit activation checkpoint


def listed():
    return [
        # one training step's forward beside the full-scale memory layer (batch 64 x 256 tokens,
        # width 1600, four times that inside); the two projections are kept for the backward
        dict(name="ffn fwd train 16384x1600", op="ffn_fwd", dtype="bf16", act="silu", save="plain",
             N=16384, d_in=1600, d_ff=6400, d_out=1600),
        # evaluation of a ragged batch, nothing kept; the gated width 8/3 of the model's
        dict(name="ffn fwd eval 4099x1024 gelu", op="ffn_fwd", dtype="bf16", act="gelu",
             save="none", N=4099, d_in=1024, d_ff=2728, d_out=1024),
        # the forward of a step that keeps its projections in 8 bits
        dict(name="ffn fwd ckpt8 4096x1024", op="ffn_fwd", dtype="bf16", act="silu", save="int8",
             N=4096, d_in=1024, d_ff=4096, d_out=1024),
        # one decoded token: bound by reading the three weight matrices
        dict(name="ffn decode 1x1600", op="ffn_fwd", dtype="bf16", act="silu", save="none",
             N=1, d_in=1600, d_ff=6400, d_out=1600),
        # the training step's backward: dx and the three weight gradients
        dict(name="ffn bwd train 16384x1600", op="ffn_bwd", dtype="bf16", act="silu", save="plain",
             N=16384, d_in=1600, d_ff=6400, d_out=1600),
        # the backward of a ragged batch from 8-bit checkpoints
        dict(name="ffn bwd ckpt8 4099x1024", op="ffn_bwd", dtype="bf16", act="silu", save="int8",
             N=4099, d_in=1024, d_ff=2728, d_out=1024),
        # the smallest training call, 32-bit storage: a unit test or a toy model
        dict(name="ffn bwd fp32 64x64", op="ffn_bwd", dtype="fp32", act="silu", save="plain",
             N=64, d_in=64, d_ff=256, d_out=64),
        # the block's input of a large step put into 8 bits and read back
        dict(name="ckpt8 16384x6400", op="ckpt8", dtype="bf16", rows=16384, cols=6400),
        # a ragged one in 32 bits
        dict(name="ckpt8 1003x1608 fp32", op="ckpt8", dtype="fp32", rows=1003, cols=1608),
        # one token's query projection with 4-bit weights: the smallest call
        dict(name="w4 matvec 1x1600x2048", op="w4_matvec", N=1, d_in=1600, d_out=2048, group=64),
        # a decode batch against a large matrix (a vocabulary projection)
        dict(name="w4 matvec 64x1600x50264", op="w4_matvec", N=64, d_in=1600, d_out=50264,
             group=128),
        # the whole gated block with 4-bit weights for a few sequences decoded together
        dict(name="w4 ffn 8x1600", op="w4_ffn", act="silu", N=8, d_in=1600, d_ff=6400, d_out=1600,
             group=64),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, uniform in its logarithm."""
    return int(round(lo * (hi / lo) ** rng.random()))


def _mult(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd", "ckpt8", "w4_matvec", "w4_ffn"])
    if op == "ckpt8":
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), rows=_log(rng, 1, 16384),
                    cols=_mult(_log(rng, 8, 6400), 8))
    if op == "w4_matvec":
        return dict(op=op, N=_log(rng, 1, 64), d_in=_mult(_log(rng, 64, 2048), 32),
                    d_out=_log(rng, 64, 50000), group=rng.choice([32, 64, 128]))
    act = rng.choice(["silu", "gelu"])
    if op == "w4_ffn":
        return dict(op=op, act=act, N=_log(rng, 1, 64), d_in=_mult(_log(rng, 64, 2048), 32),
                    d_ff=_mult(_log(rng, 128, 8192), 32), d_out=_log(rng, 64, 2048),
                    group=rng.choice([32, 64, 128]))
    if rng.random() < 0.15:  # 32-bit storage: small models
        d = _mult(_log(rng, 32, 256), 8)
        return dict(op=op, dtype="fp32", act=act, save="plain", N=_log(rng, 1, 512), d_in=d,
                    d_ff=_mult(_log(rng, 64, 1024), 8), d_out=d)
    d_in = _mult(_log(rng, 64, 2048), 8)
    d_ff = _mult(_log(rng, 128, 8192), 8)
    most = 16384 * 1600 * 6400 // (max(d_in, 1600) * max(d_ff, 6400))
    save = rng.choice(["plain", "int8"] if op == "ffn_bwd" else ["none", "plain", "int8"])
    return dict(op=op, dtype="bf16", act=act, save=save, N=_log(rng, 1, most), d_in=d_in,
                d_ff=d_ff, d_out=rng.choice([d_in, _mult(_log(rng, 64, 1600), 8)]))


# ------------------------------------------------------------------ inputs
def _dt(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _activations(gen, n, d, dtype):
    """Normalised activations with a few loud channels, as layers see them."""
    x = torch.randn(n, d, device="cuda", generator=gen)
    loud = 1.0 + 7.0 * (torch.rand(d, device="cuda", generator=gen) < 0.01).float()
    return (x * loud).to(dtype)


def _weight(gen, o, i, dtype):
    return (torch.randn(o, i, device="cuda", generator=gen) * i ** -0.5).to(dtype)


def _padded(v):
    """[rows][groups][32] view of v, zeros behind the last column."""
    n, c = v.shape
    g = -(-c // CKPT)
    return torch.nn.functional.pad(v, (0, g * CKPT - c)).view(n, g, CKPT)


def _quant8(v):
    """Codes [rows][32 * groups] int8 and scales [rows][groups] of fp32 values.  The quotients
    are formed in 64 bits, so that those halfway between two codes go to the even one."""
    p = _padded(v)
    top = p.abs().amax(-1)
    safe = torch.where(top > 0, top, torch.ones_like(top)).double()
    codes = torch.round(p.double() * 127.0 / safe[..., None]).to(torch.int8)
    return codes.view(v.shape[0], -1), top / 127.0


def _value8(codes, scale, cols):
    p = codes.view(scale.shape[0], scale.shape[1], CKPT).to(scale.dtype)
    return (p * scale[..., None]).view(scale.shape[0], -1)[:, :cols]


def _random_w4(gen, o, i, group):
    """4-bit weights as stored: two codes a byte (even column low), bf16 scales by group."""
    codes = torch.randint(0, 256, (o, i // 2), device="cuda", generator=gen, dtype=torch.uint8)
    ng = -(-i // group)
    scale = (0.5 + torch.rand(o, ng, device="cuda", generator=gen)) * (0.2 * i ** -0.5)
    return codes, scale.to(torch.bfloat16)


def _w4_values(codes, scale, group, dtype):
    i = 2 * codes.shape[1]
    v = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], i).to(dtype) - 8
    return v * scale.to(dtype).repeat_interleave(group, 1)[:, :i]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "ckpt8":
        s["x"] = _activations(gen, case["rows"], case["cols"], _dt(case))
    elif op == "w4_matvec":
        s["x"] = _activations(gen, case["N"], case["d_in"], torch.bfloat16)
        s["W"] = _random_w4(gen, case["d_out"], case["d_in"], case["group"])
    else:
        n, di, f, do = case["N"], case["d_in"], case["d_ff"], case["d_out"]
        s["x"] = _activations(gen, n, di, _dt(case))
        if op == "w4_ffn":
            for name, (o, i) in dict(Wg=(f, di), Wu=(f, di), Wd=(do, f)).items():
                s[name] = _random_w4(gen, o, i, case["group"])
            return s
        s["Wg"] = _weight(gen, f, di, _dt(case))
        s["Wu"] = _weight(gen, f, di, _dt(case))
        s["Wd"] = _weight(gen, do, f, _dt(case))
        if op == "ffn_bwd":  # what the forward of the step has left
            s["dy"] = torch.randn(n, do, device="cuda", generator=gen).to(_dt(case))
            g, u = (s["x"].float() @ s[w].float().t() for w in ("Wg", "Wu"))
            if case["save"] == "int8":
                s["g"], s["g_scale"] = _quant8(g)
                s["u"], s["u_scale"] = _quant8(u)
            else:
                s["g"], s["u"] = g.to(_dt(case)), u.to(_dt(case))
    return s


# ------------------------------------------------------------------ plain form
def _act(name, g):
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g / (1.0 + torch.exp(-g))


def _act_and_slope(name, g):
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) * 0.3989422804014327
    sg = 1.0 / (1.0 + torch.exp(-g))
    return g * sg, sg * (1.0 + g * (1.0 - sg))


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _dt(case)
    x = s["x"].float()
    if op == "ckpt8":
        codes, scale = _quant8(x)
        return {"values": _value8(codes, scale, case["cols"]).to(dt), "scale": scale}
    if op == "w4_matvec":
        return {"y": x @ _w4_values(*s["W"], case["group"], torch.float32).t()}
    if op == "w4_ffn":
        wg, wu, wd = (_w4_values(*s[w], case["group"], torch.float32) for w in ("Wg", "Wu", "Wd"))
        h = _act(case["act"], x @ wg.t()) * (x @ wu.t())
        return {"y": (h @ wd.t()).to(torch.bfloat16)}
    wg, wu, wd = s["Wg"].float(), s["Wu"].float(), s["Wd"].float()
    if op == "ffn_fwd":
        g, u = x @ wg.t(), x @ wu.t()
        out = {"y": ((_act(case["act"], g) * u) @ wd.t()).to(dt)}
        if case["save"] == "plain":
            out["g"], out["u"] = g.to(dt), u.to(dt)
        elif case["save"] == "int8":
            out["g"], out["u"] = (_value8(*_quant8(v), case["d_ff"]).to(dt) for v in (g, u))
        return out
    if case["save"] == "int8":
        g = _value8(s["g"], s["g_scale"], case["d_ff"])
        u = _value8(s["u"], s["u_scale"], case["d_ff"])
    else:
        g, u = s["g"].float(), s["u"].float()
    dy = s["dy"].float()
    a, slope = _act_and_slope(case["act"], g)
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    return {"dx": (dg @ wg + du @ wu).to(dt), "dWg": (dg.t() @ x).to(dt),
            "dWu": (du.t() @ x).to(dt), "dWd": (dy.t() @ (a * u)).to(dt)}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from product_key_memory_pkm_b200 import pkm as P
    case = s["case"]
    op, dt = case["op"], _dt(case)
    b = s.setdefault("buffers", {})  # a program's outputs and workspaces, allocated once
    if op == "ckpt8":
        if not b:
            b["codes"], b["scale"] = P.alloc_ckpt8(case["rows"], case["cols"])
            b["values"] = torch.empty_like(s["x"])
        P.pkm_ckpt8_pack(s["x"], b["codes"], b["scale"])
        P.pkm_ckpt8_unpack(b["codes"], b["scale"], b["values"])
        return {"values": b["values"], "scale": b["scale"]}
    if op == "w4_matvec":
        if not b:
            b["y"] = torch.empty(case["N"], case["d_out"], device="cuda")
        P.pkm_w4_matvec(s["x"], *s["W"], b["y"], group=case["group"])
        return {"y": b["y"]}
    if not b:
        flags = P.PKM_F_FP32 if dt == torch.float32 else 0
        if case.get("save") == "int8":
            flags |= P.PKM_FFN_CKPT8
        if op == "ffn_bwd" and dt == torch.bfloat16:
            flags |= P.PKM_FFN_GRAD_BF16
        act = P.PKM_ACT_GELU if case["act"] == "gelu" else P.PKM_ACT_SILU
        d = P.FfnDims(case["N"], case["d_in"], case["d_ff"], case["d_out"], act, flags)
        b["dims"] = d
        b["ws"] = P.alloc_ffn_workspace(d, P.PKM_BWD if op == "ffn_bwd" else P.PKM_FWD)
        if op == "ffn_bwd":
            b["saved"] = {k: s.get(k) for k in ("g", "u", "g_scale", "u_scale")}
            b["dx"] = torch.empty_like(s["x"])
            for w in ("Wg", "Wu", "Wd"):
                b["d" + w] = torch.empty_like(s[w])
        else:
            b["y"] = torch.empty(case["N"], case["d_out"], device="cuda", dtype=dt)
            if case.get("save", "none") != "none":
                b["saved"] = P.alloc_ffn_saved(d)
                b["g"] = torch.empty(case["N"], case["d_ff"], device="cuda", dtype=dt)
                b["u"] = torch.empty_like(b["g"])
    if op == "w4_ffn":
        P.pkm_w4_ffn(b["dims"], s["x"], s["Wg"], s["Wu"], s["Wd"], b["y"], group=case["group"],
                     workspace=b["ws"])
        return {"y": b["y"]}
    if op == "ffn_fwd":
        P.pkm_ffn_forward(b["dims"], s["x"], s["Wg"], s["Wu"], s["Wd"], b["y"],
                          saved=b.get("saved"), workspace=b["ws"])
        if case["save"] == "none":
            return {"y": b["y"]}
        if case["save"] == "plain":
            return {"y": b["y"], "g": b["saved"]["g"], "u": b["saved"]["u"]}
        for k in ("g", "u"):
            P.pkm_ckpt8_unpack(b["saved"][k], b["saved"][k + "_scale"], b[k])
        return {"y": b["y"], "g": b["g"], "u": b["u"]}
    grads = {k: b[k] for k in ("dWg", "dWu", "dWd")}
    if dt == torch.float32:  # 32-bit gradients accumulate: a step starts from zeros
        for v in grads.values():
            v.zero_()
    P.pkm_ffn_backward(b["dims"], s["x"], s["Wg"], s["Wu"], s["Wd"], b["saved"], s["dy"],
                       dx=b["dx"], workspace=b["ws"], **grads)
    return {"dx": b["dx"], **grads}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    e = 4 if case.get("dtype") == "fp32" else 2
    if op == "ckpt8":  # the pack reads the values once, the unpack writes them once
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * e * n + 2 * (n + 4 * case["rows"] * -(-case["cols"] // CKPT)),
                "flops": 4 * n}
    n, di, do = case["N"], case["d_in"], case["d_out"]

    def w4(o, i):
        return o * i / 2 + 2 * o * -(-i // case["group"])

    if op == "w4_matvec":
        return {"bytes": w4(do, di) + 2 * n * di + 4 * n * do, "flops": 2 * n * di * do}
    f = case["d_ff"]
    if op == "w4_ffn":
        return {"bytes": 2 * w4(f, di) + w4(do, f) + 2 * n * (di + do),
                "flops": 2 * n * f * (2 * di + do)}
    kept = {"none": 0, "plain": 2 * e * n * f, "int8": 2 * n * (f + 4 * -(-f // CKPT))}[case["save"]]
    weights = e * f * (2 * di + do)
    if op == "ffn_fwd":
        return {"bytes": weights + e * n * (di + do) + kept, "flops": 2 * n * f * (2 * di + do)}
    return {"bytes": 2 * weights + e * n * (2 * di + do) + kept,
            "flops": 4 * n * f * (2 * di + do)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64

    def groups(v):
        return v.split(CKPT, dim=1)

    def through8(v):
        """The values that an 8-bit checkpoint of v stands for."""
        out = []
        for part in groups(v):
            top = part.abs().max(dim=1, keepdim=True).values
            safe = torch.where(top > 0, top, torch.ones_like(top))
            out.append((part * 127 / safe).round() * (top / 127))
        return torch.cat(out, dim=1)

    def from8(codes, scale, cols):
        wide = scale.to(D).repeat_interleave(CKPT, dim=1)
        return (codes.to(D) * wide)[:, :cols]

    def from4(codes, scale):
        o, half = codes.shape
        v = torch.empty(o, 2 * half, dtype=D, device=codes.device)
        v[:, 0::2] = (codes % 16).to(D)
        v[:, 1::2] = (codes // 16).to(D)
        at = torch.arange(2 * half, device=codes.device) // case["group"]
        return (v - 8) * scale.to(D)[:, at]

    def phi(v):
        return torch.special.ndtr(v)

    def act(v):
        return v * phi(v) if case["act"] == "gelu" else v * torch.sigmoid(v)

    def slope(v):
        if case["act"] == "gelu":
            return phi(v) + v * torch.exp(-v.square() / 2) / (2 * torch.pi) ** 0.5
        p = torch.sigmoid(v)
        return p + v * p * (1 - p)

    x = s["x"].to(D)
    if op == "ckpt8":
        scale = torch.cat([p.abs().max(dim=1, keepdim=True).values / 127 for p in groups(x)], 1)
        return {"values": through8(x), "scale": scale}
    if op == "w4_matvec":
        return {"y": torch.einsum("ni,oi->no", x, from4(*s["W"]))}
    if op == "w4_ffn":
        wg, wu, wd = (from4(*s[k]) for k in ("Wg", "Wu", "Wd"))
    else:
        wg, wu, wd = (s[k].to(D) for k in ("Wg", "Wu", "Wd"))
    if op != "ffn_bwd":
        g = torch.einsum("ni,fi->nf", x, wg)
        u = torch.einsum("ni,fi->nf", x, wu)
        out = {"y": torch.einsum("nf,of->no", act(g) * u, wd)}
        if case.get("save") == "plain":
            out.update(g=g, u=u)
        elif case.get("save") == "int8":
            out.update(g=through8(g), u=through8(u))
        return out
    if case["save"] == "int8":
        g = from8(s["g"], s["g_scale"], case["d_ff"])
        u = from8(s["u"], s["u_scale"], case["d_ff"])
    else:
        g, u = s["g"].to(D), s["u"].to(D)
    dy = s["dy"].to(D)
    dh = torch.einsum("no,of->nf", dy, wd)
    dg, du = dh * u * slope(g), dh * act(g)
    return {"dx": torch.einsum("nf,fi->ni", dg, wg) + torch.einsum("nf,fi->ni", du, wu),
            "dWg": torch.einsum("nf,ni->fi", dg, x), "dWu": torch.einsum("nf,ni->fi", du, x),
            "dWd": torch.einsum("no,nf->of", dy, act(g) * u)}
