"""The gated feed-forward block, 8-bit checkpoints and 4-bit weights in 64 bits, with bounds on
how far a kernel may be off.

A bound follows the kernel's own arithmetic.  ``r`` is the storage type's unit roundoff
(half a step, relative): 2^-8 for bf16, 2^-24 for fp32.  A sum of K products in fp32 is off by at
most K * 2^-23 of the sum of their magnitudes (2^-23 per addition: the tensor cores' accumulator
may truncate), and every value stored between two products (h, dg, du) or as a result adds r of
its magnitude.  The activation functions are good to 2^-20 of max(1, |g|) times their factors.
"""
import torch

E32 = 2.0 ** -23
FN = 2.0 ** -20
SLOPE = 1.13  # the largest |act'| of SiLU (1.10) and GELU (1.13)


def roundoff(dtype):
    return torch.finfo(dtype).eps / 2


def act_and_slope(name, g):
    if name == "gelu":
        c = torch.special.ndtr(g)
        return g * c, c + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    s = torch.sigmoid(g)
    return g * s, s * (1 + g * (1 - s))


def forward(act, x, Wg, Wu, Wd, r):
    """Values and bounds {name: (value, bound)} of g, u, y from tensors of any type."""
    x, Wg, Wu, Wd = (t.double() for t in (x, Wg, Wu, Wd))
    k, f = x.shape[1], Wg.shape[0]
    g, u = x @ Wg.t(), x @ Wu.t()
    eg, eu = k * E32 * (x.abs() @ Wg.abs().t()), k * E32 * (x.abs() @ Wu.abs().t())
    a, _ = act_and_slope(act, g)
    h = a * u
    eh = SLOPE * eg * u.abs() + a.abs() * eu + SLOPE * eg * eu + (r + FN) * (h.abs() + u.abs() * FN)
    y = h @ Wd.t()
    ey = (eh + f * E32 * h.abs()) @ Wd.abs().t()
    return {"g": (g, eg + r * g.abs()), "u": (u, eu + r * u.abs()),
            "y": (y, ey * 1.01 + r * y.abs() + 1e-30)}


def backward(act, x, Wg, Wu, Wd, g, u, dy, r, r_weight=None):
    """Values and bounds of dx, dWg, dWu, dWd; g and u as the backward reads them."""
    x, Wg, Wu, Wd, g, u, dy = (t.double() for t in (x, Wg, Wu, Wd, g, u, dy))
    rw = r if r_weight is None else r_weight
    n, f = g.shape
    o = dy.shape[1]
    a, slope = act_and_slope(act, g)
    dh = dy @ Wd
    edh = o * E32 * (dy.abs() @ Wd.abs())
    fn = FN * (1 + g.abs())
    h, dg, du = a * u, dh * u * slope, dh * a
    eh = r * h.abs() + fn * u.abs()
    edg = edh * (u * slope).abs() + (r + FN) * dg.abs() + fn * (dh.abs() + edh) * u.abs()
    edu = edh * a.abs() + (r + FN) * du.abs() + fn * (dh.abs() + edh)
    dx = dg @ Wg + du @ Wu
    edx = (edg + 2 * f * E32 * dg.abs()) @ Wg.abs() + (edu + 2 * f * E32 * du.abs()) @ Wu.abs()

    def weight(p, ep, q):
        w = p.t() @ q
        return w, (ep + n * E32 * p.abs()).t() @ q.abs() * 1.01 + rw * w.abs() + 1e-30

    return {"dx": (dx, edx * 1.01 + r * dx.abs() + 1e-30), "dWg": weight(dg, edg, x),
            "dWu": weight(du, edu, x),
            "dWd": (dy.t() @ h, dy.abs().t() @ (eh + n * E32 * h.abs()) * 1.01
                    + rw * (dy.t() @ h).abs() + 1e-30)}


def check(got, want_bound, what, rms=None):
    """Every element within its bound.  ``rms``: also the 2-norm of the error within that share
    of the result's.  The roundings of a bf16 chain are independent, each at most 2^-8 of its
    value (2^-8/sqrt(3) in the mean square), so m of them in a row stay below sqrt(m) * 2^-8."""
    want, bound = want_bound
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    worst = (off / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"
    if rms is not None and want.numel() >= 256:
        rel = (off.norm() / want.norm()).item()
        assert rel <= rms, f"{what}: relative error {rel:.3g}"


# ------------------------------------------------------------------ 8-bit checkpoints
def pack8(v, run=32):
    """Codes [rows, run * runs] and scales of values that are exact in fp32.  (Dividing two fp32
    values in 64 bits and rounding gives the correctly rounded fp32 quotient; torch's own fp32
    division by a number multiplies by its reciprocal on the GPU.)"""
    n, c = v.shape
    runs = -(-c // run)
    p = torch.zeros(n, runs * run, dtype=torch.float64, device=v.device)
    p[:, :c] = v.double()
    p = p.view(n, runs, run)
    top = p.abs().amax(-1, keepdim=True)
    q = torch.where(top > 0, p * 127 / torch.where(top > 0, top, 1.0), 0.0).round()
    return q.view(n, -1).to(torch.int8), (top.squeeze(-1) / 127).float()


def unpack8(codes, scale, cols):
    return (codes.double() * scale.double().repeat_interleave(32, 1))[:, :cols]


# ------------------------------------------------------------------ 4-bit weights
def pack4(W, group):
    """Codes 0 .. 15 as integers [o, i] and bf16 scales of a bf16 matrix."""
    o, i = W.shape
    ng = -(-i // group)
    codes = torch.full((o, i), 8, dtype=torch.int64, device=W.device)
    scale = torch.zeros(o, ng, dtype=torch.bfloat16, device=W.device)
    for j in range(ng):
        part = W[:, j * group:(j + 1) * group].float()
        s = (part.abs().amax(1).double() / 7).float().to(torch.bfloat16)
        scale[:, j] = s
        q = torch.round(part / s.float()[:, None]).clamp(-8, 7)
        codes[:, j * group:(j + 1) * group] = torch.where(s[:, None] > 0, q, 0.0).long() + 8
    return codes, scale


def nibbles(packed):
    """Integers 0 .. 15 [o, i] of packed codes."""
    lo, hi = packed & 15, packed >> 4
    return torch.stack([lo, hi], -1).view(packed.shape[0], -1).long()


def values4(codes, scale, group):
    wide = scale.double().repeat_interleave(group, 1)[:, :codes.shape[1]]
    return (codes.double() - 8) * wide
