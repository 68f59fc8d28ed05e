"""The gated feed-forward block on the device against its formulas in 64 bits: every storage
type, both ways of keeping the projections, sizes around the kernels' tiles, and the calls a
training loop makes around it (streams, graphs, accumulation, several calls at once)."""
import pytest
import torch

from product_key_memory_pkm_b200 import pkm as P

from . import ffn_ref as R

pytestmark = pytest.mark.gpu

ACT = {"silu": P.PKM_ACT_SILU, "gelu": P.PKM_ACT_GELU}
TWO = 2 ** 0.5 * 2 ** -8  # two independent bf16 roundings on the way (ffn_ref.check)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from product_key_memory_pkm_b200 import build as B
    B.build()


def guarded(n, d, dtype, fill=7.0):
    """An [n, d] tensor that is followed in memory by two rows of `fill`."""
    t = torch.full((n + 2, d), fill, dtype=dtype, device="cuda")
    return t, t[:n]


def scratch(d, which):
    """A workspace of exactly the stated size, filled with NaN patterns."""
    return torch.full((max(P.pkm_ffn_workspace_bytes(d, which), 1),), 255, dtype=torch.uint8,
                      device="cuda")


def make(n, di, f, do, dtype, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda a, b, s: (torch.randn(a, b, device="cuda", generator=gen) * s).to(dtype)  # noqa: E731
    return dict(x=mk(n, di, scale), Wg=mk(f, di, di ** -0.5), Wu=mk(f, di, di ** -0.5),
                Wd=mk(do, f, f ** -0.5)), mk(n, do, 1.0)


def dims(n, di, f, do, dtype, act="silu", flags=0):
    if dtype == torch.float32:
        flags |= P.PKM_F_FP32
    return P.FfnDims(n, di, f, do, ACT[act], flags)


def values_of(d, saved):
    if d.flags & P.PKM_FFN_CKPT8:
        return tuple(R.unpack8(saved[k], saved[k + "_scale"], d.d_ff) for k in ("g", "u"))
    return saved["g"], saved["u"]


def check_forward(d, t, act, saved, y, rms):
    want = R.forward(act, **t, r=R.roundoff(y.dtype))
    R.check(y, want["y"], "y", rms)
    if saved is None:
        return
    for k, v in zip(("g", "u"), values_of(d, saved)):
        value, bound = want[k]
        if d.flags & P.PKM_FFN_CKPT8:  # half a step of the run's scale, and the fp32 sum's error
            exact = R.forward(act, **t, r=0.0)[k][1]
            bound = exact + saved[k + "_scale"].double().repeat_interleave(32, 1)[:, :d.d_ff] * 0.501
        R.check(v, (value, bound + 1e-30), k)


def run_backward(d, t, saved, dy, grads=None, ws=None, **kw):
    wt = torch.bfloat16 if d.flags & P.PKM_FFN_GRAD_BF16 else torch.float32
    out = grads or {"d" + k: torch.zeros_like(t[k], dtype=wt) for k in ("Wg", "Wu", "Wd")}
    out.setdefault("dx", torch.full_like(t["x"], 3.0))
    P.pkm_ffn_backward(d, **t, saved=saved, dy=dy, workspace=scratch(d, P.PKM_BWD) if ws is None else ws,
                       **out, **kw)
    return out


def check_backward(d, t, act, saved, dy, out, r, rms, base=None):
    g, u = values_of(d, saved)
    rw = 2.0 ** -8 if d.flags & P.PKM_FFN_GRAD_BF16 else 2.0 ** -23
    want = R.backward(act, *t.values(), g, u, dy, r, rw)
    for k, v in out.items():
        R.check(v, want[k], k, rms)


# (N, d_in, d_ff, d_out): one token to several tiles; widths of one group of 8, below, at and
# beyond the tile sizes 64, 128 and 256
SIZES = [(1, 8, 8, 8), (3, 64, 40, 72), (64, 64, 256, 64), (65, 136, 264, 200),
         (130, 72, 520, 136), (257, 256, 136, 264), (300, 328, 1000, 520), (515, 1600, 312, 1600)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("mode", ["bf16", "bf16-ckpt8", "fp32", "fp32-ckpt8", "simt", "simt-ckpt8"])
def test_forward_and_backward(size, mode, act):
    n, di, f, do = size
    dtype = torch.float32 if mode.startswith("fp32") else torch.bfloat16
    flags = (P.PKM_F_SIMT if mode.startswith("simt") else 0) | (
        P.PKM_FFN_CKPT8 if mode.endswith("ckpt8") else 0)
    d = dims(n, di, f, do, dtype, act, flags)
    t, dy = make(n, di, f, do, dtype, seed=n + f)
    rms = TWO if dtype == torch.bfloat16 else None
    whole, y = guarded(n, do, dtype)
    saved = P.alloc_ffn_saved(d)
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, act, saved, y, rms)
    assert (whole[n:] == 7.0).all()
    # the same block with nothing kept
    y2 = torch.empty_like(y)
    P.pkm_ffn_forward(d, **t, y=y2, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, act, None, y2, rms)
    dxw, dx = guarded(n, di, dtype)
    grads = {"d" + k: torch.zeros_like(t[k], dtype=torch.float32) for k in ("Wg", "Wu", "Wd")}
    out = run_backward(d, t, saved, dy, dict(grads, dx=dx))
    check_backward(d, t, act, saved, dy, out, R.roundoff(dtype), rms)
    assert (dxw[n:] == 7.0).all()
    if dtype == torch.bfloat16:  # bf16 gradients, overwritten
        db = dims(n, di, f, do, dtype, act, flags | P.PKM_FFN_GRAD_BF16)
        ob = run_backward(db, t, saved, dy,
                          {"d" + k: torch.full_like(t[k], 5.0) for k in ("Wg", "Wu", "Wd")})
        check_backward(db, t, act, saved, dy, ob, 2.0 ** -8, TWO)
    assert P.pkm_check_status() == P.PKM_OK


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 33, 63, 64, 65, 100, 128])
def test_few_tokens(n):
    """The decode sizes, nothing kept; rows behind the last token stay as they were."""
    t, _ = make(n, 1600, 712, 1048, torch.bfloat16, seed=n)
    d = dims(n, 1600, 712, 1048, torch.bfloat16)
    whole, y = guarded(n, 1048, torch.bfloat16)
    P.pkm_ffn_forward(d, **t, y=y, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, "silu", None, y, TWO)
    assert (whole[n:] == 7.0).all()


@pytest.mark.parametrize("mode", ["fp32", "fp32-ckpt8", "simt", "simt-ckpt8"])
def test_cuda_core_path_of_large_products(mode):
    """Beyond 2^29 multiplications a product the CUDA-core path takes its large tiles and separate
    elementwise kernels."""
    n, di, f, do = 1100, 1032, 520, 264
    assert n * f * di > 1 << 29
    dtype = torch.float32 if mode.startswith("fp32") else torch.bfloat16
    flags = (P.PKM_F_SIMT if mode.startswith("simt") else 0) | (
        P.PKM_FFN_CKPT8 if mode.endswith("ckpt8") else 0)
    act = "gelu" if mode.endswith("ckpt8") else "silu"
    d = dims(n, di, f, do, dtype, act, flags)
    t, dy = make(n, di, f, do, dtype, seed=12)
    whole, y = guarded(n, do, dtype)
    saved, rms = P.alloc_ffn_saved(d), TWO if dtype == torch.bfloat16 else None
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, act, saved, y, rms)
    assert (whole[n:] == 7.0).all()
    check_backward(d, t, act, saved, dy, run_backward(d, t, saved, dy), R.roundoff(dtype), rms)
    if dtype == torch.bfloat16:
        db = dims(n, di, f, do, dtype, act, flags | P.PKM_FFN_GRAD_BF16)
        out = run_backward(db, t, saved, dy, {"d" + k: torch.full_like(t[k], 5.0)
                                              for k in ("Wg", "Wu", "Wd")})
        check_backward(db, t, act, saved, dy, out, 2.0 ** -8, TWO)


@pytest.mark.parametrize("mode", ["bf16", "bf16-ckpt8", "fp32"])
def test_offsets_beyond_32_bits(mode):
    """More than 2^31 kept values: the last tokens' rows are right, and so is a weight gradient
    that only they feed."""
    n, di, f, do = 336_000, 64, 6400, 64
    assert n * f > 1 << 31
    dtype = torch.float32 if mode == "fp32" else torch.bfloat16
    d = dims(n, di, f, do, dtype, "silu", P.PKM_FFN_CKPT8 if mode.endswith("ckpt8") else 0)
    t, dy = make(n, di, f, do, dtype, seed=1)
    last = slice(n - 70, n)
    dy[:n - 70] = 0
    y, saved = torch.empty(n, do, dtype=dtype, device="cuda"), P.alloc_ffn_saved(d)
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    tail = {**t, "x": t["x"][last]}
    kept = {k: None if v is None else v[last] for k, v in saved.items()}
    rms = TWO if dtype == torch.bfloat16 else None
    check_forward(d, tail, "silu", kept, y[last], rms)
    out = run_backward(d, t, saved, dy)
    assert (out["dx"][:n - 70] == 0).all()
    out["dx"] = out["dx"][last]
    check_backward(d, tail, "silu", kept, dy[last], out, R.roundoff(dtype), rms)
    assert P.pkm_check_status() == P.PKM_OK


def test_the_current_stream_is_used():
    """Without a stream argument the calls go to torch's current stream."""
    n, di, f, do = 12, 256, 520, 136
    d = dims(n, di, f, do, torch.bfloat16)
    t, dy = make(n, di, f, do, torch.bfloat16, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, saved = torch.empty_like(dy), P.alloc_ffn_saved(d)
        a = torch.randn(8192, 8192, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-4          # the side stream is busy: a call elsewhere would overtake x
        t["x"] = (t["x"].float() + a[:n, :di] * 0).bfloat16()
        P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
        codes, scale = P.alloc_ckpt8(n, do)
        P.pkm_ckpt8_pack(y, codes, scale)
    side.synchronize()
    check_forward(d, t, "silu", saved, y, TWO)
    wc, ws = R.pack8(y)
    assert torch.equal(codes, wc) and torch.equal(scale, ws)


def offset16(t):
    """The same values at an address that is a multiple of 16 and of no more."""
    per = 16 // t.element_size()
    flat = torch.empty(t.numel() + 4 * per, dtype=t.dtype, device="cuda")
    start = per if flat.data_ptr() % 32 == 0 else 0
    out = flat[start:start + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


@pytest.mark.parametrize("n", [5, 300])
@pytest.mark.parametrize("flags", [0, P.PKM_FFN_CKPT8, P.PKM_F_FP32, P.PKM_F_SIMT])
def test_tensors_on_16_byte_boundaries(flags, n):
    """Every tensor at the least alignment the library takes."""
    di, f, do = 72, 160, 88
    dtype = torch.float32 if flags & P.PKM_F_FP32 else torch.bfloat16
    d = P.FfnDims(n, di, f, do, P.PKM_ACT_GELU, flags)
    t, dy = make(n, di, f, do, dtype, seed=8)
    t, dy = {k: offset16(v) for k, v in t.items()}, offset16(dy)
    saved = {k: None if v is None else offset16(v) for k, v in P.alloc_ffn_saved(d).items()}
    y, rms = offset16(torch.zeros_like(dy)), TWO if dtype == torch.bfloat16 else None
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, "gelu", saved, y, rms)
    P.pkm_ffn_forward(d, **t, y=y, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, "gelu", None, y, rms)
    out = {"d" + k: offset16(torch.zeros_like(v, dtype=dtype if k == "x" else torch.float32))
           for k, v in t.items()}
    run_backward(d, t, saved, dy, out)
    check_backward(d, t, "gelu", saved, dy, out, R.roundoff(dtype), rms)


# row tiles of 256 and column tiles of 256, 192 and less; k cut into parts (few tiles, long k) and
# not; weight gradients of one width in one launch or of two widths in two
@pytest.mark.parametrize("size", [(40, 2048, 2048, 64), (200, 64, 4104, 2048), (513, 1024, 2056, 264),
                                  (1300, 264, 640, 264), (700, 1608, 1368, 520)])
def test_tile_walks_and_split_sums(size):
    n, di, f, do = size
    d = dims(n, di, f, do, torch.bfloat16, "silu", P.PKM_FFN_GRAD_BF16)
    t, dy = make(n, di, f, do, torch.bfloat16, seed=n)
    y, saved = torch.empty(n, do, dtype=torch.bfloat16, device="cuda"), P.alloc_ffn_saved(d)
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, "silu", saved, y, TWO)
    want = run_backward(d, t, saved, dy, {"d" + k: torch.full_like(t[k], 5.0)
                                          for k in ("Wg", "Wu", "Wd")})
    check_backward(d, t, "silu", saved, dy, want, 2.0 ** -8, TWO)
    for keep in (("dWg",), ("dWu",), ("dWd",), ("dWu", "dWd"), ("dWg", "dWu"), ("dx", "dWd")):
        out = {k: torch.full_like(want[k], 5.0) for k in keep}
        P.pkm_ffn_backward(d, **t, saved=saved, dy=dy, workspace=scratch(d, P.PKM_BWD), **out)
        for k, v in out.items():  # the same sums in the same order, whatever else is asked for
            assert torch.equal(v, want[k]), (keep, k)
    assert P.pkm_check_status() == P.PKM_OK


@pytest.mark.parametrize("flags", [0, P.PKM_FFN_CKPT8])
def test_a_training_size(flags):
    """Several tiles in every direction, ragged in all of them."""
    n, di, f, do = 2065, 1032, 2728, 1096
    d = dims(n, di, f, do, torch.bfloat16, "silu", flags)
    t, dy = make(n, di, f, do, torch.bfloat16, seed=5)
    y, saved = torch.empty(n, do, dtype=torch.bfloat16, device="cuda"), P.alloc_ffn_saved(d)
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    check_forward(d, t, "silu", saved, y, TWO)
    check_backward(d, t, "silu", saved, dy, run_backward(d, t, saved, dy), 2.0 ** -8, TWO)


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_fp32_gradients_accumulate_and_any_may_be_skipped(mode):
    dtype = torch.float32 if mode == "fp32" else torch.bfloat16
    n, di, f, do = 70, 72, 136, 40
    d = dims(n, di, f, do, dtype)
    t, dy = make(n, di, f, do, dtype, seed=2)
    saved = P.alloc_ffn_saved(d)
    y = torch.empty(n, do, dtype=dtype, device="cuda")
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    once = run_backward(d, t, saved, dy)
    base = {"d" + k: torch.randn(t[k].shape, device="cuda") for k in ("Wg", "Wu", "Wd")}
    twice = run_backward(d, t, saved, dy, {k: v.clone() for k, v in base.items()})
    for k, b in base.items():  # one fp32 addition to each
        assert ((twice[k] - (b + once[k])).abs() <= 2.0 ** -23 * (b.abs() + once[k].abs())).all()
    for skip in ("dx", "dWg", "dWu", "dWd"):
        out = {k: v.clone().zero_() for k, v in once.items() if k != skip}
        P.pkm_ffn_backward(d, **t, saved=saved, dy=dy, workspace=scratch(d, P.PKM_BWD), **out)
        for k, v in out.items():
            assert torch.equal(v, once[k]), (skip, k)
    P.pkm_ffn_backward(d, **t, saved=saved, dy=dy, workspace=scratch(d, P.PKM_BWD))
    assert P.pkm_check_status() == P.PKM_OK


@pytest.mark.parametrize("flags", [0, P.PKM_FFN_CKPT8])
def test_device_gradient_against_differences(flags):
    """fp32 storage: the directional derivative of sum(dy * y) by central differences."""
    n, di, f, do = 37, 40, 72, 24
    d = dims(n, di, f, do, torch.float32, "gelu")
    dc = dims(n, di, f, do, torch.float32, "gelu", flags)
    t, dy = make(n, di, f, do, torch.float32, seed=9)

    def loss(tt):
        y = torch.empty(n, do, device="cuda")
        P.pkm_ffn_forward(d, **tt, y=y, workspace=scratch(d, P.PKM_FWD))
        return (y.double() * dy.double()).sum().item()

    saved = P.alloc_ffn_saved(dc)
    P.pkm_ffn_forward(dc, **t, y=torch.empty(n, do, device="cuda"), saved=saved,
                      workspace=scratch(dc, P.PKM_FWD))
    out = run_backward(dc, t, saved, dy)
    for name, g in (("x", "dx"), ("Wg", "dWg"), ("Wu", "dWu"), ("Wd", "dWd")):
        v = torch.randn_like(t[name])
        eps = 2.0 ** -8
        diff = (loss({**t, name: t[name] + eps * v}) - loss({**t, name: t[name] - eps * v})) / (2 * eps)
        dot = (out[g].double() * v.double()).sum().item()
        # fp32 noise of two losses (n * do terms of order 1, 2^-24 each, over 2 eps) and eps^2
        # times a third derivative of order 10 times the gradient's size; with 8-bit
        # checkpoints g and u are off by up to 1/254 of their run's largest
        size = out[g].double().norm().item() * v.double().norm().item()
        tol = (0.004 if flags else 0.0) * size + 10 * eps * eps * size + 1e-3
        assert abs(diff - dot) <= tol, (name, diff, dot)


def test_non_finite_values_stay_in_their_rows():
    """A token with a NaN or an infinity spoils its own row of y and dx only; kept in 8 bits it
    reads as NaN."""
    n, di, f, do = 200, 64, 136, 72
    for flags in (0, P.PKM_FFN_CKPT8):
        d = dims(n, di, f, do, torch.bfloat16, "silu", flags)
        t, dy = make(n, di, f, do, torch.bfloat16, seed=4)
        t["x"][7, 3], t["x"][150, 1] = float("nan"), float("inf")
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[[7, 150]] = True
        y, saved = torch.empty(n, do, dtype=torch.bfloat16, device="cuda"), P.alloc_ffn_saved(d)
        P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
        assert torch.isfinite(y[~bad]).all() and not torch.isfinite(y[bad]).any()
        if flags:
            assert torch.isnan(saved["g_scale"][bad]).all()
            assert torch.isfinite(saved["g_scale"][~bad]).all()
        dx = torch.empty(n, di, dtype=torch.bfloat16, device="cuda")
        P.pkm_ffn_backward(d, **t, saved=saved, dy=dy, dx=dx, workspace=scratch(d, P.PKM_BWD))
        assert torch.isfinite(dx[~bad]).all() and not torch.isfinite(dx[bad]).any()


def test_extreme_projections():
    """Projections far out in both tails: the gate saturates without a NaN."""
    n, di, f, do = 66, 64, 72, 64
    for act in ("silu", "gelu"):
        d = dims(n, di, f, do, torch.bfloat16, act)
        t, dy = make(n, di, f, do, torch.bfloat16, seed=6, scale=300.0)
        y, saved = torch.empty(n, do, dtype=torch.bfloat16, device="cuda"), P.alloc_ffn_saved(d)
        P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
        check_forward(d, t, act, saved, y, TWO)
        check_backward(d, t, act, saved, dy, run_backward(d, t, saved, dy), 2.0 ** -8, TWO)


def test_two_streams_two_workspaces_and_a_replayed_graph():
    n, di, f, do = 600, 200, 520, 136
    d = dims(n, di, f, do, torch.bfloat16, "silu", P.PKM_FFN_CKPT8 | P.PKM_FFN_GRAD_BF16)
    sets = []
    for seed in (1, 2):
        t, dy = make(n, di, f, do, torch.bfloat16, seed=seed)
        b = dict(t=t, dy=dy, y=torch.empty(n, do, dtype=torch.bfloat16, device="cuda"),
                 saved=P.alloc_ffn_saved(d), fw=scratch(d, P.PKM_FWD), bw=scratch(d, P.PKM_BWD),
                 out={"d" + k: torch.empty_like(v) for k, v in t.items()})
        sets.append(b)

    def step(b, stream=None):
        P.pkm_ffn_forward(d, **b["t"], y=b["y"], saved=b["saved"], workspace=b["fw"], stream=stream)
        P.pkm_ffn_backward(d, **b["t"], saved=b["saved"], dy=b["dy"], workspace=b["bw"],
                           stream=stream, **b["out"])

    want = []
    for b in sets:
        step(b)
        torch.cuda.synchronize()
        want.append([b["y"].clone()] + [v.clone() for v in b["out"].values()])
    streams = [torch.cuda.Stream() for _ in sets]
    for b in sets:
        b["y"].zero_()
        for v in b["out"].values():
            v.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(sets, streams):
            step(b, s)
    torch.cuda.synchronize()
    for b, w in zip(sets, want):
        assert all(torch.equal(p, q) for p, q in zip([b["y"], *b["out"].values()], w))
    # captured once, replayed on new contents of the same buffers
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(sets[0])
    for k in sets[0]["t"]:
        sets[0]["t"][k].copy_(sets[1]["t"][k])
    sets[0]["dy"].copy_(sets[1]["dy"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q)
               for p, q in zip([sets[0]["y"], *sets[0]["out"].values()], want[1]))


def test_no_tokens_touch_nothing():
    d = dims(0, 64, 64, 64, torch.bfloat16)
    t, dy = make(0, 64, 64, 64, torch.bfloat16)
    P.pkm_ffn_forward(d, **t, y=torch.empty_like(dy), saved=P.alloc_ffn_saved(d))
    grads = {"d" + k: torch.ones_like(t[k], dtype=torch.float32) for k in ("Wg", "Wu", "Wd")}
    P.pkm_ffn_backward(d, **t, saved=P.alloc_ffn_saved(d), dy=dy, dx=torch.empty_like(t["x"]), **grads)
    assert all((v == 1).all() for v in grads.values())


def test_memory_layer_then_block_with_checkpointed_inputs():
    """A layer pair as a model runs it: the memory layer's output joins the residual stream, the
    gated block follows; the step keeps the memory layer's input and the block's projections in
    8 bits.  The weight gradients of the query network from the unpacked input stay within the
    checkpoint's step of those from the input itself."""
    N, dm, f = 320, 128, 264
    cfg = dict(N=N, d_in=dm, h=2, dk=128, C1=64, C2=64, k=8, d_v=dm)
    gen = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    md = P.Dims(**cfg)
    x = rnd(N, dm).bfloat16()
    Wq = (rnd(256, dm) * dm ** -0.5).bfloat16()
    bn = torch.stack([torch.zeros(256), torch.ones(256), torch.ones(256), torch.zeros(256)]).cuda()
    sub, val = (rnd(2, 128, 64) * 0.1).bfloat16(), (rnd(64 * 64, dm) * dm ** -0.5).bfloat16()
    msaved, ymem = P.alloc_saved(md), torch.empty(N, dm, device="cuda")
    P.pkm_forward(md, x, Wq, bn, sub, val, ymem, msaved)
    z = (x.float() + ymem).bfloat16()
    fd = P.FfnDims(N, dm, f, dm, P.PKM_ACT_SILU, P.PKM_FFN_CKPT8)
    t = make(N, dm, f, dm, torch.bfloat16, seed=3)[0]
    t["x"] = z
    y, fsaved = torch.empty(N, dm, dtype=torch.bfloat16, device="cuda"), P.alloc_ffn_saved(fd)
    P.pkm_ffn_forward(fd, **t, y=y, saved=fsaved, workspace=P.alloc_ffn_workspace(fd, P.PKM_FWD))
    check_forward(fd, t, "silu", fsaved, y, TWO)
    codes, scale = P.alloc_ckpt8(N, dm)
    P.pkm_ckpt8_pack(x, codes, scale)

    dy = rnd(N, dm).bfloat16()
    out = run_backward(fd, t, fsaved, dy)
    check_backward(fd, t, "silu", fsaved, dy, out, 2.0 ** -8, TWO)
    dmem = (out["dx"].float() + dy.float()).contiguous()  # the residual's gradient
    x8 = torch.empty_like(x)
    P.pkm_ckpt8_unpack(codes, scale, x8)
    ws = P.alloc_workspace(md, P.PKM_BWD)
    got = {}
    for name, xin in (("kept", x), ("ckpt", x8)):
        dWq, dxm = torch.zeros(256, dm, device="cuda"), torch.zeros(N, dm, device="cuda")
        P.pkm_backward(md, xin, Wq, bn, sub, val, msaved, dmem, dx=dxm, dWq=dWq, workspace=ws)
        got[name] = (dWq, dxm)
    assert torch.equal(got["kept"][1], got["ckpt"][1])  # dx does not read x
    # dWq = dq^T x: each x is off by at most half its run's step and one bf16 rounding
    step = scale.double().repeat_interleave(32, 1)[:, :dm] * 0.5 + 2.0 ** -8 * x.double().abs() * 1.01
    dq_abs = got["kept"][0].double()
    rel = (got["ckpt"][0].double() - dq_abs).norm() / dq_abs.norm()
    assert rel <= step.norm() / x.double().norm()
    assert P.pkm_check_status() == P.PKM_OK


@pytest.mark.parametrize("kind", ["bf16", "w4"])
@pytest.mark.parametrize("n", [1, 8, 16])
def test_few_token_calls_back_to_back_read_their_own_inner_values(n, kind):
    """Calls of two inputs in turn through one workspace: each result is its own input's, although
    the second kernel of a call starts while the first still writes what it reads."""
    di, f, do, group = 1600, 1056, 264, 32
    t, _ = make(n, di, f, do, torch.bfloat16, seed=n)
    xs = [t.pop("x"), torch.randn(n, di, device="cuda").bfloat16()]
    d = dims(n, di, f, do, torch.bfloat16)
    ws = scratch(d, P.PKM_FWD)
    if kind == "w4":
        packed = {k: P.alloc_w4(*W.shape, group) for k, W in t.items()}
        for k, W in t.items():
            P.pkm_w4_pack(W, *packed[k], group=group)

    def call(x, y):
        if kind == "w4":
            P.pkm_w4_ffn(d, x, packed["Wg"], packed["Wu"], packed["Wd"], y, group=group, workspace=ws)
        else:
            P.pkm_ffn_forward(d, x, t["Wg"], t["Wu"], t["Wd"], y, workspace=ws)

    want = []
    for x in xs:
        y = torch.empty(n, do, dtype=torch.bfloat16, device="cuda")
        call(x, y)
        torch.cuda.synchronize()
        want.append(y)
    assert not torch.equal(*want)
    got = torch.zeros(200, n, do, dtype=torch.bfloat16, device="cuda")
    for i in range(200):
        call(xs[i & 1], got[i])
    for i in range(200):
        assert torch.equal(got[i], want[i & 1]), i


class Fenced:
    """Tensors that lie between two KiB of a known pattern; check() finds what wrote there."""
    EDGE = 1024

    def __init__(self):
        self.raw = []

    def __call__(self, shape, dtype, fill=None):
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        raw = torch.full((n + 2 * self.EDGE,), 255, dtype=torch.uint8, device="cuda")
        raw[:self.EDGE] = raw[self.EDGE + n:] = 0xA5
        self.raw.append((raw, n))
        t = raw[self.EDGE:self.EDGE + n].view(dtype).view(shape)
        return t if fill is None else t.fill_(fill)

    def like(self, t, fill=None):
        return None if t is None else self(t.shape, t.dtype, fill)

    def check(self):
        for raw, n in self.raw:
            assert (raw[:self.EDGE] == 0xA5).all() and (raw[self.EDGE + n:] == 0xA5).all(), n


@pytest.mark.parametrize("mode", ["bf16", "bf16-ckpt8", "fp32", "fp32-ckpt8", "simt", "simt-ckpt8"])
@pytest.mark.parametrize("size", [(1, 8, 8, 8), (3, 64, 40, 72), (65, 136, 264, 200),
                                  (300, 328, 1000, 520), (40, 2048, 2048, 64), (513, 1024, 2056, 264),
                                  (1100, 1032, 520, 264)])
def test_nothing_is_written_outside_the_buffers(size, mode):
    """Results, kept values, gradients and a workspace of exactly the stated size, each between
    fences; what is inside has the same bits as without them."""
    n, di, f, do = size
    dtype = torch.float32 if mode.startswith("fp32") else torch.bfloat16
    flags = (P.PKM_F_SIMT if mode.startswith("simt") else 0) | (
        P.PKM_FFN_CKPT8 if mode.endswith("ckpt8") else 0)
    t, dy = make(n, di, f, do, dtype, seed=n)
    for grad16 in (0, P.PKM_FFN_GRAD_BF16)[:1 if dtype == torch.float32 else 2]:
        d, fence = dims(n, di, f, do, dtype, "gelu", flags | grad16), Fenced()
        wt = torch.bfloat16 if grad16 else torch.float32

        def workspace(which):
            need = P.pkm_ffn_workspace_bytes(d, which)
            return dict(workspace=fence((need,), torch.uint8), workspace_bytes=need)

        plain = dict(y=torch.empty_like(dy), none=torch.empty_like(dy), saved=P.alloc_ffn_saved(d),
                     grads={"d" + k: torch.zeros_like(v, dtype=v.dtype if k == "x" else wt)
                            for k, v in t.items()})
        fenced = dict(y=fence.like(dy), none=fence.like(dy),
                      saved={k: fence.like(v) for k, v in plain["saved"].items()},
                      grads={k: fence.like(v, 0) for k, v in plain["grads"].items()})
        for b, ws in ((plain, lambda w: dict(workspace=scratch(d, w))), (fenced, workspace)):
            P.pkm_ffn_forward(d, **t, y=b["none"], **ws(P.PKM_FWD))
            P.pkm_ffn_forward(d, **t, y=b["y"], saved=b["saved"], **ws(P.PKM_FWD))
            P.pkm_ffn_backward(d, **t, saved=b["saved"], dy=dy, **b["grads"], **ws(P.PKM_BWD))
        fence.check()
        assert torch.equal(fenced["y"], plain["y"]) and torch.equal(fenced["none"], plain["none"])
        for part in ("saved", "grads"):
            for k, v in plain[part].items():
                assert v is None or torch.equal(fenced[part][k], v), k
    assert P.pkm_check_status() == P.PKM_OK


def _norm_off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("ckpt8", [0, P.PKM_FFN_CKPT8])
@pytest.mark.parametrize("size", [(64, 64, 256, 64), (130, 72, 520, 136), (515, 1600, 312, 1600),
                                  (1100, 1032, 520, 264)])
@pytest.mark.parametrize("store", ["fp32", "simt"])
def test_everything_between_the_products_stays_in_32_bits(size, store, ckpt8, act):
    """fp32 storage, and bf16 storage with PKM_F_SIMT, whose h, dg and du are fp32 too.

    The 2-norm of an error.  Adding K terms of random sign rounds K times by at most 2^-24 of a
    partial sum whose mean square grows evenly up to the result's, so the error is at most
    sqrt(K / 6) 2^-24 of it.  With g of variance 1, the errors of g and u enter h at most 1.9 times
    (the largest act' over the norm of act: 1.84 for SiLU, 1.73 for GELU) and once, together
    sqrt(4.6 d_in / 6), below sqrt(d_in); the functions are good to 8 * 2^-24.  So y stays within
    2^-24 sqrt(d_in + d_ff + 64), and the gradients, sums over d_out, 2 d_ff and the tokens of
    factors that are read exactly, within 2^-24 sqrt(d_out + 2 d_ff + N + 64).  A loss of three or
    four bits passes neither.  A result in bf16 is rounded once more, elementwise by 2^-8 of its
    value and in the norm by 2^-8 / sqrt(3) = 2.26e-3 at most: evenly within the step, and no
    significand is below 1.  (With h in bf16 as well it is 2.35e-3.)"""
    n, di, f, do = size
    dtype = torch.float32 if store == "fp32" else torch.bfloat16
    once = 0.0 if store == "fp32" else 2.0 ** -8
    d = dims(n, di, f, do, dtype, act, ckpt8 | (P.PKM_F_SIMT if store == "simt" else 0))
    t, dy = make(n, di, f, do, dtype, seed=n + 1)
    y, saved = torch.empty(n, do, dtype=dtype, device="cuda"), P.alloc_ffn_saved(d)
    P.pkm_ffn_forward(d, **t, y=y, saved=saved, workspace=scratch(d, P.PKM_FWD))
    value, bound = R.forward(act, **t, r=2.0 ** -24)["y"]
    R.check(y, (value, bound + once * value.abs()), "y")
    limit = 2.0 ** -24 * (di + f + 64) ** 0.5
    assert _norm_off(y, value) <= (limit if store == "fp32" else 2.0 ** -8 / 3 ** 0.5)
    out = run_backward(d, t, saved, dy)
    want = R.backward(act, *t.values(), *values_of(d, saved), dy, 2.0 ** -24, 2.0 ** -23)
    for k, v in out.items():
        value, bound = want[k]
        R.check(v, (value, bound + (once * value.abs() if k == "dx" else 0)), k)
        if store == "fp32" or k != "dx":  # weight gradients are fp32
            assert _norm_off(v, value) <= 2.0 ** -24 * (do + 2 * f + n + 64) ** 0.5, k
