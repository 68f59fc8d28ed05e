"""8-bit activation checkpoints and 4-bit weight products on the device against their
definitions in 64 bits."""
import pytest
import torch

from product_key_memory_pkm_b200 import pkm as P

from . import ffn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from product_key_memory_pkm_b200 import build as B
    B.build()


def rnd(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=gen)


# ------------------------------------------------------------------ 8-bit checkpoints
def pack(x):
    rows, cols = x.shape
    codes, scale = P.alloc_ckpt8(rows + 1, cols)
    codes.fill_(99)
    scale.fill_(99.0)
    P.pkm_ckpt8_pack(x, codes[:rows], scale[:rows])
    assert (codes[rows] == 99).all() and (scale[rows] == 99).all()
    return codes[:rows], scale[:rows]


def unpack(codes, scale, cols, dtype):
    rows = codes.shape[0]
    out = torch.full((rows + 1, cols), 5.0, dtype=dtype, device="cuda")
    P.pkm_ckpt8_unpack(codes, scale, out[:rows])
    assert (out[rows] == 5.0).all()
    return out[:rows]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 32), (2, 24), (3, 40), (5, 64), (7, 136),
                                       (130, 1000), (33, 6400), (1000, 72), (2500, 1608)])
def test_checkpoint_round_trip(rows, cols, dtype):
    x = (rnd(rows + cols, rows, cols) * 3).to(dtype)
    codes, scale = pack(x)
    wc, ws = R.pack8(x)
    assert torch.equal(codes, wc) and torch.equal(scale, ws)
    for out in (torch.bfloat16, torch.float32):
        v = unpack(codes, scale, cols, out)
        want = (wc.float() * ws.repeat_interleave(32, 1))[:, :cols]
        assert torch.equal(v, want.to(out))


@pytest.mark.parametrize("cols", [3200, 3208])
def test_checkpoint_offsets_beyond_32_bits(cols):
    rows = (1 << 31) // cols + 100
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-50:] = rnd(1, 50, cols).bfloat16()
    codes, scale = P.alloc_ckpt8(rows, cols)
    P.pkm_ckpt8_pack(x, codes, scale)
    wc, ws = R.pack8(x[-60:])
    assert torch.equal(codes[-60:], wc) and torch.equal(scale[-60:], ws)
    x[-50:] = 0
    P.pkm_ckpt8_unpack(codes, scale, x)
    want = (wc.float() * ws.repeat_interleave(32, 1))[:, :cols].bfloat16()
    assert torch.equal(x[-60:], want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_checkpoint_halves_go_to_the_even_code(dtype):
    """Runs whose values lie exactly between two codes, and one step to either side of it."""
    k = torch.arange(-126, 126, 2, device="cuda").float()
    rows = []
    for top in (127.0, 254.0, 127.0 / 64, 1016.0):
        half = (k + 0.5) * (top / 127)
        up = torch.nextafter(half, torch.full_like(half, 1e9))
        down = torch.nextafter(half, torch.full_like(half, -1e9))
        for v in (half, up, down, half + top / 127):
            v = torch.nn.functional.pad(v, (0, 29)).view(5, 31)
            rows.append(torch.cat([torch.full((5, 1), top, device="cuda"), v], 1).to(dtype))
    x = torch.cat(rows)
    x = x.contiguous()
    codes, scale = pack(x)
    wc, ws = R.pack8(x)
    assert torch.equal(codes, wc) and torch.equal(scale, ws)


def test_checkpoint_of_zeros_extremes_and_non_finite_values():
    x = rnd(0, 12, 96)
    x[0] = 0
    x[1, :32] = 0
    x[2] *= 1e-38
    x[3] *= 1e-42                        # subnormal
    x[4, 5] = 3.4e38
    x[5, 40] = float("inf")
    x[6, 41] = float("-inf")
    x[7, 70] = float("nan")
    x[8] = -0.0
    x[9] = 1e-45
    codes, scale = pack(x)
    bad = torch.zeros_like(scale, dtype=torch.bool)
    for r, run in ((5, 1), (6, 1), (7, 2)):
        bad[r, run] = True
    assert torch.isnan(scale[bad]).all() and torch.isfinite(scale[~bad]).all()
    assert (codes.view(12, 3, 32)[bad] == 0).all()
    clean = x.clone().view(12, 3, 32)
    clean[bad] = 0
    wc, ws = R.pack8(clean.view(12, 96))
    assert torch.equal(codes, wc) and torch.equal(scale[~bad], ws[~bad])
    v = unpack(codes, scale, 96, torch.float32).view(12, 3, 32)
    assert torch.isnan(v[bad]).all() and torch.isfinite(v[~bad]).all()


# ------------------------------------------------------------------ 4-bit weights
@pytest.mark.parametrize("group", [32, 64, 128, 96, 4096])
@pytest.mark.parametrize("o,i", [(1, 32), (7, 64), (40, 160), (129, 1600), (300, 2016)])
def test_w4_pack_and_unpack(o, i, group):
    W = rnd(o + i, o, i).bfloat16()
    W[0, :32] = 0
    codes, scale = P.alloc_w4(o, i, group)
    P.pkm_w4_pack(W, codes, scale, group=group)
    wc, ws = R.pack4(W, group)
    assert torch.equal(scale, ws) and torch.equal(R.nibbles(codes), wc)
    out = torch.empty_like(W)
    P.pkm_w4_unpack(codes, scale, out, group=group)
    assert torch.equal(out, R.values4(wc, ws, group).bfloat16())


def test_w4_pack_of_non_finite_weights():
    W = rnd(1, 3, 128).bfloat16()
    W[0, 5], W[1, 70], W[2, 100] = float("nan"), float("inf"), 3e38
    codes, scale = P.alloc_w4(3, 128, 64)
    P.pkm_w4_pack(W, codes, scale, group=64)
    bad = torch.tensor([[1, 0], [0, 1], [0, 0]], device="cuda").bool()
    assert torch.isnan(scale[bad]).all() and torch.isfinite(scale[~bad]).all()


def random_w4(seed, o, i, group):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (o, i // 2), device="cuda", generator=gen, dtype=torch.uint8)
    scale = (torch.rand(o, -(-i // group), device="cuda", generator=gen) * 0.1 + 0.01).bfloat16()
    return codes, scale


@pytest.mark.parametrize("group", [32, 64, 96, 128, 512])
@pytest.mark.parametrize("n,i,o", [(1, 32, 1), (1, 64, 9), (2, 96, 17), (1, 1600, 2048),
                                   (3, 1600, 100), (8, 2016, 333), (9, 1024, 64), (16, 640, 1000),
                                   (17, 4128, 72), (33, 160, 50), (64, 1600, 515), (64, 32, 8),
                                   # many rows: whole rounds of the SMs and ragged ones, x in
                                   # one piece and in several
                                   (17, 96, 19001), (32, 1600, 40000), (40, 2016, 18944),
                                   (64, 32, 19999), (64, 4128, 19000), (16, 160, 20000),
                                   # large matrices of few tokens, and k in one to eight parts
                                   (1, 1600, 50264), (9, 2016, 33333), (20, 8192, 700),
                                   (48, 6400, 1600), (33, 1056, 129), (17, 16384, 64)])
def test_w4_matvec(n, i, o, group):
    x = rnd(n, n, i).bfloat16()
    codes, scale = random_w4(i, o, i, group)
    y = torch.full((n + 1, o), 5.0, device="cuda")
    P.pkm_w4_matvec(x, codes, scale, y[:n], group=group)
    W = R.values4(R.nibbles(codes), scale, group)
    mag = x.double().abs() @ W.abs().t()
    R.check(y[:n], (x.double() @ W.t(), (i + 8) * R.E32 * mag + 1e-30), "y")
    assert (y[n] == 5.0).all()
    # the sums do not depend on how many tokens share the call beyond their fp32 order
    assert P.pkm_check_status() == P.PKM_OK


def test_w4_matvec_is_reproducible_and_keeps_non_finite_tokens_apart():
    x = rnd(3, 20, 1600).bfloat16()
    codes, scale = random_w4(5, 700, 1600, 64)
    y1, y2 = (torch.empty(20, 700, device="cuda") for _ in range(2))
    P.pkm_w4_matvec(x, codes, scale, y1)
    P.pkm_w4_matvec(x, codes, scale, y2)
    assert torch.equal(y1, y2)
    x[4, 9], x[11, 100] = float("nan"), float("inf")
    P.pkm_w4_matvec(x, codes, scale, y2)
    keep = [r for r in range(20) if r not in (4, 11)]
    assert torch.equal(y1[keep], y2[keep])
    assert torch.isnan(y2[4]).all() and not torch.isfinite(y2[11]).any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n,i,f,o,group", [(1, 32, 32, 1, 32), (1, 1600, 6400, 1600, 64),
                                           (3, 96, 160, 50, 64), (8, 1600, 704, 333, 128),
                                           (17, 416, 512, 668, 32), (64, 640, 1056, 129, 96),
                                           (5, 2048, 8192, 2048, 128), (40, 1600, 6400, 1600, 64),
                                           (64, 96, 20000, 72, 32)])
def test_w4_block(n, i, f, o, group, act):
    x = rnd(n + i, n, i).bfloat16()
    packed = {k: random_w4(s, a, b, group)
              for s, (k, a, b) in enumerate((("Wg", f, i), ("Wu", f, i), ("Wd", o, f)))}
    d = P.FfnDims(n, i, f, o, P.PKM_ACT_GELU if act == "gelu" else P.PKM_ACT_SILU)
    ws = torch.full((P.pkm_ffn_workspace_bytes(d, P.PKM_FWD),), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((n + 1, o), 5.0, dtype=torch.bfloat16, device="cuda")
    P.pkm_w4_ffn(d, x, packed["Wg"], packed["Wu"], packed["Wd"], y[:n], group=group, workspace=ws)
    W = {k: R.values4(R.nibbles(c), s, group) for k, (c, s) in packed.items()}
    want = R.forward(act, x, W["Wg"], W["Wu"], W["Wd"], 2.0 ** -8)
    R.check(y[:n], want["y"], "y", 2 ** 0.5 * 2 ** -8)
    assert (y[n] == 5.0).all()


def test_w4_block_in_a_graph_and_against_the_unpacked_block():
    """Decode with packed weights, captured; prefill of the same weights through the unpacked
    bf16 block gives the same layer up to the weights' own rounding to bf16."""
    i, f, o, group = 256, 704, 256, 64
    Wf = {k: (rnd(s, a, b) * b ** -0.5).bfloat16()
          for s, (k, a, b) in enumerate((("Wg", f, i), ("Wu", f, i), ("Wd", o, f)))}
    packed, flat = {}, {}
    for k, W in Wf.items():
        packed[k] = P.alloc_w4(*W.shape, group)
        P.pkm_w4_pack(W, *packed[k], group=group)
        flat[k] = torch.empty_like(W)
        P.pkm_w4_unpack(*packed[k], flat[k], group=group)
    x = rnd(9, 6, i).bfloat16()
    d = P.FfnDims(6, i, f, o)
    ws = P.alloc_ffn_workspace(d, P.PKM_FWD)
    y = torch.empty(6, o, dtype=torch.bfloat16, device="cuda")

    def step():
        P.pkm_w4_ffn(d, x, packed["Wg"], packed["Wu"], packed["Wd"], y, group=group, workspace=ws)

    step()
    torch.cuda.synchronize()
    eager = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, eager)
    y2 = torch.empty_like(y)
    P.pkm_ffn_forward(d, x, flat["Wg"], flat["Wu"], flat["Wd"], y2, workspace=ws)
    want = R.forward("silu", x, flat["Wg"], flat["Wu"], flat["Wd"], 2.0 ** -8)
    R.check(y2, want["y"], "y", 2 ** 0.5 * 2 ** -8)
    # three layers of weights each within 2^-8 (bf16 of code * scale) move y by at most that
    # share of the magnitudes on the way, beside the bounds of the two calls
    a, sl = R.act_and_slope("silu", x.double() @ flat["Wg"].double().t())
    gm, um = (x.double().abs() @ flat[k].double().abs().t() for k in ("Wg", "Wu"))
    u = x.double() @ flat["Wu"].double().t()
    move = (R.SLOPE * gm * (u.abs() + um * 2 ** -7) + a.abs() * um + a.abs() * u.abs()) * 2 ** -7.9
    bound = move @ flat["Wd"].double().abs().t() + 2.1 * want["y"][1]
    assert ((y.double() - y2.double()).abs() <= bound).all()


# Each has the same power of two as its small twin, so that the kernels' columns per scale agree:
# 32, 64 and 128 columns in one load.
@pytest.mark.parametrize("group,twin", [(0x7fffffe0, 1632), (0x7fffffc0, 1728), (0x7fffff80, 1664)])
def test_w4_groups_near_the_largest_integer_are_one_group_per_row(group, twin):
    i, o = 1600, 100
    W = rnd(2, o, i).bfloat16()
    W[:, 0] *= torch.linspace(1, 9, o, device="cuda").bfloat16()  # a scale of its own for each row
    want = P.alloc_w4(o, i, twin)
    P.pkm_w4_pack(W, *want, group=twin)
    assert (R.nibbles(want[0]) == R.pack4(W, twin)[0]).all() and want[1].unique().numel() > o // 2
    codes, scale = P.alloc_w4(o + 1, i, group)
    codes.fill_(99)
    scale.fill_(5.0)
    P.pkm_w4_pack(W, codes[:o], scale[:o], group=group)
    assert torch.equal(codes[:o], want[0]) and torch.equal(scale[:o], want[1])
    assert (codes[o] == 99).all() and (scale[o] == 5.0).all()
    out, out2 = torch.empty_like(W), torch.empty_like(W)
    P.pkm_w4_unpack(*want, out, group=group)
    P.pkm_w4_unpack(*want, out2, group=twin)
    assert torch.equal(out, out2)
    for n, rows in ((1, o), (20, o), (20, 9600)):  # the last: the form for many rows
        x = rnd(n, n, i).bfloat16()
        q = want if rows == o else random_w4(4, rows, i, twin)
        y, y2 = (torch.empty(n, rows, device="cuda") for _ in range(2))
        P.pkm_w4_matvec(x, *q, y, group=group)
        P.pkm_w4_matvec(x, *q, y2, group=twin)
        assert torch.equal(y, y2)
    f = 1472  # of one group too
    packed = [random_w4(s, *shape, twin) for s, shape in enumerate(((f, i), (f, i), (o, f)))]
    d = P.FfnDims(7, i, f, o)
    ws, x = P.alloc_ffn_workspace(d, P.PKM_FWD), rnd(7, 7, i).bfloat16()
    y, y2 = (torch.empty(7, o, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    P.pkm_w4_ffn(d, x, *packed, y, group=group, workspace=ws)
    P.pkm_w4_ffn(d, x, *packed, y2, group=twin, workspace=ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,i,o", [(1, 64, 300), (5, 1600, 2048), (16, 8192, 700), (64, 1600, 515),
                                   (12, 1600, 9600), (64, 4128, 9600)])
def test_w4_sums_keep_their_bits(n, i, o, group):
    """The 2-norm of a product's error.  An instruction adds 16 exact products to a sum, each of
    the 17 cut at 2^-23 of the largest; with products of variance v the largest is about 4 sqrt(v),
    so the i / 16 instructions of a row leave (i / 16) (17 / 3) 2^-46 16 v in the mean square, or
    5.7 * 2^-46 of the result's i v; the i / 32 scaled additions leave i / 32 / 6 * 2^-48.  Twice the
    root of the two covers the scales' spread."""
    x = rnd(n + 1, n, i).bfloat16()
    codes, scale = random_w4(i, o, i, group)
    y = torch.empty(n, o, device="cuda")
    P.pkm_w4_matvec(x, codes, scale, y, group=group)
    want = x.double() @ R.values4(R.nibbles(codes), scale, group).t()
    off = ((y.double() - want).norm() / want.norm()).item()
    assert off <= 2 * 2.0 ** -23 * (5.7 + i / 768) ** 0.5


@pytest.mark.parametrize("n,i,f,o,group", [(1, 96, 160, 50, 32), (8, 1600, 704, 333, 64),
                                           (64, 640, 1056, 129, 96)])
def test_w4_block_writes_nothing_outside_its_buffers(n, i, f, o, group):
    packed = [random_w4(s, *shape, group) for s, shape in enumerate(((f, i), (f, i), (o, f)))]
    x, d, edge = rnd(n, n, i).bfloat16(), P.FfnDims(n, i, f, o), 1024
    need = P.pkm_ffn_workspace_bytes(d, P.PKM_FWD)
    raws = [torch.full((k + 2 * edge,), 0xA5, dtype=torch.uint8, device="cuda") for k in (2 * n * o, need)]
    y = raws[0][edge:edge + 2 * n * o].view(torch.bfloat16).view(n, o)
    P.pkm_w4_ffn(d, x, *packed, y, group=group, workspace=raws[1][edge:edge + need],
                 workspace_bytes=need)
    for raw, k in zip(raws, (2 * n * o, need)):
        assert (raw[:edge] == 0xA5).all() and (raw[edge + k:] == 0xA5).all()
    y2 = torch.empty_like(y)
    P.pkm_w4_ffn(d, x, *packed, y2, group=group, workspace=P.alloc_ffn_workspace(d, P.PKM_FWD))
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_checkpoint_halves_at_every_magnitude(dtype):
    """Runs from 1e-36 to 3e38 that hold their largest value's half (63.5 steps), its neighbours and
    other halves: the codes are those of 64 bits wherever 127 a still is a number and beyond."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    top = 10.0 ** torch.linspace(-36, 38.4, 6000, device="cuda", dtype=torch.float64)
    top = (top * (1 + torch.rand(6000, device="cuda", generator=gen, dtype=torch.float64))).clamp(max=3.3e38)
    top = top.to(dtype).float()
    odd = torch.randint(0, 127, (6000, 28), device="cuda", generator=gen) * 2 + 1
    v = (top.double()[:, None] * odd / 254).to(dtype).float()      # halves, to within a rounding
    half = (top / 2)[:, None]
    near = [torch.nextafter(half, half * s) for s in (0.5, 2.0)]
    x = torch.cat([top[:, None], half, *near, v], 1)
    x = (x * torch.where(torch.rand(x.shape, device="cuda", generator=gen) < 0.5, -1.0, 1.0)).to(dtype)
    codes, scale = pack(x)
    wc, ws = R.pack8(x)
    assert torch.equal(scale, ws)
    assert torch.equal(codes, wc)


@pytest.mark.parametrize("o", [300, 9600])
def test_w4_sums_depend_on_the_other_tokens_by_their_order_only(o):
    """A token's results have the same bits in calls of the same blocks of 8 tokens, whatever else
    is in the call, and between such groups differ by no more than two fp32 sums may."""
    i, group = 1600, 64
    x = rnd(6, 64, i).bfloat16()
    codes, scale = random_w4(3, o, i, group)
    W = R.values4(R.nibbles(codes), scale, group)
    bound = 2 * (i + 8) * R.E32 * (x.double().abs() @ W.abs().t())
    whole = torch.empty(64, o, device="cuda")
    P.pkm_w4_matvec(x, codes, scale, whole, group=group)
    for sizes in ((8, 1, 5), (16, 9, 13), (32, 17, 30), (64, 33, 50)):
        first = torch.empty(sizes[0], o, device="cuda")
        P.pkm_w4_matvec(x[:sizes[0]], codes, scale, first, group=group)
        assert ((first.double() - whole[:sizes[0]]).abs() <= bound[:sizes[0]]).all()
        for n in sizes[1:]:
            xs = x[:n].clone()
            xs[1:] = -xs[1:] * 3  # other tokens beside the first
            y = torch.empty(n, o, device="cuda")
            P.pkm_w4_matvec(xs, codes, scale, y, group=group)
            assert torch.equal(y[0], first[0])
