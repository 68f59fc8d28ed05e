"""Host-side behaviour of the gated feed-forward block, the 8-bit checkpoints and the 4-bit
products (no GPU): sizes, refusals before any device work, and the reference's own gradients
against differences."""
import ctypes

import pytest
import torch

from product_key_memory_pkm_b200 import build as B
from product_key_memory_pkm_b200 import pkm as P

from . import ffn_ref as R

FAKE = 1 << 20  # aligned, never dereferenced: every call below is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return P.load()


def _d(**kw):
    base = dict(N=64, d_in=64, d_ff=136, d_out=72)
    base.update(kw)
    return P.FfnDims(**base)


def test_struct_sizes():
    assert ctypes.sizeof(P.pkm_ffn_dims) == 32
    assert ctypes.sizeof(P.pkm_ffn_saved) == 4 * ctypes.sizeof(ctypes.c_void_p)
    assert ctypes.sizeof(P.pkm_w4) == 2 * ctypes.sizeof(ctypes.c_void_p)


def test_dims_can_be_copied_and_pickled():
    import copy
    import dataclasses
    import pickle
    d = _d(act=P.PKM_ACT_GELU)
    for e in (copy.deepcopy(d), pickle.loads(pickle.dumps(d))):
        assert e == d and P.pkm_ffn_saved_bytes(e, "g") == P.pkm_ffn_saved_bytes(d, "g")
    assert P.pkm_ffn_saved_bytes(dataclasses.replace(d, N=7), "g") == 7 * 136 * 2


def test_saved_and_workspace_sizes():
    d = _d()
    assert P.pkm_ffn_saved_bytes(d, "g") == 64 * 136 * 2
    assert P.pkm_ffn_saved_bytes(_d(flags=P.PKM_F_FP32), "u") == 64 * 136 * 4
    assert P.pkm_ffn_saved_bytes(d, "g_scale") == 0
    c8 = _d(flags=P.PKM_FFN_CKPT8)
    assert P.pkm_ffn_saved_bytes(c8, "g") == 64 * 160       # 136 columns in runs of 32
    assert P.pkm_ffn_saved_bytes(c8, "u_scale") == 64 * 5 * 4
    saved = P.alloc_ffn_saved(c8, device="cpu")
    for f in P.FFN_SAVED_FIELDS:
        assert saved[f].numel() * saved[f].element_size() == P.pkm_ffn_saved_bytes(c8, f)
    for which in (P.PKM_FWD, P.PKM_BWD):
        assert P.pkm_ffn_workspace_bytes(d, which) > 0
        assert P.pkm_ffn_workspace_bytes(_d(N=0), which) == 0
        assert P.pkm_ffn_workspace_bytes(_d(act=7), which) == 0
    assert P.pkm_ffn_workspace_bytes(d, P.PKM_FWD_FUSED) == 0


BAD_DIMS = [dict(N=-1), dict(d_in=0), dict(d_ff=-8), dict(d_out=0), dict(d_in=60), dict(d_ff=132),
            dict(d_out=71), dict(act=2), dict(act=-1), dict(flags=0x400), dict(flags=P.PKM_F_IDW),
            dict(flags=P.PKM_F_FP32 | P.PKM_FFN_GRAD_BF16)]


def _fwd(d, x=FAKE, y=FAKE, Wg=FAKE, Wd=FAKE, saved=None, ws=FAKE, wsb=1 << 30):
    s = None if saved is None else ctypes.byref(P.pkm_ffn_saved(*saved))
    return P.load().pkm_ffn_forward(ctypes.byref(d.c()), x, Wg, FAKE, Wd, y, s, ws, wsb, None)


def _bwd(d, saved=(FAKE, FAKE, None, None), dy=FAKE, dx=FAKE, dWg=FAKE, ws=FAKE, wsb=1 << 30):
    s = None if saved is None else ctypes.byref(P.pkm_ffn_saved(*saved))
    return P.load().pkm_ffn_backward(ctypes.byref(d.c()), FAKE, FAKE, FAKE, FAKE, s, dy, dx, dWg,
                                     None, None, ws, wsb, None)


@pytest.mark.parametrize("kw", BAD_DIMS)
def test_bad_dims_are_refused(kw):
    assert _fwd(_d(**kw)) == P.PKM_ERR_INVALID_ARG
    assert _bwd(_d(**kw)) == P.PKM_ERR_INVALID_ARG
    assert P.pkm_ffn_saved_bytes(_d(**kw), "g") == 0


def test_block_refusals():
    d, c8 = _d(), _d(flags=P.PKM_FFN_CKPT8)
    bad = P.PKM_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(x=FAKE + 2), dict(y=None), dict(Wg=FAKE + 8), dict(Wd=None),
               dict(saved=(None, FAKE, None, None)), dict(saved=(FAKE, FAKE + 4, None, None))):
        assert _fwd(d, **kw) == bad
    assert _fwd(c8, saved=(FAKE, FAKE, FAKE, None)) == bad   # 8-bit codes need both scales
    for kw in (dict(saved=None), dict(dy=None), dict(dx=FAKE + 4), dict(dWg=FAKE + 4)):
        assert _bwd(d, **kw) == bad
    assert _bwd(c8) == bad
    need = P.pkm_ffn_workspace_bytes(d, P.PKM_FWD)
    assert _fwd(d, ws=None) == P.PKM_ERR_WORKSPACE
    assert _fwd(d, wsb=need - 1) == P.PKM_ERR_WORKSPACE
    assert _fwd(d, ws=FAKE + 128) == P.PKM_ERR_WORKSPACE
    assert _bwd(d, wsb=P.pkm_ffn_workspace_bytes(d, P.PKM_BWD) - 1) == P.PKM_ERR_WORKSPACE
    assert _fwd(_d(d_ff=(1 << 20) + 8)) == P.PKM_ERR_UNSUPPORTED
    assert _fwd(_d(N=(1 << 26) + 1)) == P.PKM_ERR_UNSUPPORTED
    assert _fwd(_d(N=(1 << 26), d_ff=1 << 19)) == P.PKM_ERR_UNSUPPORTED
    assert _bwd(_d(N=(1 << 22) + 1, flags=P.PKM_F_FP32)) == P.PKM_ERR_UNSUPPORTED
    assert _fwd(_d(N=0), x=None, y=None, ws=None, wsb=0) == P.PKM_OK
    assert _bwd(_d(N=0), saved=None, dy=None, ws=None, wsb=0) == P.PKM_OK
    assert P.load().pkm_ffn_forward(None, *[FAKE] * 5, None, FAKE, 1 << 30, None) == bad


def test_checkpoint_refusals():
    L = P.load()
    for fn in (L.pkm_ckpt8_pack, L.pkm_ckpt8_unpack):
        assert fn(-1, 64, 0, FAKE, FAKE, FAKE, None) == P.PKM_ERR_INVALID_ARG
        assert fn(4, 0, 0, FAKE, FAKE, FAKE, None) == P.PKM_ERR_INVALID_ARG
        assert fn(4, 60, 0, FAKE, FAKE, FAKE, None) == P.PKM_ERR_INVALID_ARG
        assert fn(4, 64, P.PKM_F_SIMT, FAKE, FAKE, FAKE, None) == P.PKM_ERR_INVALID_ARG
        for i in range(3):
            for bad in (None, FAKE + 4):
                p = [FAKE] * 3
                p[i] = bad
                assert fn(4, 64, 0, *p, None) == P.PKM_ERR_INVALID_ARG
        assert fn(0, 64, 0, None, None, None, None) == P.PKM_OK


def test_w4_refusals():
    L = P.load()
    W = P.pkm_w4(FAKE, FAKE)

    def mv(N=4, d_in=64, d_out=72, group=64, x=FAKE, w=W, y=FAKE):
        return L.pkm_w4_matvec(N, d_in, d_out, group, x, None if w is None else ctypes.byref(w),
                               y, None)

    bad = P.PKM_ERR_INVALID_ARG
    for kw in (dict(N=-1), dict(d_in=48), dict(d_in=0), dict(d_out=0), dict(group=0),
               dict(group=-32), dict(group=48), dict(x=None), dict(y=FAKE + 4), dict(w=None),
               dict(w=P.pkm_w4(FAKE + 8, FAKE)), dict(w=P.pkm_w4(FAKE, None))):
        assert mv(**kw) == bad, kw
    assert mv(N=P.PKM_W4_MAX_TOKENS + 1) == P.PKM_ERR_UNSUPPORTED
    assert mv(d_out=(1 << 20) + 1) == P.PKM_ERR_UNSUPPORTED
    assert mv(N=0, x=None, y=None) == P.PKM_OK
    assert L.pkm_w4_pack(8, 48, 32, FAKE, FAKE, FAKE, None) == bad
    assert L.pkm_w4_pack(8, 64, 32, None, FAKE, FAKE, None) == bad
    assert L.pkm_w4_unpack(8, 64, 32, ctypes.byref(W), None, None) == bad

    def ffn(d, group=64, ws=FAKE, wsb=1 << 30, wd=W):
        return L.pkm_w4_ffn(ctypes.byref(d.c()), group, FAKE, ctypes.byref(W), ctypes.byref(W),
                            ctypes.byref(wd), FAKE, ws, wsb, None)

    d = _d(N=8, d_ff=96)
    assert ffn(_d(N=8, d_ff=136)) == bad             # d_ff not a multiple of 32
    assert ffn(_d(N=8, d_ff=96, flags=P.PKM_F_FP32)) == bad
    assert ffn(_d(N=65, d_ff=96)) == P.PKM_ERR_UNSUPPORTED
    assert ffn(d, group=16) == bad
    assert ffn(d, wd=P.pkm_w4(None, FAKE)) == bad
    assert ffn(d, wsb=16) == P.PKM_ERR_WORKSPACE
    assert ffn(_d(N=0, d_ff=96), ws=None, wsb=0) == P.PKM_OK


def _apart(*names):
    """Addresses far enough apart for every buffer of the small calls below."""
    return {n: (i + 1) << 24 for i, n in enumerate(names)}


FWD = ("x", "Wg", "Wu", "Wd", "y", "g", "u", "sg", "su", "ws")
BWD = FWD[:4] + ("g", "u", "sg", "su", "dy", "dx", "dWg", "dWu", "dWd", "ws")


def _call_block(L, d, a, which):
    s = ctypes.byref(P.pkm_ffn_saved(a["g"], a["u"], a["sg"], a["su"]))
    if which == P.PKM_FWD:
        return L.pkm_ffn_forward(ctypes.byref(d.c()), *(a[k] for k in FWD[:5]), s, a["ws"],
                                 1 << 20, None)
    return L.pkm_ffn_backward(ctypes.byref(d.c()), *(a[k] for k in FWD[:4]), s,
                              *(a[k] for k in BWD[8:13]), a["ws"], 1 << 20, None)


@pytest.mark.parametrize("flags", [0, P.PKM_FFN_CKPT8, P.PKM_F_FP32])
@pytest.mark.parametrize("which", [P.PKM_FWD, P.PKM_BWD])
def test_outputs_that_share_bytes_are_refused(which, flags):
    """Every output against every other buffer: the same address, and the last bytes only."""
    d = _d(flags=flags)
    names, outs = (FWD, FWD[4:]) if which == P.PKM_FWD else (BWD, BWD[9:])
    scales = ("sg", "su")
    esz = 4 if flags & P.PKM_F_FP32 else 2
    size = dict(x=64 * 64 * esz, y=64 * 72 * esz, dy=64 * 72 * esz, dx=64 * 64 * esz,
                Wg=136 * 64 * esz, Wu=136 * 64 * esz, Wd=72 * 136 * esz, dWg=136 * 64 * 4,
                dWu=136 * 64 * 4, dWd=72 * 136 * 4, ws=P.pkm_ffn_workspace_bytes(d, which),
                g=P.pkm_ffn_saved_bytes(d, "g"), u=P.pkm_ffn_saved_bytes(d, "u"),
                sg=P.pkm_ffn_saved_bytes(d, "g_scale"), su=P.pkm_ffn_saved_bytes(d, "u_scale"))
    L = P.load()
    for o in outs:
        for n in names:
            if n == o or not flags & P.PKM_FFN_CKPT8 and (n in scales or o in scales):
                continue
            a = _apart(*names)
            assert _call_block(L, d, {**a, o: a[n]}, which) == P.PKM_ERR_INVALID_ARG, (o, n)
            if o != "ws":  # whose alignment is larger
                last = a[n] + (size[n] - 1) // 16 * 16
                assert _call_block(L, d, {**a, o: last}, which) == P.PKM_ERR_INVALID_ARG, (o, n)
    if not torch.cuda.is_available():
        # tied weights and neighbouring buffers pass the checks (and end where a GPU is needed)
        a = _apart(*names)
        assert _call_block(L, d, {**a, "Wu": a["Wg"]}, which) == P.PKM_ERR_CUDA
        for o in set(outs) - {"ws"}:
            for n in set(names) - {o}:
                nxt = a[n] + (size[n] + 15) // 16 * 16
                assert _call_block(L, d, {**a, o: nxt}, which) == P.PKM_ERR_CUDA, (o, n)


def test_packing_and_products_in_place_are_refused():
    L, bad = P.load(), P.PKM_ERR_INVALID_ARG
    a, b, c, e = ((i + 1) << 24 for i in range(4))
    for p in ((a, a, b), (a, b, a), (a, b, b), (a, a + 16, b)):
        assert L.pkm_ckpt8_pack(4, 64, 0, *p, None) == bad
        assert L.pkm_w4_pack(8, 64, 32, *p, None) == bad
    for p in ((a, b, a), (a, b, b), (a, b, a + 16)):
        assert L.pkm_ckpt8_unpack(4, 64, 0, *p, None) == bad
        assert L.pkm_w4_unpack(8, 64, 32, ctypes.byref(P.pkm_w4(*p[:2])), p[2], None) == bad
    for x, y in ((a, a), (a, b), (a, c), (a, a + 16)):
        assert L.pkm_w4_matvec(4, 64, 8, 32, x, ctypes.byref(P.pkm_w4(b, c)), y, None) == bad
    d, W = _d(N=8, d_ff=96), ctypes.byref(P.pkm_w4(b, c))
    for y, ws in ((a, e), (b, e), (c, e), (e, e), (e, a), (e, b), (e, c)):
        assert L.pkm_w4_ffn(ctypes.byref(d.c()), 32, a, W, W, W, y, ws, 1 << 20, None) == bad


def test_workspace_bytes_beyond_the_tensor_are_refused():
    class Anywhere(P._Checked):
        __slots__ = ()

        def place(self, t, name):
            pass

    ws = torch.empty(256, dtype=torch.uint8)
    assert Anywhere().workspace(ws, 128) == (ws.data_ptr(), 128)
    with pytest.raises(ValueError, match="256 bytes"):
        Anywhere().workspace(ws, 512)


def test_binding_checks_its_tensors():
    """Wrong type, shape, order or place is refused before the library is called."""
    d = _d(N=2)
    t = dict(x=torch.zeros(2, 64), Wg=torch.zeros(136, 64), Wu=torch.zeros(136, 64),
             Wd=torch.zeros(72, 136), y=torch.zeros(2, 72))
    with pytest.raises(TypeError):
        P.pkm_ffn_forward(d, **t)                                  # fp32 for bf16
    t = {k: v.bfloat16() for k, v in t.items()}
    with pytest.raises(ValueError, match="not on a GPU"):
        P.pkm_ffn_forward(d, **t)
    with pytest.raises(ValueError, match="shape"):
        P.pkm_ffn_forward(d, **{**t, "x": t["x"][:1]})
    with pytest.raises(ValueError, match="missing"):
        P.pkm_ffn_forward(d, **{**t, "x": None})
    with pytest.raises(ValueError, match="contiguous"):
        P.pkm_ffn_forward(d, **{**t, "x": torch.zeros(64, 2).bfloat16().t()})
    with pytest.raises(TypeError):
        P.pkm_ckpt8_pack(torch.zeros(2, 64, dtype=torch.float16), *P.alloc_ckpt8(2, 64, "cpu"))
    with pytest.raises(ValueError):
        P.pkm_w4_matvec(t["x"], *P.alloc_w4(72, 64, 64, "cpu"), torch.zeros(2, 72))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_gradients_against_differences(act):
    """The formulas every kernel is held to are the derivatives of the forward's formula."""
    gen = torch.Generator().manual_seed(3)
    n, di, f, do = 5, 8, 16, 8
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    t = dict(x=mk(n, di), Wg=mk(f, di), Wu=mk(f, di), Wd=mk(do, f))
    dy = mk(n, do)
    fw = R.forward(act, **t, r=0.0)
    gr = R.backward(act, *t.values(), fw["g"][0], fw["u"][0], dy, 0.0)
    eps = 1e-5
    for name, grad in (("x", "dx"), ("Wg", "dWg"), ("Wu", "dWu"), ("Wd", "dWd")):
        v = mk(*t[name].shape)
        side = [(R.forward(act, **{**t, name: t[name] + s * eps * v}, r=0.0)["y"][0] * dy).sum()
                for s in (1, -1)]
        diff = (side[0] - side[1]) / (2 * eps)
        # the difference's own error: eps^2 times the third derivative (order 1e3 here at most)
        assert abs((diff - (gr[grad][0] * v).sum()).item()) <= 1e-7 * (1 + abs(diff.item()))


def test_kernels_that_wait_for_their_producer_take_no_restrict_pointers():
    """A kernel of the block that starts before its producer has ended reads what that one is still
    writing.  Loads of a __restrict__ pointer to const may take the read-only path, which allows no
    such writer, and need not stay behind the wait."""
    import os
    import re
    seen = []
    for name in ("k_few.cu", "k_ffn_simt.cu", "k_ffn_tc.cu"):
        with open(os.path.join(B.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in text.split("__global__")[1:]:
            head, body = kernel.split("{", 1)
            body = body.split("\n}\n", 1)[0]
            if "grid_dependency_wait()" in body:
                seen.append(re.findall(r"(\w+)\s*\(", head)[-1])
                assert "__restrict__" not in head, seen[-1]
    assert seen == ["few_kernel", "small_jobs_kernel", "sum_parts_kernel"]


def test_sizes_beyond_the_librarys_integers_are_refused(monkeypatch):
    """ctypes passes the low bits of what does not fit: a group of 2^32 + 64 as 64, so that the
    kernels would read more scales than the caller's tensor holds."""
    for kw in (dict(N=1 << 64), dict(d_in=(1 << 32) + 64), dict(d_ff=(1 << 31)), dict(d_out=-1 << 32),
               dict(act=1 << 32), dict(flags=1 << 32), dict(flags=-1)):
        with pytest.raises(ValueError, match="beyond the library's integers"):
            _d(**kw)

    class Anywhere(P._Checked):
        __slots__ = ()

        def place(self, t, name):
            pass

        def stream(self, stream):
            return None

    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or P.PKM_OK

    monkeypatch.setattr(P, "_Checked", Anywhere)
    monkeypatch.setattr(P, "load", Library)
    big = (1 << 32) + 64

    def t(*shape, dtype=torch.bfloat16):  # no memory behind it
        return torch.empty(*shape, dtype=dtype, device="meta")

    def w4(o, i, group):
        return P.alloc_w4(o, i, group, "meta")

    d = _d(N=2, d_ff=96, d_out=64)
    f32 = torch.float32
    P.pkm_w4_matvec(t(2, 64), *w4(8, 64, 64), t(2, 8, dtype=f32))
    assert calls == ["pkm_w4_matvec"]  # a call in range goes through
    calls.clear()
    for call in (
            lambda: P.pkm_w4_matvec(t(2, 128), *w4(8, 128, big), t(2, 8, dtype=f32), group=big),
            lambda: P.pkm_w4_matvec(t(2, big), *w4(8, big, 64), t(2, 8, dtype=f32)),
            lambda: P.pkm_w4_matvec(t(2, 64), *w4(big, 64, 64), t(2, big, dtype=f32)),
            lambda: P.pkm_w4_pack(t(8, 128), *w4(8, 128, big), group=big),
            lambda: P.pkm_w4_pack(t(8, big), *w4(8, big, 64)),
            lambda: P.pkm_w4_pack(t(big, 64), *w4(big, 64, 64)),
            lambda: P.pkm_w4_unpack(*w4(8, 128, big), t(8, 128), group=big),
            lambda: P.pkm_w4_unpack(*w4(big, 64, 64), t(big, 64)),
            lambda: P.pkm_w4_ffn(d, t(2, 64), w4(96, 64, big), w4(96, 64, big), w4(64, 96, big),
                                 t(2, 64), group=big),
            lambda: P.pkm_ckpt8_pack(t(2, big), *P.alloc_ckpt8(2, big, "meta")),
            lambda: P.pkm_ckpt8_unpack(*P.alloc_ckpt8(2, big, "meta"), t(2, big, dtype=f32))):
        with pytest.raises(ValueError, match="beyond the library's integers"):
            call()
    assert not calls


def test_negative_workspace_sizes_are_refused():
    """size_t makes -1 the largest size there is: every workspace would look large enough."""
    class Anywhere(P._Checked):
        __slots__ = ()

        def place(self, t, name):
            pass

    for ws in (torch.empty(256, dtype=torch.uint8), FAKE):
        with pytest.raises(ValueError, match="workspace_bytes"):
            Anywhere().workspace(ws, -1)
    assert Anywhere().workspace(FAKE, 64) == (FAKE, 64)
