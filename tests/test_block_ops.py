"""The operators around the experts' products without a GPU: the C entry
points and the Python calls refuse what they cannot do before anything is
launched, and the 64-bit forms that the GPU tests compare with hold against
differences."""
import ctypes as C

import pytest
import torch

import block_reference as ref
import swiglu_mlp_top_gb300 as mm
from swiglu_mlp_top_gb300 import _lib as L

F = C.c_void_p(1 << 20)           # never dereferenced: validation fails first
ODD = C.c_void_p((1 << 20) + 2)
BF, F32 = L.MM_DTYPE_BF16, L.MM_DTYPE_F32
BAD, UNS, WS, OK = L.MM_ERR_INVALID_ARG, L.MM_ERR_UNSUPPORTED, L.MM_ERR_WORKSPACE, L.MM_OK


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return L.load()


def norm(lib, x=F, f=F, post=F, gate=F, per_token=0, pre=F, s=1.0, eps=1e-5, T=10, H=768, dt=BF, r=F, n=F, sp=F, sr=F):
    return lib.mm_block_norm(x, f, post, gate, per_token, pre, s, eps, T, H, dt, r, n, sp, sr, None)


def test_block_norm_refusals(lib):
    for kw in (dict(dt=7), dict(T=-1), dict(H=0), dict(x=None), dict(x=ODD), dict(r=None), dict(n=None), dict(pre=None, sr=None),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(s=float("nan")),
               dict(post=None), dict(f=None), dict(f=None, r=None, post=None, sp=None), dict(post=ODD), dict(gate=ODD),
               dict(sp=ODD), dict(f=None, r=None, post=None, sp=None, gate=None, s=0.5)):
        assert norm(lib, **kw) == BAD, kw
    assert norm(lib, H=L.MM_NORM_MAX_H + 1) == UNS
    assert norm(lib, T=0, x=None, f=None) == OK


def norm_bwd(lib, dn=F, dr=F, r=F, f=F, post=F, gate=F, per_token=0, pre=F, sp=F, sr=F, s=1.0, T=10, H=768, dt=BF, dx=F, df=F,
             dpost=F, dgate=F, dpre=F, ws=F, wsb=1 << 34):
    return lib.mm_block_norm_backward(dn, dr, r, f, post, gate, per_token, pre, sp, sr, s, T, H, dt, dx, df, dpost, dgate, dpre,
                                      ws, wsb, None)


def test_block_norm_backward_refusals(lib):
    for kw in (dict(dt=7), dict(T=-1), dict(H=0), dict(dx=None), dict(dn=None), dict(r=None), dict(f=None), dict(df=None),
               dict(sp=None), dict(sr=None), dict(dpost=None), dict(dgate=None), dict(dpre=None), dict(post=None),
               dict(gate=None), dict(pre=None), dict(dn=ODD), dict(df=ODD), dict(dpre=ODD), dict(sr=ODD), dict(s=float("inf")),
               dict(pre=None, dpre=None, dn=None, dr=None)):
        assert norm_bwd(lib, **kw) == BAD, kw
    assert norm_bwd(lib, H=L.MM_NORM_MAX_H + 1) == UNS
    if lib.mm_block_norm_backward_workspace_bytes(10000, 768, BF):                # several blocks: there is a GPU
        assert norm_bwd(lib, T=10000, wsb=10) == WS and norm_bwd(lib, T=10000, ws=None) == WS and norm_bwd(lib, T=10000, ws=ODD) == WS
    assert lib.mm_block_norm_backward_workspace_bytes(10, 768, 7) == 0
    assert lib.mm_block_norm_backward_workspace_bytes(10, L.MM_NORM_MAX_H + 1, BF) == 0
    assert lib.mm_block_norm_backward_workspace_bytes(0, 768, BF) == 0            # none needed


def test_permute_refusals(lib):
    def call(x=F, idx=F, T=10, H=64, E=4, k=2, align=1, dt=BF, xs=F, off=F, cnt=F, perm=F, pos=F, ws=F, wsb=1 << 34):
        return lib.mm_moe_permute(x, idx, T, H, E, k, align, dt, xs, off, cnt, perm, pos, ws, wsb, None)
    for kw in (dict(dt=7), dict(T=-1), dict(H=0), dict(E=0), dict(k=0), dict(align=0), dict(x=None), dict(x=ODD), dict(idx=None),
               dict(xs=None), dict(off=None), dict(cnt=None), dict(perm=None), dict(pos=None), dict(pos=ODD)):
        assert call(**kw) == BAD, kw
    for kw in (dict(E=65), dict(k=9), dict(align=1025), dict(T=1 << 30), dict(H=L.MM_PERMUTE_MAX_H + 1)):
        assert call(**kw) == UNS, kw
    assert call(T=5000, ws=None) == WS and call(T=5000, wsb=0) == WS and call(T=5000, ws=ODD) == WS
    assert lib.mm_moe_permute_workspace_bytes(10, 4, 2) == 0                      # none needed
    assert lib.mm_moe_permuted_rows(10, 4, 2, 8) == 20 + 4 * 7
    assert lib.mm_moe_permuted_rows(1, 64, 2, 8) == 2 + 2 * 7          # no more groups than assignments
    assert lib.mm_moe_permuted_rows(0, 4, 2, 8) == 0
    assert lib.mm_moe_permuted_rows(10, 65, 2, 8) == -1 and lib.mm_moe_permuted_rows(1 << 30, 4, 2, 8) == -1
    assert lib.mm_moe_permute_workspace_bytes(10, 65, 2) == 0

    def back(ys=F, pos=F, w=F, T=10, H=64, k=2, rows=20, dt=BF, y=F):
        return lib.mm_moe_unpermute(ys, pos, w, T, H, k, rows, dt, y, None)
    for kw in (dict(dt=7), dict(T=-1), dict(H=0), dict(k=0), dict(rows=-1), dict(ys=None), dict(pos=None), dict(y=None), dict(w=ODD)):
        assert back(**kw) == BAD, kw
    assert back(k=9) == UNS and back(H=L.MM_PERMUTE_MAX_H + 1) == UNS and back(T=0, y=None) == OK

    def grad(dy=F, ys=F, pos=F, w=F, off=F, cnt=F, T=10, H=64, E=4, k=2, rows=20, dt=BF, dys=F, dw=F):
        return lib.mm_moe_unpermute_backward(dy, ys, pos, w, off, cnt, T, H, E, k, rows, dt, dys, dw, None)
    for kw in (dict(dt=7), dict(T=-1), dict(H=0), dict(E=0), dict(k=0), dict(rows=-1), dict(dy=None), dict(ys=None),
               dict(pos=None), dict(off=None), dict(cnt=None), dict(dys=None), dict(w=None), dict(dys=ODD), dict(dw=ODD)):
        assert grad(**kw) == BAD, kw
    assert grad(k=9) == UNS and grad(E=65) == UNS and grad(H=L.MM_PERMUTE_MAX_H + 1) == UNS and grad(T=0, dy=None) == OK


def test_checkpoint_refusals(lib):
    for fn, order in ((lib.mm_checkpoint_pack, lambda x, c, e, R, C, dt: (x, R, C, dt, c, e, None)),
                      (lib.mm_checkpoint_unpack, lambda x, c, e, R, C, dt: (c, e, R, C, dt, x, None))):
        def call(x=F, c=F, e=F, R=4, C=64, dt=BF):
            return fn(*order(x, c, e, R, C, dt))
        for kw in (dict(dt=7), dict(R=-1), dict(C=0), dict(x=None), dict(c=None), dict(e=None), dict(x=ODD), dict(c=ODD), dict(e=ODD)):
            assert call(**kw) == BAD, kw
        assert call(C=L.MM_CHECKPOINT_MAX_COLS + 1) == UNS and call(R=1 << 40) == UNS and call(R=0, x=None) == OK

    def act(gu=F, R=4, I=64, dt=BF, rows=F, h=F, c=F, e=F):
        return lib.mm_swiglu_act(gu, R, I, dt, rows, h, c, e, None)
    for kw in (dict(dt=7), dict(R=-1), dict(I=0), dict(gu=None), dict(h=None), dict(c=None), dict(e=None), dict(rows=ODD), dict(c=ODD)):
        assert act(**kw) == BAD, kw
    assert act(I=L.MM_CHECKPOINT_MAX_COLS // 2 + 1) == UNS and act(R=0, gu=None) == OK

    def act_bwd(c=F, e=F, dh=F, R=4, I=64, dt=BF, rows=F, dgu=F, h=F):
        return lib.mm_swiglu_act_backward(c, e, dh, R, I, dt, rows, dgu, h, None)
    for kw in (dict(dt=7), dict(R=-1), dict(I=0), dict(c=None), dict(e=None), dict(dh=None), dict(dgu=None), dict(h=ODD)):
        assert act_bwd(**kw) == BAD, kw
    assert act_bwd(I=L.MM_CHECKPOINT_MAX_COLS // 2 + 1) == UNS and act_bwd(R=0, c=None) == OK


def test_python_calls_refuse_what_is_not_on_the_gpu():
    x, idx = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    plan = {"pos": idx, "counts": idx[0], "offsets": idx[0], "perm": idx[0]}
    ck = {"codes": x.to(torch.float8_e4m3fn), "exps": torch.zeros(4, 2, dtype=torch.uint8), "segments": 2}
    for call in (lambda: mm.block_norm(x, x), lambda: mm.block_norm_backward(None, x, None, x, None),
                 lambda: mm.moe_permute(x, idx, 4), lambda: mm.moe_unpermute(x, plan, idx.float()),
                 lambda: mm.moe_permute_backward(x, plan), lambda: mm.moe_unpermute_backward(x, x, plan, idx.float()),
                 lambda: mm.checkpoint_pack(x), lambda: mm.checkpoint_unpack(ck), lambda: mm.swiglu_act(x),
                 lambda: mm.swiglu_act_backward(ck, x[:, :32])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_a_gradient_without_its_output_is_refused():
    """dn belongs to the norm behind r; without that norm it must not be dropped in silence."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dn needs pre_weight"):
        mm.block_norm_backward(x, x, x, x, None)


# ---------------------------------- the 64-bit forms against differences
D = 2.0 ** -14
# a central difference is off by D^2 / 6 times a third derivative (a few
# hundred times the terms at most) and by roundings of 2^-52 over D
SLOPE = 512 * D * D + 2.0 ** -34


def test_norm_gradient_against_differences():
    gen = torch.Generator().manual_seed(0)
    T, H, s, eps = 6, 20, 0.9, 1e-5
    rand = lambda *shape: torch.randn(*shape, generator=gen, dtype=torch.float64)  # noqa: E731
    for per_token in (False, True):
        p = dict(x=rand(T, H), f=rand(T, H), post=1 + 0.1 * rand(H), gate=rand(T, H) if per_token else rand(H), pre=1 + 0.1 * rand(H))
        dn, dr = rand(T, H), rand(T, H)

        def loss(q):
            o = ref.norm_forward(q["x"], q["f"], q["post"], q["gate"], q["pre"], s, eps)
            return (o["r"] * dr).sum() + (o["n"] * dn).sum()

        o = ref.norm_forward(p["x"], p["f"], p["post"], p["gate"], p["pre"], s, eps)
        got = ref.norm_backward(dn, dr, o["r"], p["f"], p["post"], p["gate"], p["pre"], s, o["rstd_post"], o["rstd_pre"])
        size = (o["r"] * dr).abs().sum() + (o["n"] * dn).abs().sum()
        for name, key in (("x", "dx"), ("f", "df"), ("post", "d_post_weight"), ("gate", "d_gate"), ("pre", "d_pre_weight")):
            way = rand(*p[name].shape)
            slope = (loss(dict(p, **{name: p[name] + D * way})) - loss(dict(p, **{name: p[name] - D * way}))) / (2 * D)
            assert abs(slope - (got[key] * way).sum()) <= SLOPE * size, name


def test_swiglu_gradient_against_differences():
    gen = torch.Generator().manual_seed(9)
    g, u, dh = (torch.randn(40, 64, generator=gen, dtype=torch.float64) * 3 for _ in range(3))
    dG, dU, _ = ref.swiglu_backward(g, u, dh)
    num = (ref.swiglu(g + D, u) - ref.swiglu(g - D, u)) / (2 * D) * dh
    assert bool(((num - dG).abs() <= SLOPE * (1 + g.abs()) * (u * dh).abs()).all())
    num = (ref.swiglu(g, u + D) - ref.swiglu(g, u - D)) / (2 * D) * dh
    assert bool(((num - dU).abs() <= SLOPE * (1 + u.abs()) * (g * dh).abs()).all())


def test_e4m3_values_are_the_formats():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(codes.float().double(), ref.E4M3)
    v = (torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 60).clamp(-448, 448)
    assert torch.equal(ref.nearest_e4m3(v.double()), v.to(torch.float8_e4m3fn).double())
