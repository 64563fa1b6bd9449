"""block_norm and its gradient against the 64-bit forms of block_reference.

Bounds: r = s x + g p is at most 8 roundings from its inputs besides rho, whose
mean of squares is a sum of H positive terms: a thread adds at most 64 of them,
the tree and the block at most 16 more, and the square root halves what is left
of it: (80 / 2 + 3) + 8 < 64 roundings.  The gradients hold one such sum more
(c, over the same H terms, whose error counts on the terms' magnitudes): 2 * 80
+ 16 < 192; df holds two: 384.  A column's sum over T tokens: T more.
"""
import pytest
import torch

import block_reference as ref
import swiglu_mlp_top_gb300 as mm
from block_reference import U, U32, close

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


def make(T, H, dtype, post=True, gate="channel", pre=True, seed=0, branch=True):
    gen = torch.Generator().manual_seed(1000 * T + H + seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen) * std + mean).to(dtype).cuda()

    return dict(x=normal(T, H, std=2.0), f=normal(T, H, std=0.5) if branch else None,
                post=normal(H, std=0.1, mean=1.0) if post and branch else None,
                gate=None if gate is None or not branch else normal(*((T, H) if gate == "token" else (H,)), std=0.3, mean=0.5),
                pre=normal(H, std=0.1, mean=1.0) if pre else None,
                dn=normal(T, H, std=0.05) if pre else None, dr=normal(T, H, std=0.02))


def forward(d, s=1.0, **kw):
    stats = {}
    r, n = mm.block_norm(d["x"], d["f"], post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"],
                         residual_scale=s, eps=EPS, stats=stats, **kw)
    return r, n, stats


def backward(d, r, stats, s=1.0, dr=True, **kw):
    return mm.block_norm_backward(d["dn"], d["dr"] if dr else None, r, d["f"], stats, post_weight=d["post"],
                                  gate=d["gate"], pre_weight=d["pre"], residual_scale=s, **kw)


def check_forward(d, r, n, stats, s=1.0):
    u = U[d["x"].dtype]
    want = ref.norm_forward(d["x"], d["f"], d["post"], d["gate"], d["pre"], s, EPS, r_stored=r)
    if d["f"] is not None:
        close(r, want["r"], u * want["r"].abs() + (u + 1) * 64 * U32 * want["r_terms"], "r")
    for key in ("rstd_post", "rstd_pre"):
        assert (key in want) == (key in stats)
        if key in want:
            close(stats[key], want[key], 64 * U32 * want[key], key)
    if d["pre"] is None:
        assert n is None
    else:
        close(n, want["n"], (u + (u + 1) * 64 * U32) * want["n"].abs(), "n")


def check_backward(d, r, stats, got, s=1.0, dr=True):
    u, T = U[d["x"].dtype], d["x"].shape[0]
    want = ref.norm_backward(d["dn"], d["dr"] if dr else None, r, d["f"], d["post"], d["gate"], d["pre"], s,
                             stats.get("rstd_post"), stats.get("rstd_pre"))
    keys = [k for k in want if not k.endswith("_terms")]
    assert sorted(got) == sorted(keys)
    for k in keys:
        terms = want[k + "_terms"]
        if got[k].dim() == 1:                                   # fp32 sums over the tokens
            bound = (384 + T) * U32 * terms
        else:
            bound = u * want[k].abs() + (u + 1) * 384 * U32 * terms
        close(got[k], want[k], bound, k)


SHAPES = [(1, 768), (1, 1), (3, 8), (5, 7), (33, 64), (70, 1000), (129, 1001), (200, 2432), (17, 4096), (9, 8192), (7, 8191), (6, 4097),
          (5, 16384), (3, 16383), (1500, 768), (2100, 96)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_all_parts(T, H, dtype):
    d = make(T, H, dtype)
    r, n, stats = forward(d, s=0.9)
    check_forward(d, r, n, stats, s=0.9)
    check_backward(d, r, stats, backward(d, r, stats, s=0.9), s=0.9)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("T,H", [(37, 768), (6, 1001), (700, 200)])
def test_parts_left_out(T, H, post, gate, pre, dtype):
    d = make(T, H, dtype, post, gate, pre)
    r, n, stats = forward(d, s=-0.5)
    check_forward(d, r, n, stats, s=-0.5)
    check_backward(d, r, stats, backward(d, r, stats, s=-0.5), s=-0.5)
    if pre:
        check_backward(d, r, stats, backward(d, r, stats, s=-0.5, dr=False), s=-0.5, dr=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 768), (50, 320), (4, 333)])
def test_plain_norm(T, H, dtype):
    d = make(T, H, dtype, branch=False)
    r, n, stats = forward(d)
    assert r is d["x"]
    check_forward(d, r, n, stats)
    check_backward(d, r, stats, backward(d, r, stats))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,post,gate,pre,branch", [
    (20000, 256, True, "channel", True, True), (9733, 8, True, "token", True, True), (9999, 24, False, None, True, True),
    (10001, 40, True, None, False, True), (12345, 768, False, "channel", True, True), (10000, 64, True, "channel", True, False),
    (3000, 2432, True, "token", False, True), (5003, 1000, True, "channel", True, True), (640, 6528, True, "channel", True, True), (1300, 8192, False, None, True, True), (700, 8192, True, "token", True, True),
    (650, 12288, True, None, True, True), (40, 12288, True, "token", True, True), (11000, 33, True, "channel", True, True)])
def test_many_tokens(T, H, post, gate, pre, branch, dtype):
    d = make(T, H, dtype, post, gate, pre, branch=branch)
    r, n, stats = forward(d, s=0.9 if branch else 1.0)
    check_forward(d, r, n, stats, s=0.9 if branch else 1.0)
    check_backward(d, r, stats, backward(d, r, stats, s=0.9 if branch else 1.0), s=0.9 if branch else 1.0)


@pytest.mark.parametrize("dtype,T,H", [(BF, 40, 768), (F32, 40, 101), (BF, 10000, 96)])
def test_in_place(dtype, T, H):
    d = make(T, H, dtype)
    r, n, stats = forward(d)
    x, f = d["x"].clone(), d["f"].clone()
    r2, n2 = mm.block_norm(x, f, post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"], eps=EPS, out=x, normed=f)
    assert r2 is x and n2 is f and torch.equal(x, r) and torch.equal(f, n)


def test_a_bad_row_stays_alone_and_zeros_are_fine():
    d = make(64, 768, BF)
    d["x"][9] = 0
    d["f"][9] = 0
    r, n, stats = forward(d)
    check_forward(d, r, n, stats)
    assert not n[9].any() and abs(stats["rstd_pre"][9].item() - EPS ** -0.5) <= 64 * U32 * EPS ** -0.5
    clean = backward(d, r, stats)
    check_backward(d, r, stats, clean)
    for bad in (float("nan"), float("inf"), -float("inf")):
        e = dict(d, x=d["x"].clone(), f=d["f"].clone())
        e["x"][5, 3] = bad
        e["f"][7, 11] = bad
        r2, n2, _ = forward(e)
        keep = [i for i in range(64) if i not in (5, 7)]
        assert torch.equal(r2[keep], r[keep]) and torch.equal(n2[keep], n[keep])
        assert not n2[5].isfinite().all() and not n2[7].isfinite().all()
        # the gradient's rows too (its sums hold every row)
        r3 = r.clone()
        r3[5, 3] = bad
        got = backward(d, r3, stats)
        assert torch.equal(got["dx"][keep], clean["dx"][keep]) and torch.equal(got["df"][keep], clean["df"][keep])


def test_no_tokens():
    d = make(0, 768, BF)
    d["gate"][3], d["post"][4] = float("inf"), float("nan")
    r, n, stats = forward(d)
    assert r.shape == n.shape == (0, 768)
    got = backward(d, r, stats)
    for k in ("d_post_weight", "d_gate", "d_pre_weight"):
        assert got[k].shape == (768,) and not got[k].any()


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (True, True)])
def test_rows_of_several_warps_many_times(post, pre):
    """Sums of consecutive rows go through the same few words of shared memory:
    one or two sums a row, the same bits every time."""
    d = make(6000, 2048, BF, post=post, pre=pre)
    r, n, stats = forward(d)
    check_forward(d, r, n, stats)
    for _ in range(20):
        r2, n2, stats2 = forward(d)
        assert torch.equal(r, r2) and (n is None or torch.equal(n, n2)) and all(torch.equal(stats[k], stats2[k]) for k in stats)


def test_same_bits_every_time():
    d = make(3000, 768, BF)
    r, n, stats = forward(d)
    a, b = backward(d, r, stats), backward(d, r, stats)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradient_against_differences():
    """Along a random direction, (L(+h) - L(-h)) / 2h of the fp32 forward for
    L = <r, dr> + <n, dn>.  L's own rounding: its sums are taken in 64 bits of
    values each 64 roundings off, so at most 64 * 2^-24 * sum of |terms|, over
    h; the difference itself is off by h^2 / 6 times a third derivative, which
    for rows of unit scale and a direction of length one per element is of the
    size of the terms: h = 2^-7 gives 2^-17."""
    d = make(24, 768, F32, seed=5)
    r, n, stats = forward(d, s=0.9)
    grads = backward(d, r, stats, s=0.9)
    gen = torch.Generator().manual_seed(3)
    h = 2.0 ** -7
    for name, key in (("x", "dx"), ("f", "df"), ("post", "d_post_weight"), ("gate", "d_gate"), ("pre", "d_pre_weight")):
        way = torch.randn(d[name].shape, generator=gen).cuda()

        def loss(sign):
            e = dict(d, **{name: d[name] + sign * h * way})
            r, n, _ = forward(e, s=0.9)
            return (r.double() * d["dr"]).sum() + (n.double() * d["dn"]).sum()

        terms = ((r.double() * d["dr"]).abs().sum() + (n.double() * d["dn"]).abs().sum()).item()
        slope = ((loss(1) - loss(-1)) / (2 * h)).item()
        want = (grads[key].double() * way).sum().item()
        assert abs(slope - want) <= (64 * U32 / h + 2.0 ** -17) * terms, (name, slope, want, terms)


def test_more_elements_than_32_bits_count():
    """Rows on both sides of element 2^31, against the 64-bit forms."""
    T, H = 2 ** 21 + 40, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    big = lambda: torch.randn(T, H, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x, f, dn = big(), big(), big()
    w = torch.rand(H, generator=gen, device="cuda").to(BF) + 0.5
    stats = {}
    r, n = mm.block_norm(x, f, post_weight=w, pre_weight=w, eps=EPS, stats=stats)
    got = mm.block_norm_backward(dn, None, r, f, stats, post_weight=w, pre_weight=w)
    rows = [0, 7, 2 ** 20, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 39]
    some = dict(x=x[rows], f=f[rows], post=w, gate=None, pre=w, dn=dn[rows], dr=None)
    part = {k: v[rows] for k, v in stats.items()}
    check_forward(some, r[rows], n[rows], part)
    want = ref.norm_backward(some["dn"], None, r[rows], some["f"], w, None, w, 1.0, part["rstd_post"], part["rstd_pre"])
    for k in ("dx", "df"):
        close(got[k][rows], want[k], 2 ** -8 * want[k].abs() + 1.01 * 384 * U32 * want[k + "_terms"], k)


def test_side_stream_and_graph():
    d = make(300, 768, BF)
    r, n, stats = forward(d)
    g = backward(d, r, stats)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2, n2, stats2 = forward(d, stream=side)
    g2 = backward(d, r2, stats2, stream=side)
    side.synchronize()
    assert torch.equal(r, r2) and torch.equal(n, n2) and all(torch.equal(g[k], g2[k]) for k in g)
    # captured: the graph follows its inputs
    ws = mm.new_workspace(mm.block_norm_backward_workspace_bytes(300, 768, BF))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3, n3, stats3 = forward(d)
        g3 = backward(d, r3, stats3, workspace=ws)
    for _ in range(2):
        d["f"].mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        r, n, stats = forward(d)
        g = backward(d, r, stats)
        assert torch.equal(r, r3) and torch.equal(n, n3) and all(torch.equal(g[k], g3[k]) for k in g)


def test_refusals():
    d = make(4, 64, BF)
    x, f, w = d["x"], d["f"], d["post"]
    for kw in (dict(post_weight=w[:32]), dict(post_weight=w.float()), dict(gate=x[:2]), dict(pre_weight=w, normed=x.t()),
               dict(normed=x), dict(pre_weight=w, out=x.float())):
        with pytest.raises(ValueError):
            mm.block_norm(x, f, **kw)
    with pytest.raises(ValueError):
        mm.block_norm(x.t(), f.t(), pre_weight=d["post"][:4])            # not contiguous
    with pytest.raises(ValueError):
        mm.block_norm(x.half(), f.half())
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(residual_scale=float("inf"))):
        with pytest.raises(mm._lib.MMError):
            mm.block_norm(x, f, pre_weight=w, **kw)
    for kw in (dict(), dict(pre_weight=w, gate=w), dict(pre_weight=w, residual_scale=0.5)):
        with pytest.raises(mm._lib.MMError):
            mm.block_norm(x, **kw)
    with pytest.raises(ValueError):
        mm.block_norm(x, pre_weight=w, out=torch.empty_like(x))
    wide = torch.zeros(1, 16392, dtype=BF, device="cuda")
    with pytest.raises(mm._lib.MMError):
        mm.block_norm(wide, wide)
    odd = torch.zeros(4 * 64 + 1, dtype=BF, device="cuda")[1:].view(4, 64)    # 2 bytes behind a 16-byte boundary
    with pytest.raises(mm._lib.MMError):
        mm.block_norm(odd, f)
    r, n, stats = forward(d)
    with pytest.raises(ValueError):
        mm.block_norm_backward(d["dn"], d["dr"], r, f, {}, pre_weight=w)
    with pytest.raises(ValueError):
        mm.block_norm_backward(d["dn"], d["dr"], r, None, stats, pre_weight=w, gate=w)
    d = make(1000, 64, BF)
    r, n, stats = forward(d)
    with pytest.raises(mm._lib.MMError):
        backward(d, r, stats, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# widths on both sides of what the looping kernel holds in shared memory, where
# the element count a thread is the widest, the next or the narrowest that fits
@pytest.mark.parametrize("dtype,gate,H", [
    (F32, "token", 640), (F32, "token", 2304), (F32, "token", 5120), (F32, "token", 7168), (F32, "token", 7172),
    (F32, "channel", 5380), (F32, "channel", 6144), (F32, "channel", 9216), (F32, "channel", 9220),
    (BF, "token", 10752), (BF, "token", 10760), (BF, "channel", 12288), (BF, "channel", 12296), (BF, "channel", 8193), (F32, "channel", 4097)])
@pytest.mark.parametrize("T", [1, 610])
def test_widths_at_the_border_of_shared_memory(T, H, gate, dtype):
    d = make(T, H, dtype, gate=gate)
    r, n, stats = forward(d, s=0.9)
    check_forward(d, r, n, stats, s=0.9)
    check_backward(d, r, stats, backward(d, r, stats, s=0.9), s=0.9)
