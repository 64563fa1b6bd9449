"""8-bit checkpoints and the SwiGLU activation on them against the 64-bit
forms of block_reference.  Codes, exponents and unpacked values exactly (the
scaling is exact and the rounding defined).  SiLU: an exponential (2 ulp), a
sum, a division and at most 4 products: 16 roundings on the magnitudes of the
terms; values below fp32's normal range are left out of the relative bound
(2^-120)."""
import pytest
import torch

import block_reference as ref
import swiglu_mlp_top_gb300 as mm
from block_reference import U, U32, close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -120


def spread(R, C, dtype, seed=0):
    """Rows of very different sizes, zeros and whole groups of zeros among them."""
    gen = torch.Generator().manual_seed(R * 7 + C + seed)
    x = torch.randn(R, C, generator=gen) * torch.exp(4 * torch.randn(R, 1, generator=gen))
    x = x * (torch.rand(R, C, generator=gen) > 0.1)
    if C > 40:
        x[::3, 32:64] = 0
    return x.to(dtype)


def same(got, want):
    got, want = ref.f64(got), want.double()
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])


SHAPES = [(3, 100), (70, 36), (5, 2051), (4, 20000), (2, 4100), (3, 8193), (1, 1), (1, 2432), (3, 31), (5, 32), (4, 33), (100, 768), (17, 1000), (9, 1001), (64, 4864), (300, 200), (7, 48),
          (2000, 96), (33, 24)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C", SHAPES)
def test_pack_and_unpack(R, C, dtype):
    x = spread(R, C, dtype)
    ck = mm.checkpoint_pack(x.cuda())
    codes, exps, values = ref.checkpoint(x)
    assert torch.equal(ck["exps"].cpu(), exps) and same(ck["codes"].float(), codes)
    for out in (F32, BF):
        assert same(mm.checkpoint_unpack(ck, out), values.to(out))
    # the stated bound on a value's error
    scale = torch.ldexp(torch.ones((), dtype=torch.float64), exps.int() - 127).repeat_interleave(32, 1)[:, :C]
    err = (x.double() - values).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scale)).all())


def test_borders_and_special_values():
    """Group maxima at the border between two scales, ties between two codes,
    the smallest and largest floats, infinities and NaN.  What a code stands
    for is rounded to the type that is asked for: the largest bf16 (255 * 2^120)
    has the code of 256 * 2^120 = 2^128, which fp32 has only as an infinity."""
    rows = []
    for top in (448.0, 449.0, 447.0, 450.0, 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -149, 2.0 ** -118, 3.3895314e38, 0.0):
        r = torch.zeros(32)
        r[0] = top
        r[1:20] = -top * torch.linspace(0, 1, 19)
        rows.append(r)
    ties = torch.zeros(32)
    ties[0] = 448.0
    ties[1:17] = torch.tensor([(8 + i + 0.5) * 2.0 for i in range(8)] + [(i + 0.5) * 2.0 ** -9 for i in range(8)])
    odd = torch.randn(32, generator=torch.Generator().manual_seed(1))
    for bad in (float("inf"), -float("inf"), float("nan")):
        odd = odd.clone()
        odd[5] = bad
        rows.append(odd)
    rows += [ties, torch.full((32,), float("nan")), torch.full((32,), float("-inf"))]
    x = torch.stack(rows)
    for dtype in (F32, BF):
        v = x.to(dtype)
        ck = mm.checkpoint_pack(v.cuda())
        codes, exps, values = ref.checkpoint(v)
        assert torch.equal(ck["exps"].cpu(), exps) and same(ck["codes"].float(), codes)
        assert same(mm.checkpoint_unpack(ck, F32), values.to(F32))


def test_every_code_comes_back():
    codes = torch.arange(256, dtype=torch.uint8).view(8, 32).cuda().view(torch.float8_e4m3fn)
    for e in (1, 100, 127, 200, 247):
        ck = {"codes": codes, "exps": torch.full((8, 1), e, dtype=torch.uint8, device="cuda"), "segments": 1}
        want = codes.cpu().float().double() * 2.0 ** (e - 127)
        assert same(mm.checkpoint_unpack(ck, F32), want.to(F32))     # 448 * 2^120 is beyond fp32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,I", [(3, 100), (70, 36), (5, 2051), (3, 20000), (2, 4100), (3, 8193), (1, 1), (1, 2432), (3, 31), (100, 768), (17, 1000), (9, 1001), (130, 48), (31, 24), (600, 96)])
def test_swiglu_and_its_gradient(R, I, dtype):
    u_ = U[dtype]
    gu = torch.cat([spread(R, I, dtype), spread(R, I, dtype, seed=1)], 1)
    gu[0, 0] = -100.0                                   # sigmoid below fp32's range
    ck = {}
    h = mm.swiglu_act(gu.cuda(), checkpoint=ck)
    g, u = gu.double().split(I, 1)
    want = ref.swiglu(g, u)
    close(h, want, (u_ + 16 * U32 * (1 + u_)) * want.abs() + TINY * (1 + u.abs()), "h")
    assert torch.equal(mm.swiglu_act(gu.cuda()), h)
    codes, exps, values = ref.checkpoint(gu.view(2 * R, I))
    assert torch.equal(ck["exps"].cpu().view(2 * R, -1), exps) and same(ck["codes"].float().view(2 * R, I), codes)
    assert same(mm.checkpoint_unpack(ck, F32), values.view(R, 2 * I))
    # the backward from what was kept
    dh = spread(R, I, dtype, seed=2) * 0.01
    dgu, h2 = mm.swiglu_act_backward(ck, dh.cuda())
    g, u = values.view(R, 2 * I).split(I, 1)
    dG, dU, terms = ref.swiglu_backward(g, u, dh.double())
    big = 1 + u.abs() + dh.double().abs() + (u * dh.double()).abs()
    close(dgu[:, :I], dG, u_ * dG.abs() + 16 * U32 * (1 + u_) * terms + TINY * big, "dG")
    close(dgu[:, I:], dU, (u_ + 16 * U32 * (1 + u_)) * dU.abs() + TINY * big, "dU")
    want = ref.swiglu(g, u)
    close(h2, want, (u_ + 16 * U32 * (1 + u_)) * want.abs() + TINY * big, "h again")
    only, none = mm.swiglu_act_backward(ck, dh.cuda(), want_h=False)
    assert none is None and torch.equal(only, dgu)


def test_not_finite_values_stay_visible():
    gu = torch.randn(4, 128, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    gu[1, 3], gu[2, 70] = float("nan"), float("inf")
    ck = {}
    h = mm.swiglu_act(gu, checkpoint=ck)
    dgu, h2 = mm.swiglu_act_backward(ck, torch.ones(4, 64, dtype=BF, device="cuda"))
    for t in (h, h2):
        assert t[[0, 3]].isfinite().all() and not t[1, 3].isfinite() and not t[2, 6].isfinite()
        assert (~t.isfinite()).sum() == 2
    assert dgu[[0, 3]].isfinite().all() and dgu[1, 3].isnan() and dgu[2, 6].isnan()


@pytest.mark.parametrize("I", [96, 33])
def test_rows_behind_the_last_are_left_alone(I):
    R, n = 50, 37
    gu = torch.randn(R, 2 * I, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    full, ck = {}, {"codes": torch.full((R, 2 * I), 1.0, device="cuda").to(torch.float8_e4m3fn),
                    "exps": torch.full((R, 2 * -(-I // 32)), 9, dtype=torch.uint8, device="cuda")}
    h = mm.swiglu_act(gu, checkpoint=full)
    rows = torch.tensor([n], dtype=torch.int32, device="cuda")
    mark = torch.full((R, I), 7.0, dtype=BF, device="cuda")
    part = mm.swiglu_act(gu, checkpoint=ck, out=mark, rows=rows)
    assert torch.equal(part[:n], h[:n]) and bool((part[n:] == 7).all())
    assert torch.equal(ck["exps"][:n], full["exps"][:n]) and bool((ck["exps"][n:] == 9).all())
    assert torch.equal(ck["codes"][:n].float(), full["codes"][:n].float()) and bool((ck["codes"][n:].float() == 1).all())
    dh = torch.randn(R, I, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    dgu, h2 = mm.swiglu_act_backward(full, dh)
    out, hm = torch.full((R, 2 * I), 7.0, dtype=BF, device="cuda"), torch.full((R, I), 7.0, dtype=BF, device="cuda")
    mm.swiglu_act_backward(full, dh, out=out, h_out=hm, rows=rows)
    assert torch.equal(out[:n], dgu[:n]) and torch.equal(hm[:n], h2[:n])
    assert bool((out[n:] == 7).all()) and bool((hm[n:] == 7).all())
    for count in (0, -5, R + 9):                        # none of them, and more than there are
        rows.fill_(count)
        got = mm.swiglu_act(gu, out=torch.full((R, I), 7.0, dtype=BF, device="cuda"), rows=rows)
        assert torch.equal(got, h) if count > 0 else bool((got == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("I", [32, 33])
def test_infinite_gate(I, dtype):
    """SiLU(inf) = inf; the product with u carries its sign."""
    gu = torch.ones(2, 2 * I, dtype=dtype, device="cuda")
    gu[0, 5] = float("inf")
    gu[1, 5], gu[1, I + 5] = float("inf"), -2.0
    h = mm.swiglu_act(gu)
    assert h[0, 5] == float("inf") and h[1, 5] == -float("inf") and (~h.isfinite()).sum() == 2


def test_more_elements_than_32_bits_count():
    """Rows on both sides of byte 2^32 of the codes and of gu."""
    R, I = 1_100_000, 2048
    gen = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.randn(R, 2 * I, generator=gen, device="cuda", dtype=BF)
    ck = {}
    h = mm.swiglu_act(gu, checkpoint=ck)
    dgu, h2 = mm.swiglu_act_backward(ck, h)
    rows = [0, 2 ** 19 - 1, 2 ** 19, 2 ** 20 - 1, 2 ** 20, R - 1]
    small = {}
    hs = mm.swiglu_act(gu[rows], checkpoint=small)
    ds, hs2 = mm.swiglu_act_backward(small, h[rows])
    assert torch.equal(h[rows], hs) and torch.equal(dgu[rows], ds) and torch.equal(h2[rows], hs2)
    assert torch.equal(ck["exps"][rows], small["exps"])
    assert torch.equal(ck["codes"].view(torch.uint8)[rows], small["codes"].view(torch.uint8))


def test_no_rows():
    ck = {}
    h = mm.swiglu_act(torch.empty(0, 128, dtype=BF, device="cuda"), checkpoint=ck)
    dgu, h2 = mm.swiglu_act_backward(ck, h)
    assert h.shape == h2.shape == (0, 64) and dgu.shape == (0, 128)
    assert mm.checkpoint_unpack(mm.checkpoint_pack(h)).shape == (0, 64)


def test_side_stream_and_graph():
    gu = torch.randn(700, 512, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    dh = torch.randn(700, 256, generator=torch.Generator().manual_seed(6)).to(BF).cuda()

    def step(stream=None):
        ck = {}
        h = mm.swiglu_act(gu, checkpoint=ck, stream=stream)
        x = mm.checkpoint_unpack(mm.checkpoint_pack(h, stream=stream), stream=stream)
        return (h, x, *mm.swiglu_act_backward(ck, dh, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(2):
        gu.mul_(-1.5)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_checkpointed_input_feeds_the_ffn_backward():
    """x kept in 8 bits, unpacked, and given to swiglu_ffn_backward: the
    gradients are those of that x, bit for bit."""
    from swiglu_mlp_top_gb300.inputs import make_inputs
    T, H, I = 300, 256, 384
    inp = {k: v.cuda() for k, v in make_inputs(T, H, I, "bf16").items()}
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).to(BF).cuda()
    x8 = mm.checkpoint_unpack(mm.checkpoint_pack(inp["x"]))
    values = ref.checkpoint(inp["x"])[2].to(BF).cuda()
    a = mm.swiglu_ffn_backward(x8, inp["Wg"], inp["Wu"], inp["Wd"], dy)
    b = mm.swiglu_ffn_backward(values, inp["Wg"], inp["Wu"], inp["Wd"], dy)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_refusals():
    gu = torch.zeros(4, 64, dtype=BF, device="cuda")
    ck = {}
    h = mm.swiglu_act(gu, checkpoint=ck)
    with pytest.raises(ValueError):
        mm.swiglu_act(gu[:, :63].contiguous())
    with pytest.raises(ValueError):
        mm.swiglu_act(gu[:, ::2])
    with pytest.raises(ValueError):
        mm.swiglu_act(gu.half())
    with pytest.raises(ValueError):
        mm.swiglu_act(gu, rows=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mm.swiglu_act(gu, checkpoint={"codes": ck["codes"][:2]})
    with pytest.raises(ValueError):
        mm.swiglu_act_backward(mm.checkpoint_pack(gu), h)         # holds no g and u
    with pytest.raises(ValueError):
        mm.swiglu_act_backward(ck, h[:3])
    with pytest.raises(ValueError):
        mm.swiglu_act_backward(ck, h, want_h=False, h_out=h)
    with pytest.raises(ValueError):
        mm.checkpoint_unpack(ck, torch.float16)
    with pytest.raises(ValueError):
        mm.checkpoint_unpack(dict(ck, exps=ck["exps"][:, :1]))
    odd = torch.zeros(4 * 64 + 1, dtype=BF, device="cuda")[1:].view(4, 64)
    with pytest.raises(mm._lib.MMError):
        mm.checkpoint_pack(odd)


def test_a_refused_call_leaves_the_checkpoint_alone():
    """100 columns in one segment and twice 50 columns both take four exponents
    a row: a checkpoint that a refused call relabels would unpack to other values."""
    x = spread(6, 100, BF).cuda()
    ck = mm.checkpoint_pack(x)
    want = mm.checkpoint_unpack(ck, F32)
    wide, kept = torch.zeros(6, 120, dtype=BF, device="cuda"), dict(ck)
    for kw in (dict(), dict(out=torch.zeros(6, 61, dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            mm.swiglu_act(wide, checkpoint=ck, **kw)
        assert ck == kept and torch.equal(mm.checkpoint_unpack(ck, F32), want)
    empty = {}
    with pytest.raises(ValueError):
        mm.swiglu_act(wide, checkpoint=empty, out=torch.zeros(6, 61, dtype=BF, device="cuda"))
    assert not empty
