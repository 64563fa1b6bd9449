"""block_norm's gradient where a value must not reach a result that the formula
keeps it out of, and its column sums where every row counts exactly."""
import pytest
import torch

import swiglu_mlp_top_gb300 as mm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# widths of the kernel that keeps a row in registers (aligned and not) and of
# the one that walks a wide row twice
@pytest.mark.parametrize("dtype,H", [(BF, 768), (BF, 1001), (BF, 16384), (BF, 5001), (F32, 256), (F32, 77), (F32, 9000)])
@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_without_a_post_norm_df_does_not_see_f(dtype, H, T, gate, bad):
    """df = gate * D then, whatever f holds; D = dr without a norm behind r."""
    gen = torch.Generator().manual_seed(H + T)
    rand = lambda *shape: torch.randn(*shape, generator=gen).to(dtype).cuda()  # noqa: E731
    f, dr = rand(T, H), rand(T, H)
    g = None if gate is None else rand(H) if gate == "channel" else rand(T, H)
    f[1, ::7] = bad
    f[T - 1] = bad
    got = mm.block_norm_backward(None, dr, None, f, None, gate=g, residual_scale=0.5)
    assert torch.equal(got["dx"], dr / 2)
    assert torch.equal(got["df"], dr if g is None else (dr.float() * g.float()).to(dtype))
    # with a norm behind r, D comes from the stored r, and df from D
    r, dn, w, stats = rand(T, H), rand(T, H), rand(H), {}
    mm.block_norm(r, pre_weight=w, stats=stats)
    a = mm.block_norm_backward(dn, dr, r, f, stats, gate=g, pre_weight=w)
    b = mm.block_norm_backward(dn, dr, r, torch.zeros_like(f), stats, gate=g, pre_weight=w)
    assert b["df"].isfinite().all()
    for key in ("dx", "df", "d_pre_weight"):
        assert torch.equal(a[key], b[key]), key


@pytest.mark.parametrize("H", [768, 16384])
@pytest.mark.parametrize("pre", [False, True])
def test_f_is_not_needed_without_a_post_norm_and_a_gate(H, pre):
    """df = D, through the C entry with no f at all."""
    T, lib = 300, mm._lib.load()
    gen = torch.Generator().manual_seed(H)
    rand = lambda *shape: torch.randn(*shape, generator=gen).to(BF).cuda()  # noqa: E731
    r, f, dr, dn, w, stats = rand(T, H), rand(T, H), rand(T, H), rand(T, H), rand(H), {}
    mm.block_norm(r, pre_weight=w, stats=stats)
    kw = dict(pre_weight=w) if pre else {}
    want = mm.block_norm_backward(dn if pre else None, dr, r, f, stats, residual_scale=0.5, **kw)
    dx, df, dw = torch.empty_like(r), torch.empty_like(r), torch.empty(H, device="cuda")
    ws = mm.new_workspace(mm.block_norm_backward_workspace_bytes(T, H, BF))
    ptr = lambda t: t.data_ptr() if pre else None  # noqa: E731
    assert lib.mm_block_norm_backward(
        ptr(dn), dr.data_ptr(), ptr(r), None, None, None, 0, ptr(w), None, ptr(stats["rstd_pre"]), 0.5, T, H,
        mm._lib.MM_DTYPE_BF16, dx.data_ptr(), df.data_ptr(), None, None, ptr(dw), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream) == mm._lib.MM_OK
    assert torch.equal(dx, want["dx"]) and torch.equal(df, want["df"])
    assert not pre or torch.equal(dw, want["d_pre_weight"])


@pytest.mark.parametrize("T,H", [(5000, 768), (5000, 1001), (200, 16384), (3, 768)])
@pytest.mark.parametrize("gate", [None, "token"])
def test_no_sums_need_no_workspace(T, H, gate):
    lib = mm._lib.load()
    gen = torch.Generator().manual_seed(H)
    rand = lambda *shape: torch.randn(*shape, generator=gen).to(BF).cuda()  # noqa: E731
    f, dr, g = rand(T, H), rand(T, H), rand(T, H) if gate else None
    dx, df, dg = torch.empty_like(f), torch.empty_like(f), torch.empty_like(f)
    assert lib.mm_block_norm_backward(
        None, dr.data_ptr(), None, f.data_ptr(), None, g.data_ptr() if gate else None, 1, None, None, None, 0.5, T, H,
        mm._lib.MM_DTYPE_BF16, dx.data_ptr(), df.data_ptr(), None, dg.data_ptr() if gate else None, None, None, 0,
        torch.cuda.current_stream().cuda_stream) == mm._lib.MM_OK
    assert torch.equal(dx, dr / 2)
    assert torch.equal(df, (dr.float() * g.float()).to(BF) if gate else dr)
    assert not gate or torch.equal(dg, (dr.float() * f.float()).to(BF))


# ------------------------------------------------- every row counts, exactly
def whole_numbers(T, H, dtype):
    """[T, H] of a row's number (1 .. 5) times a column's (1 or 2), and their
    sums over the rows: whole numbers below 2^24, which fp32 adds without a
    rounding in any order."""
    rows = (torch.arange(T, device="cuda") * 7 // 3 % 5 + 1)[:, None]
    cols = torch.arange(H, device="cuda")[None] % 2 + 1
    total = rows.sum() * cols[0]
    assert int(total.max()) < 2 ** 24
    return (rows * cols).to(dtype), total.float()


def check_sums(T, H, dtype):
    v, total = whole_numbers(T, H, dtype)
    one, w = torch.ones(T, H, dtype=dtype, device="cuda"), torch.ones(H, dtype=dtype, device="cuda")
    stats = {k: torch.ones(T, device="cuda") for k in ("rstd_post", "rstd_pre")}
    # d_pre_weight = sum dn r rho_r of dn = v, r = rho_r = 1, and of dn = 1, r = v
    for dn, r in ((v, one), (one, v)):
        got = mm.block_norm_backward(dn, None, r, None, stats, pre_weight=w)
        assert torch.equal(got["d_pre_weight"], total)
    # D = dr without a norm behind r: d_post_weight = sum g D f rho_f and d_gate
    # = sum D p, of D = v and f = p = 1; twice and half of it by the other factor
    got = mm.block_norm_backward(None, v, None, one, stats, post_weight=2 * w, gate=w / 2)
    assert torch.equal(got["d_post_weight"], total / 2) and torch.equal(got["d_gate"], 2 * total)
    got = mm.block_norm_backward(None, one, None, v, stats, gate=w)
    assert torch.equal(got["d_gate"], total)
    got = mm.block_norm_backward(None, v, None, one, stats, post_weight=w, gate=one)
    assert torch.equal(got["d_post_weight"], total)


@pytest.mark.parametrize("dtype,H", [(BF, 8), (BF, 96), (BF, 256), (BF, 768), (BF, 2048), (BF, 4104), (BF, 12288), (BF, 16384), (BF, 33),
                                     (BF, 1001), (BF, 4095), (BF, 5001), (F32, 64), (F32, 768), (F32, 8192), (F32, 8196), (F32, 1001)])
@pytest.mark.parametrize("waves", [0, 1, 2, 5])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_column_sums_hold_every_row_once(H, dtype, waves, more):
    """Token counts around one, whole rounds of the grid's groups of threads (1
    to 16 a block, a block an SM at most), and the border to a single block."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for groups in (1, 2, 4, 5, 8, 16):
        T = max(1, (groups if waves == 0 else sms * groups * waves) + more)
        if T * H <= 2 ** 26:
            check_sums(T, H, dtype)


def test_column_sums_of_more_elements_than_32_bits_count():
    check_sums(2 ** 21 + 41, 1024, BF)
