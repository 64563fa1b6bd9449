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
