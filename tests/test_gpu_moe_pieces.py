"""An MoE block's training step from its pieces: norm, route, sort, the
experts' products (plain matrix products here), SwiGLU with its 8-bit
checkpoint, back to token order, norm, gate and residual with the next norm -
and every gradient, against the same steps in 64 bits.

The gradient is the 8-bit checkpoint's own: the 64-bit side takes g and u from
it too.  Each of the nine steps of a chain adds at most (384 + K) roundings of
2^-24 on its terms, K <= 192 the longest product's sum, and terms outweigh
results by no more than sqrt(K) ~ 14 (sums of K independent terms): 9 * 576 *
14 * 2^-24 = 4.4e-3 at the very worst; roundings that add up as a random walk
give sqrt of their number, 3e-4.  The bar is 1e-3 in the 2-norm.
"""
import pytest
import torch

import block_reference as ref
import swiglu_mlp_top_gb300 as mm
from block_reference import f64

pytestmark = pytest.mark.gpu
EPS, BAR = 1e-5, 1e-3


def near(got, want, what, terms=None):
    """Within BAR of want in the 2-norm, or of the norm of its terms' magnitudes."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape
    off = (got - want).norm() / (want if terms is None else terms).norm()
    assert off <= BAR, f"{what}: {off:.2e} off"


@pytest.fixture
def full_fp32():
    kept = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = kept


@pytest.mark.parametrize("T,H,I,E,k,align", [(1, 64, 96, 4, 2, 1), (77, 128, 192, 8, 2, 16), (300, 96, 100, 4, 1, 64)])
def test_training_step(full_fp32, T, H, I, E, k, align):
    gen = torch.Generator().manual_seed(T)
    rand = lambda *shape, std=1.0, mean=0.0: (torch.randn(*shape, generator=gen) * std + mean).cuda()  # noqa: E731
    x, Wr = rand(T, H), rand(E, H, std=0.1)
    Wgu, Wd = rand(E, 2 * I, H, std=0.1), rand(E, H, I, std=0.1)
    w1, w2, post, gate = (rand(H, std=0.1, mean=1.0) for _ in range(4))
    dn, dr = rand(T, H), rand(T, H)

    # forward
    s1, s2 = {}, {}
    _, n1 = mm.block_norm(x, pre_weight=w1, eps=EPS, stats=s1)
    idx, w, _, _ = mm.moe_route(n1, Wr, k, 0.0)
    R = mm.moe_permuted_rows(T, E, k, align)
    xs, plan = mm.moe_permute(n1, idx, E, align=align, out=torch.zeros(R, H, device="cuda"))
    at = [slice(a, b) for a, b in zip(plan["offsets"].tolist(), plan["offsets"][1:].tolist())]
    end = plan["offsets"][-1:]
    gu, ys, ck = torch.zeros(R, 2 * I, device="cuda"), torch.zeros(R, H, device="cuda"), {}
    for e in range(E):
        gu[at[e]] = xs[at[e]] @ Wgu[e].T
    h = mm.swiglu_act(gu, checkpoint=ck, rows=end)
    for e in range(E):
        ys[at[e]] = h[at[e]] @ Wd[e].T
    f = mm.moe_unpermute(ys, plan, w)
    r, n = mm.block_norm(x, f, post_weight=post, gate=gate, pre_weight=w2, eps=EPS, stats=s2)

    # backward
    g2 = mm.block_norm_backward(dn, dr, r, f, s2, post_weight=post, gate=gate, pre_weight=w2)
    dys, dw = mm.moe_unpermute_backward(g2["df"], ys, plan, w, out=torch.zeros(R, H, device="cuda"))
    dh, dxs = torch.zeros(R, I, device="cuda"), torch.zeros(R, H, device="cuda")
    for e in range(E):
        dh[at[e]] = dys[at[e]] @ Wd[e]
    dgu, h8 = mm.swiglu_act_backward(ck, dh, rows=end)
    for e in range(E):
        dxs[at[e]] = dgu[at[e]] @ Wgu[e]
    dWd = torch.stack([dys[at[e]].T @ h8[at[e]] for e in range(E)])
    dWgu = torch.stack([dgu[at[e]].T @ xs[at[e]] for e in range(E)])
    dn1 = mm.moe_permute_backward(dxs, plan)
    g1 = mm.block_norm_backward(dn1, g2["dx"], x, None, s1, pre_weight=w1)

    # the same in 64 bits, on the same routing
    X, P = f64(x), plan["pos"].cpu()
    o1 = ref.norm_forward(x, None, None, None, w1, 1.0, EPS)
    flat, tok = idx.cpu().reshape(-1).long(), torch.arange(T * k) // k
    A, B = f64(Wgu), f64(Wd)
    xa = o1["n"][tok]
    gua = torch.stack([A[e] @ v for e, v in zip(flat, xa)])
    ha = ref.swiglu(gua[:, :I], gua[:, I:])
    ya = torch.stack([B[e] @ v for e, v in zip(flat, ha)]).view(T, k, H)
    W = f64(w)
    fa = (ya * W[..., None]).sum(1)
    o2 = ref.norm_forward(x, fa, post, gate, w2, 1.0, EPS)
    near(n, o2["n"], "n")
    near(r, o2["r"], "r")
    b2 = ref.norm_backward(dn, dr, o2["r"], fa, post, gate, w2, 1.0, o2["rstd_post"], o2["rstd_pre"])
    near(g2["df"], b2["df"], "df")
    # dw = <df, ys> cancels: f = sum_s w ys, and a norm does not change with the
    # length of its input, so sum_s w dw = <df, f> = eps rho_f^2 <rho_f w_post q, f>
    # ~ 1e-5 of its terms (for k = 1 that is dw itself): held to its terms
    near(dw, (ya * b2["df"][:, None]).sum(2), "dw", terms=(ya * b2["df"][:, None]).abs().sum(2))
    dya = (b2["df"][:, None] * W[..., None]).reshape(T * k, H)
    dha = torch.stack([v @ B[e] for e, v in zip(flat, dya)])
    rows = P.reshape(-1).long()
    kept = f64(mm.checkpoint_unpack(ck, torch.float32))[rows]
    gk, uk = kept[:, :I], kept[:, I:]
    dG, dU, _ = ref.swiglu_backward(gk, uk, dha)
    dga = torch.cat([dG, dU], 1)
    hk = ref.swiglu(gk, uk)
    pick = lambda M: torch.stack([(M * (flat == e)[:, None, None]).sum(0) for e in range(E)])  # noqa: E731
    near(dWd, pick(dya[:, :, None] * hk[:, None, :]), "dWd")
    near(dWgu, pick(dga[:, :, None] * xa[:, None, :]), "dWgu")
    dxa = torch.stack([v @ A[e] for e, v in zip(flat, dga)]).view(T, k, H).sum(1)
    b1 = ref.norm_backward(dxa, b2["dx"], X, None, None, None, w1, 1.0, None, o1["rstd_pre"])
    near(g1["dx"], b1["dx"], "dx")
    for got, key in ((g1["d_pre_weight"], b1["d_pre_weight"]), (g2["d_pre_weight"], b2["d_pre_weight"]),
                     (g2["d_post_weight"], b2["d_post_weight"]), (g2["d_gate"], b2["d_gate"])):
        near(got, key, "a norm's or gate's gradient")
    # what the 8 bits cost against the unquantised gradient: a step of 2^-4 on g and u
    true = torch.cat(ref.swiglu_backward(gua[:, :I], gua[:, I:], dha)[:2], 1)
    assert (dga - true).norm() <= 2 * 2.0 ** -4 * true.norm()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, H, E, k = 3000, 768, 8, 2
    side = [torch.cuda.Stream(), torch.cuda.Stream()]

    def inputs():
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        return dict(x=rand(T, H), f=rand(T, H), w=rand(H), dn=rand(T, H), w_route=torch.rand(T, k, generator=gen, device="cuda"),
                    idx=torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32))

    def step(q, stream):
        stats, ck = {}, {}
        r, n = mm.block_norm(q["x"], q["f"], post_weight=q["w"], gate=q["w"], pre_weight=q["w"], stats=stats, stream=stream)
        g = mm.block_norm_backward(q["dn"], None, r, q["f"], stats, post_weight=q["w"], gate=q["w"], pre_weight=q["w"], stream=stream)
        xs, plan = mm.moe_permute(n, q["idx"], E, stream=stream)
        h = mm.swiglu_act(xs, checkpoint=ck, stream=stream)
        dgu, _ = mm.swiglu_act_backward(ck, h, stream=stream)
        return [r, n, *(g[k] for k in sorted(g)), xs, mm.moe_unpermute(dgu, plan, q["w_route"], stream=stream)]

    qs = [inputs(), inputs()]
    alone = [step(q, None) for q in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [step(q, s) for q, s in zip(qs, side)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_share_a_workspace_on_one_stream():
    gen = torch.Generator(device="cuda").manual_seed(12)
    H, sizes = 512, (2500, 4000)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    w = rand(H)
    ws = mm.new_workspace(max(mm.block_norm_backward_workspace_bytes(T, H, torch.bfloat16) for T in sizes))
    qs, graphs, outs = [(rand(T, H), rand(T, H)) for T in sizes], [], []

    def step(x, dn, **kw):
        stats = {}
        mm.block_norm(x, pre_weight=w, stats=stats)
        return mm.block_norm_backward(dn, None, x, None, stats, pre_weight=w, **kw)

    want = [step(*q) for q in qs]
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*q, workspace=ws))
    for i in (0, 1, 0, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(a[k], b[k]) for k in a)
