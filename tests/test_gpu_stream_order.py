"""Calls one behind the other on a stream, nothing between them: a call reads
what the call before it wrote, however early its kernels may start.  Each call
gets new inputs in the same buffers, so that a read that comes too early finds
the last call's values, and its result is compared bit for bit with the same
call made alone (every kernel is deterministic); one call of each kind is held
to the fp64 oracle too."""
import numpy as np
import pytest
import torch

import oracle
import swiglu_mlp_top_gb300 as mm
from swiglu_mlp_top_gb300.inputs import to_f64

from parity import Y_TOL, check_route, moe_inputs, ref_y_rows, rel_err, to_dev

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CALLS = 12


def x_makers(T, H):
    """For each operator that can make a layer's input: call(round) enqueues it
    and returns the tensor that it writes, the same one every round."""
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    raw = [torch.randn(T, H, generator=gen, device="cuda").to(BF) for _ in range(CALLS)]
    w = torch.ones(H, dtype=BF, device="cuda")
    n, x, y = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(3))
    idx = torch.randint(0, 4, (T, 2), generator=gen, device="cuda", dtype=torch.int32)
    half = torch.full((T, 2), 0.5, device="cuda")
    plans = [mm.moe_permute(r, idx, 4) for r in raw]
    packed = [mm.checkpoint_pack(r) for r in raw]

    def in_place(i):
        x.copy_(raw[i])
        return mm.block_norm(x, raw[(i + 1) % CALLS], gate=w, out=x)[0]

    return {"norm": lambda i: mm.block_norm(raw[i], pre_weight=w, normed=n)[1],
            "residual in place": in_place,
            "combine": lambda i: mm.moe_unpermute(plans[i][0], plans[i][1], half, out=y),
            "gradient of the permute": lambda i: mm.moe_permute_backward(plans[i][0], plans[i][1], out=y),
            "unpack": lambda i: mm.checkpoint_unpack(packed[i], BF, out=y)}


# E > 16 or separate_routing: the router and the dispatch as two kernels, whose
# second one copies rows of x before it waits for the first; the last case is
# the router and dispatch in one kernel
@pytest.mark.parametrize("T,H,I,E,k,separate", [(2048, 768, 256, 32, 4, False), (700, 832, 128, 8, 2, False),
                                                (4096, 512, 128, 8, 2, True), (4096, 512, 128, 8, 2, False)])
@pytest.mark.parametrize("maker", ["norm", "residual in place", "combine", "gradient of the permute", "unpack"])
def test_moe_forward_behind_the_operator_that_makes_x(T, H, I, E, k, separate, maker):
    inp = moe_inputs(T, H, I, E, "bf16", seed=T)
    g = to_dev(inp)
    make = x_makers(T, H)[maker]
    ws = mm.new_workspace(mm.moe_workspace_bytes(T, H, I, E, k, BF))

    def forward(x, ws):
        return mm.moe_forward(x, g["Wr"], g["Wg"], g["Wu"], g["Wd"], k, 0.01, workspace=ws, path="tensor",
                              separate_routing=separate)

    def outputs():
        return dict(out=torch.empty(T, H, dtype=BF, device="cuda"), topk_idx=torch.empty(T, k, dtype=torch.int32, device="cuda"),
                    topk_w=torch.empty(T, k, device="cuda"), aux_loss=torch.empty((), device="cuda"))

    forward(make(0), ws)                               # kernels loaded, attributes set
    bufs = [outputs() for _ in range(CALLS)]
    torch.cuda.synchronize()
    xs = []
    for i in range(CALLS):
        x = make(i)
        mm.moe_forward(x, g["Wr"], g["Wg"], g["Wu"], g["Wd"], k, 0.01, workspace=ws, path="tensor",
                       separate_routing=separate, **bufs[i])
        xs.append(x.clone())
    torch.cuda.synchronize()
    assert mm.check_status(ws) == 0
    assert not torch.equal(xs[0], xs[1])
    for x, b in zip(xs, bufs):
        alone = forward(x, mm.new_workspace(ws.numel()))
        torch.cuda.synchronize()
        for got, want in zip((b["out"], b["topk_idx"], b["topk_w"], b["aux_loss"]), alone):
            assert torch.equal(got, want)
    if maker == "norm":
        x, b = xs[-1], bufs[-1]
        inp64 = {n: to_f64(v) for n, v in inp.items() if v is not None}
        inp64["x"] = to_f64(x.cpu())
        ref = oracle.moe_route(inp64["x"], inp64["Wr"], k, 0.01)
        idx = b["topk_idx"].cpu().numpy()
        check_route(idx, b["topk_w"].cpu().numpy(), b["aux_loss"], ref, k)
        rows = np.linspace(0, T - 1, 40).astype(int)
        want = ref_y_rows(inp64, ref, idx, rows, k)
        assert rel_err(b["out"].double().cpu().numpy()[rows], want) <= Y_TOL["bf16"]


# the streaming kernel of 5 to 128 tokens, with its two unit sizes, and the
# paths on both sides of it
@pytest.mark.parametrize("T", [1, 16, 64, 100, 300])
@pytest.mark.parametrize("made,by", [(m, b) for m in ("x", "Wg", "Wu", "Wd") for b in ("unpack", "norm")] + [("x", "a call before")])
def test_swiglu_ffn_behind_the_operator_that_makes_an_operand(T, made, by):
    H, I = 256, 128
    g = to_dev(moe_inputs(T, H, I, 0, "bf16", seed=T))
    shape = g[made].shape
    gen = torch.Generator(device="cuda").manual_seed(T)
    raw = [(g[made].float().std() * torch.randn(shape, generator=gen, device="cuda")).to(BF) for _ in range(CALLS)]
    packed = [mm.checkpoint_pack(r) for r in raw]
    ones, buf = torch.full(shape[1:], 0.05, dtype=BF, device="cuda"), torch.empty(shape, dtype=BF, device="cuda")
    ws = mm.new_workspace(mm.ffn_workspace_bytes(T, H, I, BF))
    outs = [torch.empty(T, H, dtype=BF, device="cuda") for _ in range(CALLS)]

    def make(i):
        if by == "unpack":
            mm.checkpoint_unpack(packed[i], BF, out=buf)
        elif by == "norm":
            mm.block_norm(raw[i], pre_weight=ones, normed=buf)
        else:
            mm.swiglu_ffn(raw[i], g["Wg"], g["Wu"], g["Wd"], out=buf, workspace=ws)

    def ffn(**kw):
        p = dict(g, **{made: buf})
        return mm.swiglu_ffn(p["x"], p["Wg"], p["Wu"], p["Wd"], **kw)

    make(0)
    ffn(workspace=ws)                                  # kernels loaded, attributes set
    torch.cuda.synchronize()
    for i in range(CALLS):
        make(i)
        ffn(out=outs[i], workspace=ws)
    torch.cuda.synchronize()
    for i in range(CALLS):
        make(i)
        torch.cuda.synchronize()
        alone = ffn(workspace=mm.new_workspace(ws.numel()))
        assert torch.equal(outs[i], alone), i
    p = {n: to_f64(v.cpu()) for n, v in dict(g, **{made: buf}).items() if v is not None}
    want = oracle.swiglu_ffn(p["x"], p["Wg"], p["Wu"], p["Wd"])
    # more than 128 tokens: h is kept in fp16, whose step below 2^-14 is 2^-24.
    # An h that small is off by up to 2^-25 whatever its size, and with every
    # one of them off y is by 2^-25 sum_i |Wd|: nothing beside the tolerance for
    # y of order one, but the FFN of an FFN's output is y ~ 1e-6 here.
    tiny = 2.0 ** -25 * np.abs(p["Wd"]).sum(1).max() / np.sqrt(np.mean(want ** 2)) if T > 128 else 0.0
    assert rel_err(outs[-1].double().cpu().numpy(), want) <= Y_TOL["bf16"] + tiny
