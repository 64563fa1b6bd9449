"""Workloads of the experts' matrix products of an MoE block:

  grouped_matmul    rows sorted by expert times each expert's matrix, and the backward
  mx4_quantize      values in microscaled 4-bit floating point (e2m1, a power of two per 32 columns), and back
  mx4_matmul        products of them: 4-bit rows or bf16 rows with 4-bit weights, dense or by expert

run() computes an operator in elementary torch operations in 32 bits, or, with
`own`, through the package.  exact() is the definition in 64 bits.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32          # columns that share one scale of a 4-bit tensor
WORD = 4            # scales of one row that lie next to each other


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decode step, both projections of its two experts: latency
        dict(name="gmm_t1_e8k2", op="gmm", T=1, K=768, N=4864, E=8, k=2, align=1, drop=0.0, dtype="bf16"),
        # the top-2 workload's tokens through gate and up in one product
        dict(name="gmm_t16384_e8k2_gateup", op="gmm", T=16384, K=768, N=4864, E=8, k=2, align=64, drop=0.0, dtype="bf16"),
        # many experts of a wider model, ragged groups without padding, a width that fills no tile
        dict(name="gmm_t8191_e64k8_n1000", op="gmm", T=8191, K=2048, N=1000, E=64, k=8, align=1, drop=0.0, dtype="bf16"),
        # top-1 routing in fp32
        dict(name="gmm_t1000_e4k1_f32", op="gmm", T=1000, K=768, N=2432, E=4, k=1, align=1, drop=0.0, dtype="f32"),
        # gradients of the down product of the training batch
        dict(name="gmm_bwd_t16384_e8k2_down", op="gmm_bwd", T=16384, K=2432, N=768, E=8, k=2, align=64, drop=0.0, dtype="bf16"),
        # a small batch, odd width, a quarter of the assignments on another device
        dict(name="gmm_bwd_t511_e16k4_k1001", op="gmm_bwd", T=511, K=1001, N=520, E=16, k=4, align=1, drop=0.25, dtype="bf16"),
        # the eight experts' gate and up weights, laid out once and read back
        dict(name="mx4_pack_weights_e8", op="mx4_pack", R=8 * 4864, C=768, dtype="bf16"),
        # activations of the top-2 workload before the down product
        dict(name="mx4_pack_r32768_c2432", op="mx4_pack", R=32768, C=2432, dtype="bf16"),
        # one token of a decode step with weights in 4 bits
        dict(name="mx4w_t1_e8k2", op="mx4w", T=1, K=768, N=4864, E=8, k=2, align=1, drop=0.0, dtype="bf16"),
        # a decode batch through the down product with weights in 4 bits
        dict(name="mx4w_t64_e8k2_down", op="mx4w", T=64, K=2432, N=768, E=8, k=2, align=1, drop=0.0, dtype="bf16"),
        # a prompt's tokens by expert, both operands in 4 bits
        dict(name="mx4_mm_t16384_e8k2_gateup", op="mx4_mm", T=16384, K=768, N=4864, E=8, k=2, align=64, drop=0.0, dtype="bf16"),
        # a wide dense product, both operands in 4 bits
        dict(name="mx4_mm_dense_t8192_k4096", op="mx4_mm", T=8192, K=4096, N=8192, E=1, k=1, align=1, drop=0.0, dtype="bf16"),
    ]


MOST_FLOPS = {"bf16": 500e9, "f32": 30e9}
MOST_BYTES = 750e6
MOST_WEIGHTS = 200e6        # elements


def _between(rng, lo, hi):
    """Log-uniform whole number in [lo, hi]."""
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def _width(rng):
    width = _between(rng, 64, 8192)
    return max(64, width // 64 * 64) if rng.random() < 0.75 else width      # model widths; the rest are odd ones


def draw(rng):
    op = rng.choice(["gmm", "gmm", "gmm_bwd", "gmm_bwd", "mx4_pack", "mx4_mm", "mx4w"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"]) if op in ("gmm", "gmm_bwd", "mx4_pack") else "bf16"
    if op == "mx4_pack":
        c = dict(op=op, R=_between(rng, 1, 65536), C=_width(rng), dtype=dtype)
        while work(c)["bytes"] > MOST_BYTES:
            c["R"] //= 2
        return c
    E = rng.choice([1, 2, 4, 8, 8, 16, 32, 64])
    c = dict(op=op, T=_between(rng, 1, 16384), K=_width(rng), N=_width(rng), E=E, k=rng.randint(1, min(8, E)),
             align=rng.choice([1, 1, 16, 64, 128]) if E > 1 else 1, drop=rng.choice([0.0, 0.0, 0.5]) if E > 1 else 0.0, dtype=dtype)
    while c["E"] * c["N"] * c["K"] > MOST_WEIGHTS:
        c["N" if c["N"] > c["K"] else "K"] //= 2
    while work(c)["flops"] > MOST_FLOPS[dtype] or work(c)["bytes"] > MOST_BYTES:
        if c["T"] == 1:
            c["N" if c["N"] > c["K"] else "K"] //= 2
        else:
            c["T"] //= 2
    return c


def total_rows(c):
    """Rows of the sorted tensor: every assignment, and each group's padding at its most."""
    return c["T"] * c["k"] + min(c["E"], c["T"] * c["k"]) * (c["align"] - 1)


def work(c):
    """Each input read once, each output written once; of the experts, those that have a row."""
    op, es = c["op"], 2 if c["dtype"] == "bf16" else 4
    if op == "mx4_pack":
        n = c["R"] * c["C"]
        return {"bytes": 2 * n * (es + 0.5 + 1 / GROUP), "flops": 4 * n}
    rows = c["T"] * c["k"] * (1 - c["drop"])
    used = c["E"] * (1 - (1 - 1 / c["E"]) ** rows) if c["E"] > 1 else 1
    mat, four = c["K"] * c["N"], 0.5 + 1 / GROUP
    flops = 2 * rows * mat
    if op == "gmm":
        return {"bytes": es * (rows * (c["K"] + c["N"]) + used * mat), "flops": flops}
    if op == "gmm_bwd":
        return {"bytes": es * (rows * (2 * c["K"] + c["N"]) + used * mat) + 4 * c["E"] * mat, "flops": 2 * flops}
    if op == "mx4_mm":
        return {"bytes": four * (rows * c["K"] + used * mat) + 2 * rows * c["N"], "flops": flops}
    return {"bytes": 2 * rows * (c["K"] + c["N"]) + four * used * mat, "flops": flops}


# ------------------------------------------------------------------ inputs
def _plan(case, g):
    """The sort of a skewed routing: offsets, counts (and their host copy, which the plain form walks)."""
    T, E, k, align = case["T"], case["E"], case["k"], case["align"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, 0] += 1.0
    idx = logits.topk(k, dim=1).indices
    if case["drop"]:
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, idx)
    counts = (idx.reshape(-1, 1) == torch.arange(E, device="cuda")).sum(0)
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    return {"offsets": offsets.int(), "counts": counts.int()}, list(zip(offsets.tolist(), counts.tolist()))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def activations(rows, width):
        # a few channels of a residual stream are far larger than the rest, and rows differ in size
        loud = 1.0 + 9.0 * (torch.rand(width, generator=g, device="cuda") < 0.01)
        size = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
        return (torch.randn(rows, width, generator=g, device="cuda") * loud * size).to(dt)

    st = dict(case=case, op=op, dtype=dt)
    if op == "mx4_pack":
        st["x"] = activations(case["R"], case["C"])
        return st
    E, K, N, R = case["E"], case["K"], case["N"], total_rows(case)
    if E > 1:
        st["plan"], st["groups"] = _plan(case, g)
        w = torch.randn(E, N, K, generator=g, device="cuda")
    else:
        st["plan"], st["groups"] = None, [(0, R)]
        w = torch.randn(N, K, generator=g, device="cuda")
    w = (w * 0.02).to(dt)
    mask = torch.zeros(R, 1, dtype=dt, device="cuda")          # padding rows are zero, as the sort leaves them
    for at, n in st["groups"]:
        mask[at: at + n] = 1
    x = activations(R, K) * mask
    if op == "gmm":
        st.update(xs=x, w=w, out=torch.zeros(R, N, dtype=dt, device="cuda"))
    elif op == "gmm_bwd":
        dys = (torch.randn(R, N, generator=g, device="cuda") * 0.05).to(dt) * mask
        st.update(xs=x, w=w, dys=dys, out=torch.zeros(R, K, dtype=dt, device="cuda"))
    else:
        st["out"] = torch.zeros(R, N, dtype=dt, device="cuda")
        st["w4"] = _pack(w)                                    # weights are laid out once
        st["x"] = _pack(x) if op == "mx4_mm" else x
    return st


# ----------------------------------------------------- plain forms, 32 bits
def _pack(x):
    """e2m1 codes, two to a byte (the even column in the low half), of whole groups of 32 columns,
    and their biased exponents, word by word of four groups: [words, rows, 4]."""
    C = x.shape[-1]
    lead, x = x.shape[:-1], x.reshape(-1, C).float()
    R, G = x.shape[0], -(-C // GROUP)
    groups = torch.zeros(R, G * GROUP, device=x.device)
    groups[:, :C] = x
    groups = groups.view(R, G, GROUP)
    m, p = torch.frexp(groups.abs().amax(2))                   # amax = m 2^p, 0.5 <= m < 1;  6 = 0.75 * 2^3
    e = torch.where(m > 0.75, p - 2, p - 3)
    e = torch.where(m == 0, -126, e).clamp(min=-126)
    v = torch.ldexp(groups, -e[..., None])
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step                           # ties to even, which are the even codes
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).view(R, -1, 2)
    words = -(-G // WORD)
    exps = torch.full((R, words * WORD), 127, dtype=torch.uint8, device=x.device)
    exps[:, :G] = (e + 127).to(torch.uint8)
    return {"codes": (code[..., 0] + 16 * code[..., 1]).view(*lead, -1),
            "exps": exps.view(R, words, WORD).transpose(0, 1).contiguous(), "cols": C}


def _values(q):
    """The 32-bit values of a 4-bit tensor."""
    codes = q["codes"].reshape(-1, q["codes"].shape[-1])
    R = codes.shape[0]
    code = torch.stack([codes & 15, codes >> 4], 2).view(R, -1)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = table[(code & 7).int()]
    v = torch.where(code > 7, -v, v)
    exps = q["exps"].transpose(0, 1).reshape(R, -1)[:, : v.shape[1] // GROUP]
    v = torch.ldexp(v.view(R, -1, GROUP), exps.int()[..., None] - 127).view(R, -1)
    return v[:, : q["cols"]].reshape(*q["codes"].shape[:-1], q["cols"])


def _by_expert(st, rows, w, transposed):
    """Each group's rows times its matrix (or its transpose); zeros elsewhere."""
    w = w if w.dim() == 3 else w[None]
    out = torch.zeros(rows.shape[0], w.shape[1 if transposed else 2], dtype=st["dtype"], device=rows.device)
    for (at, n), mat in zip(st["groups"], w):
        if n:
            mat = mat.float()
            out[at: at + n] = (rows[at: at + n].float() @ (mat.T if transposed else mat)).to(st["dtype"])
    return out


def _plain(st):
    op = st["op"]
    if op == "gmm":
        return _by_expert(st, st["xs"], st["w"], True)
    if op == "gmm_bwd":
        dw = torch.zeros(st["w"].shape, device="cuda")
        each = dw if dw.dim() == 3 else dw[None]
        for (at, n), d in zip(st["groups"], each):
            if n:
                d.copy_(st["dys"][at: at + n].float().T @ st["xs"][at: at + n].float())
        return {"dxs": _by_expert(st, st["dys"], st["w"], False), "dw": dw}
    if op == "mx4_pack":
        q = _pack(st["x"])
        return {"exps": q["exps"], "x": _values(q).to(st["dtype"])}
    x = _values(st["x"]) if op == "mx4_mm" else st["x"]
    return _by_expert(st, x, _values(st["w4"]), True)


# ------------------------------------------------------ the package's calls
def _own(st):
    import swiglu_mlp_top_gb300 as mm
    op = st["op"]
    if op == "gmm":
        return mm.grouped_matmul(st["xs"], st["w"], st["plan"], out=st["out"])
    if op == "gmm_bwd":
        dxs, dw = mm.grouped_matmul_backward(st["dys"], st["xs"], st["w"], st["plan"], out=st["out"])
        return {"dxs": dxs, "dw": dw}
    if op == "mx4_pack":
        q = mm.mx4_quantize(st["x"])
        return {"exps": q["exps"], "x": mm.mx4_dequantize(q, st["dtype"])}
    return mm.mx4_matmul(st["x"], st["w4"], st["plan"], out=st["out"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition, 64 bits
def _exact_pack(x):
    """(biased exponents by row and group, the values that the codes stand for)."""
    R, C = x.shape
    G = -(-C // GROUP)
    y = torch.nn.functional.pad(x.double(), (0, G * GROUP - C)).view(R, G, GROUP)
    amax = y.abs().amax(2)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140) / 6)) - 1
    for _ in range(3):                                      # the least e with amax <= 6 * 2^e
        e = torch.where(amax > 6 * torch.exp2(e), e + 1, e)
    e = e.clamp(min=-126)
    v = (y / torch.exp2(e)[..., None]).contiguous()
    magnitudes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    middles = (magnitudes[1:] + magnitudes[:-1]) / 2
    low = torch.bucketize(v.abs(), middles)                 # middles below |v|: a tie goes down ...
    tie = (low < 7) & (v.abs() == middles[low.clamp(max=6)]) & (low % 2 == 1)
    q = magnitudes[low + tie.long()] * torch.sign(v)        # ... or up, where down is an odd code
    return e + 127, (q * torch.exp2(e)[..., None]).view(R, G * GROUP)[:, :C]


def _exact_values(q):
    """The 64-bit values of a 4-bit tensor, from the format: sign, two exponent bits, one fraction bit."""
    C, codes = q["cols"], q["codes"].reshape(-1, q["codes"].shape[-1]).int()
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        exp, frac = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(exp == 0, frac / 2, (1 + frac / 2) * torch.exp2(exp.double() - 1))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    for col in range(0, out.shape[1], GROUP):
        word, byte = divmod(col // GROUP, WORD)
        out[:, col: col + GROUP] *= torch.exp2(q["exps"][word, :, byte].double() - 127)[:, None]
    return out[:, :C].reshape(*q["codes"].shape[:-1], C)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "mx4_pack":
        return {"exps": None, "x": _exact_pack(st["x"])[1]}
    four = op in ("mx4_mm", "mx4w")
    w = _exact_values(st["w4"]) if four else st["w"].double()
    w = w.reshape(-1, *w.shape[-2:])
    if op == "gmm_bwd":
        dxs = torch.zeros(st["xs"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for e, (at, n) in enumerate(st["groups"]):
            dy, x = st["dys"][at: at + n].double(), st["xs"][at: at + n].double()
            dxs[at: at + n] = torch.einsum("rn,nk->rk", dy, w[e])
            dw[e] = torch.einsum("rn,rk->nk", dy, x)
        return {"dxs": dxs, "dw": dw.reshape(st["w"].shape)}
    x = _exact_values(st["x"]) if op == "mx4_mm" else st["x" if four else "xs"].double()
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    for e, (at, n) in enumerate(st["groups"]):
        y[at: at + n] = torch.einsum("rk,nk->rn", x[at: at + n], w[e])
    return y
