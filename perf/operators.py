"""Workloads of the operators around the experts' products of an MoE block:

  block_norm        norms before and after a block with its gate and residual scale, and the backward
  moe_permute       tokens sorted by expert and back with the routing weights, and the backward
  checkpoint        activations kept in 8 bits, and the SwiGLU backward that reads them

run() computes an operator in elementary torch operations in 32 bits, or, with
`own`, through the package.  exact() is the definition in 64 bits.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32          # columns that share one scale of an 8-bit checkpoint
EPS = 1e-5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decode step between two sub-layers: latency
        dict(name="norm_t1_h768", op="norm", T=1, H=768, dtype="bf16", post=True, pre=True, gate="channel", s=1.0),
        # the training batch of the top-2 MoE workload, sandwich norms with a learned gate
        dict(name="norm_t16384_h768", op="norm", T=16384, H=768, dtype="bf16", post=True, pre=True, gate="channel", s=0.9),
        # a wide model whose gate is computed per token, next sub-layer's norm only
        dict(name="norm_t16384_h4096_tokengate", op="norm", T=16384, H=4096, dtype="bf16", post=False, pre=True, gate="token", s=1.0),
        # gradients of the training batch: both norms' weights and the gate
        dict(name="norm_bwd_t16384_h768", op="norm_bwd", T=16384, H=768, dtype="bf16", post=True, pre=True, gate="channel", s=0.9),
        # odd width in fp32: no row but the first is aligned to 16 bytes
        dict(name="norm_bwd_t4097_h1001_f32", op="norm_bwd", T=4097, H=1001, dtype="f32", post=True, pre=True, gate=None, s=1.0),
        # a decode batch sorted by expert: latency
        dict(name="permute_t16_e8k2", op="permute", T=16, H=768, E=8, k=2, align=1, drop=0.0, dtype="bf16"),
        # the top-2 workload's tokens, skewed load
        dict(name="permute_t16384_e8k2", op="permute", T=16384, H=768, E=8, k=2, align=64, drop=0.0, dtype="bf16"),
        # and back, weighted
        dict(name="unpermute_t16384_e8k2", op="unpermute", T=16384, H=768, E=8, k=2, align=64, drop=0.0, dtype="bf16"),
        # gradient of the combine: many experts, ragged token count, a share of the experts elsewhere
        dict(name="unpermute_bwd_t8191_e64k8", op="unpermute_bwd", T=8191, H=2048, E=64, k=8, align=16, drop=0.25, dtype="bf16"),
        # the top-2 workload's expert rows: SwiGLU with its checkpoint, and the backward from it
        dict(name="act_save_r32768_i2432", op="act", R=32768, I=2432, dtype="bf16"),
        dict(name="act_bwd_r32768_i2432", op="act_bwd", R=32768, I=2432, dtype="bf16"),
        # a layer input kept in 8 bits and read back, the dense workload's tokens at an odd width
        dict(name="checkpoint_r4096_c1000", op="checkpoint", R=4096, C=1000, dtype="bf16"),
    ]


MOST_BYTES = 750e6


def _between(rng, lo, hi):
    """Log-uniform whole number in [lo, hi]."""
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "permute", "unpermute", "permute_bwd", "unpermute_bwd", "act", "act_bwd", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    width = _between(rng, 64, 8192)
    if rng.random() < 0.75:
        width = max(64, width // 64 * 64)       # model widths; the rest are odd ones
    rows = _between(rng, 1, 32768)
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, T=min(rows, 16384), H=width, dtype=dtype, post=rng.random() < 0.7, pre=rng.random() < 0.8,
                 gate=rng.choice([None, "channel", "channel", "token"]), s=rng.choice([1.0, 0.5, 0.9]))
        key = "T"
    elif op in ("permute", "unpermute", "permute_bwd", "unpermute_bwd"):
        E = rng.choice([2, 4, 8, 8, 16, 32, 64])
        c = dict(op=op, T=min(rows, 16384), H=width, E=E, k=rng.randint(1, min(8, E)), align=rng.choice([1, 1, 16, 64, 128]),
                 drop=rng.choice([0.0, 0.0, 0.5]), dtype=dtype)
        key = "T"
    elif op in ("act", "act_bwd"):
        c = dict(op=op, R=rows, I=width, dtype=dtype)
        key = "R"
    else:
        c = dict(op=op, R=rows, C=width, dtype=dtype)
        key = "R"
    while work(c)["bytes"] > MOST_BYTES:
        c[key] = c[key] // 2
    return c


def permuted_rows(c):
    """Rows of the sorted tensor: every assignment, and each group's padding at its most."""
    return c["T"] * c["k"] + min(c["E"], c["T"] * c["k"]) * (c["align"] - 1)


def work(c):
    """Each input read once, each output written once."""
    op, es = c["op"], 2 if c["dtype"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        n, vec = c["T"] * c["H"], c["H"]
        token, chan = c["gate"] == "token", c["gate"] == "channel"
        if op == "norm":
            big = 3 + c["pre"] + token                                  # x, f, (gate); r, (n)
            return {"bytes": n * es * big + vec * es * (c["post"] + c["pre"] + chan) + 4 * c["T"] * (c["post"] + c["pre"]),
                    "flops": n * (3 + 4 * c["post"] + 4 * c["pre"])}
        needs_f = c["post"] or c["gate"] is not None
        big = 3 + needs_f + 2 * c["pre"] + 2 * token                    # dr, f, (r, dn), (gate); dx, df, (d_gate)
        return {"bytes": n * es * big + vec * (es + 4) * (c["post"] + c["pre"] + chan) + 4 * c["T"] * (c["post"] + c["pre"]),
                "flops": n * (4 + 10 * c["post"] + 10 * c["pre"] + 3 * (c["gate"] is not None))}
    if op in ("permute", "unpermute", "permute_bwd", "unpermute_bwd"):
        a, row = c["T"] * c["k"] * (1 - c["drop"]), c["H"] * es
        one = c["T"] * row
        if op == "permute":
            return {"bytes": one + a * row + 12 * c["T"] * c["k"], "flops": 0}
        if op == "unpermute_bwd":
            return {"bytes": one + 2 * a * row + 12 * c["T"] * c["k"], "flops": 3 * a * c["H"]}
        return {"bytes": one + a * row + (8 if op == "unpermute" else 4) * c["T"] * c["k"], "flops": 2 * a * c["H"]}
    if op in ("act", "act_bwd"):
        n, groups = c["R"] * c["I"], c["R"] * 2 * -(-c["I"] // GROUP)
        if op == "act":
            return {"bytes": n * (3 * es + 2) + groups, "flops": 12 * n}
        return {"bytes": n * (4 * es + 2) + groups, "flops": 14 * n}
    n, groups = c["R"] * c["C"], c["R"] * -(-c["C"] // GROUP)
    return {"bytes": 2 * (n * (es + 1) + groups), "flops": 4 * n}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dt)

    st = dict(case=case, op=case["op"], dtype=dt)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        # a residual stream has channels far larger than the rest
        loud = 1.0 + 9.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        x = (torch.randn(T, H, generator=g, device="cuda") * loud).to(dt)
        st.update(x=x, f=normal(T, H, std=0.5), s=case["s"],
                  post=normal(H, std=0.1, mean=1.0) if case["post"] else None,
                  pre=normal(H, std=0.1, mean=1.0) if case["pre"] else None,
                  gate={None: None, "channel": normal(H, std=0.2, mean=0.5) if case["gate"] == "channel" else None,
                        "token": torch.sigmoid(normal(T, H).float()).to(dt) if case["gate"] == "token" else None}[case["gate"]])
        # the buffers that a step keeps
        st.update(r=torch.empty_like(x), n=torch.empty_like(x) if case["pre"] else None)
        st["stats"] = {k: torch.empty(T, device="cuda") for k in ("rstd_post", "rstd_pre")}
        if op == "norm_bwd":
            r, n, rf, rr = _norm(st)
            st.update(r=r, dr=normal(T, H, std=0.01), dn=normal(T, H, std=0.02) if case["pre"] else None)
            st["stats"] = {"rstd_post": rf, "rstd_pre": rr}
        return st
    if op in ("permute", "unpermute", "permute_bwd", "unpermute_bwd"):
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        logits = torch.randn(T, E, generator=g, device="cuda")
        logits[:, 0] += 1.5
        logits[:, 1] += 0.5
        top = logits.topk(k, dim=1)
        idx = top.indices.to(torch.int32)
        if case["drop"]:
            idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, idx)
        w = torch.softmax(top.values, dim=1).contiguous()
        R = permuted_rows(case)
        st.update(idx=idx.contiguous(), w=w, E=E, align=case["align"], R=R)
        if op == "permute":
            st.update(x=normal(T, H), xs=torch.zeros(R, H, dtype=dt, device="cuda"))
            return st
        plan = _sort(st)
        st["plan"] = plan
        st["ys"] = normal(R, H)
        if op == "unpermute_bwd":
            st.update(dy=normal(T, H, std=0.05), dys=torch.zeros(R, H, dtype=dt, device="cuda"))
        else:
            st["y"] = torch.empty(T, H, dtype=dt, device="cuda")
        return st
    if op in ("act", "act_bwd"):
        R, I = case["R"], case["I"]
        spread = torch.exp(0.5 * torch.randn(R, 1, generator=g, device="cuda"))
        gu = (torch.randn(R, 2 * I, generator=g, device="cuda") * spread).to(dt)
        if op == "act":
            st.update(gu=gu, h=torch.empty(R, I, dtype=dt, device="cuda"),
                      ckpt=dict(codes=torch.empty(R, 2 * I, dtype=torch.float8_e4m3fn, device="cuda"),
                                exps=torch.empty(R, 2 * -(-I // GROUP), dtype=torch.uint8, device="cuda"), segments=2))
            return st
        codes, exps = _quantise(gu.float().view(2 * R, I))
        st.update(ckpt=dict(codes=codes.view(R, 2 * I), exps=exps.view(R, -1), segments=2), dh=normal(R, I, std=0.02),
                  dgu=torch.empty(R, 2 * I, dtype=dt, device="cuda"), h=torch.empty(R, I, dtype=dt, device="cuda"))
        return st
    st["x"] = normal(case["R"], case["C"])
    return st


# ----------------------------------------------------- plain forms, 32 bits
def _norm(st):
    """(r, n, rstd of f, rstd of r); n is the norm of r as stored."""
    x, f, dt = st["x"].float(), st["f"].float(), st["dtype"]
    rf = rr = n = None
    p = f
    if st["post"] is not None:
        rf = torch.rsqrt((f * f).mean(1) + EPS)
        p = f * rf[:, None] * st["post"].float()
    if st["gate"] is not None:
        p = p * st["gate"].float()
    r = (st["s"] * x + p).to(dt)
    if st["pre"] is not None:
        r32 = r.float()
        rr = torch.rsqrt((r32 * r32).mean(1) + EPS)
        n = (r32 * rr[:, None] * st["pre"].float()).to(dt)
    return r, n, rf, rr


def _norm_backward(st):
    dt, f, H = st["dtype"], st["f"].float(), st["f"].shape[1]
    out = {}
    D = st["dr"].float()
    if st["pre"] is not None:
        r, dn, rr = st["r"].float(), st["dn"].float(), st["stats"]["rstd_pre"][:, None]
        v = dn * st["pre"].float()
        D = D + rr * v - r * (rr * rr * rr * ((r * v).sum(1, keepdim=True) / H))
        out["d_pre_weight"] = (dn * r * rr).sum(0)
    out["dx"] = (st["s"] * D).to(dt)
    p = f
    if st["post"] is not None:
        rf = st["stats"]["rstd_post"][:, None]
        p = f * rf * st["post"].float()
    q = D
    if st["gate"] is not None:
        dg = D * p
        out["d_gate"] = dg.to(dt) if st["gate"].dim() == 2 else dg.sum(0)
        q = D * st["gate"].float()
    if st["post"] is not None:
        v = q * st["post"].float()
        out["d_post_weight"] = (q * f * rf).sum(0)
        q = rf * v - f * (rf * rf * rf * ((f * v).sum(1, keepdim=True) / H))
    out["df"] = q.to(dt)
    return out


def _sort(st):
    """The rows of every assignment, sorted by expert, then token, then slot."""
    idx, E, align = st["idx"], st["E"], st["align"]
    flat = idx.reshape(-1).long()
    keep = (flat >= 0) & (flat < E)
    key = torch.where(keep, flat, E)
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.argsort(key, stable=True)
    first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=key.device) - first[key[order]]
    pos = torch.where(keep, offsets[key] + rank, -1)
    perm = torch.full((st["R"] + 1,), -1, dtype=torch.int32, device=key.device)     # the last one takes the dropped
    perm[torch.where(keep, pos, st["R"])] = torch.arange(order.numel(), device=key.device, dtype=torch.int32)
    return dict(offsets=offsets.int(), counts=counts.int(), perm=perm[:-1].contiguous(), pos=pos.int().view(idx.shape))


def _gather(rows, pos):
    """[T, k, H] in 32 bits: each assignment's row, zeros for a dropped one."""
    got = rows[pos.clamp(min=0).long()].float()
    return got * (pos >= 0)[..., None]


def _scatter(values, pos, R, dt):
    """Rows of [T, k, H] values at pos; zeros elsewhere."""
    out = torch.zeros(R + 1, values.shape[-1], dtype=dt, device=values.device)
    out[torch.where(pos >= 0, pos, R).long().reshape(-1)] = values.reshape(-1, values.shape[-1]).to(dt)
    return out[:-1]


def _quantise(x):
    """e4m3 codes and biased exponents of groups of 32 columns, the last one short."""
    R, C = x.shape
    G = -(-C // GROUP)
    padded = torch.zeros(R, G * GROUP, device=x.device)
    padded[:, :C] = x
    groups = padded.view(R, G, GROUP)
    m, p = torch.frexp(groups.abs().amax(2))            # amax = m 2^p, 0.5 <= m < 1;  448 = 0.875 * 2^9
    e = torch.where(m > 0.875, p - 8, p - 9)
    e = torch.where(m == 0, -126, e).clamp(min=-126)
    codes = torch.ldexp(groups, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(R, G * GROUP)[:, :C].contiguous(), (e + 127).to(torch.uint8)


def _values(codes, exps):
    C = codes.shape[1]
    scale = torch.ldexp(torch.ones((), device=codes.device), exps.int() - 127)
    return codes.float() * scale.repeat_interleave(GROUP, dim=1)[:, :C]


def _plain(st):
    op, dt = st["op"], st["dtype"]
    if op == "norm":
        r, n, rf, rr = _norm(st)
        out = {"r": r, "n": n, "rstd_post": rf, "rstd_pre": rr}
        return {k: v for k, v in out.items() if v is not None}
    if op == "norm_bwd":
        return _norm_backward(st)
    if op == "permute":
        plan = _sort(st)
        xs = _scatter(st["x"][:, None, :].expand(-1, plan["pos"].shape[1], -1), plan["pos"], st["R"], dt)
        return {"xs": xs, **plan}
    if op in ("unpermute", "permute_bwd"):
        rows = _gather(st["ys"], st["plan"]["pos"])
        if op == "unpermute":
            rows = rows * st["w"][..., None]
        return rows.sum(1).to(dt)
    if op == "unpermute_bwd":
        pos, dy = st["plan"]["pos"], st["dy"].float()
        dw = (_gather(st["ys"], pos) * dy[:, None, :]).sum(2)
        return {"dys": _scatter(dy[:, None, :] * st["w"][..., None], pos, st["R"], dt), "dw": dw}
    if op == "act":
        R, two_i = st["gu"].shape
        gu = st["gu"].float()
        g, u = gu[:, : two_i // 2], gu[:, two_i // 2:]
        codes, exps = _quantise(gu.view(2 * R, two_i // 2))
        return {"h": (g / (1 + torch.exp(-g)) * u).to(dt), "codes": codes.view(R, two_i), "exps": exps.view(R, -1)}
    if op == "act_bwd":
        codes, exps = st["ckpt"]["codes"], st["ckpt"]["exps"]
        R, two_i = codes.shape
        gu = _values(codes.view(2 * R, -1), exps.view(2 * R, -1)).view(R, two_i)
        g, u, dh = gu[:, : two_i // 2], gu[:, two_i // 2:], st["dh"].float()
        sig = 1 / (1 + torch.exp(-g))
        silu = g * sig
        return {"dgu": torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * silu], 1).to(dt), "h": (silu * u).to(dt)}
    codes, exps = _quantise(st["x"].float())
    return {"codes": codes, "exps": exps, "x": _values(codes, exps).to(dt)}


# ------------------------------------------------------ the package's calls
def _own(st):
    import swiglu_mlp_top_gb300 as mm
    op = st["op"]
    if op == "norm":
        r, n = mm.block_norm(st["x"], st["f"], post_weight=st["post"], gate=st["gate"], pre_weight=st["pre"],
                             residual_scale=st["s"], eps=EPS, out=st["r"], normed=st["n"], stats=st["stats"])
        out = {"r": r, "n": n, "rstd_post": st["stats"]["rstd_post"] if st["post"] is not None else None,
               "rstd_pre": st["stats"]["rstd_pre"] if st["pre"] is not None else None}
        return {k: v for k, v in out.items() if v is not None}
    if op == "norm_bwd":
        return mm.block_norm_backward(st["dn"], st["dr"], st["r"], st["f"], st["stats"], post_weight=st["post"],
                                      gate=st["gate"], pre_weight=st["pre"], residual_scale=st["s"])
    if op == "permute":
        xs, plan = mm.moe_permute(st["x"], st["idx"], st["E"], align=st["align"], out=st["xs"])
        return {"xs": xs, **plan}
    if op == "unpermute":
        return mm.moe_unpermute(st["ys"], st["plan"], st["w"], out=st["y"])
    if op == "permute_bwd":
        return mm.moe_permute_backward(st["ys"], st["plan"], out=st["y"])
    if op == "unpermute_bwd":
        dys, dw = mm.moe_unpermute_backward(st["dy"], st["ys"], st["plan"], st["w"], out=st["dys"])
        return {"dys": dys, "dw": dw}
    if op == "act":
        h = mm.swiglu_act(st["gu"], checkpoint=st["ckpt"], out=st["h"])
        return {"h": h, "codes": st["ckpt"]["codes"], "exps": st["ckpt"]["exps"]}
    if op == "act_bwd":
        dgu, h = mm.swiglu_act_backward(st["ckpt"], st["dh"], out=st["dgu"], h_out=st["h"])
        return {"dgu": dgu, "h": h}
    ckpt = mm.checkpoint_pack(st["x"])
    return {"codes": ckpt["codes"], "exps": ckpt["exps"], "x": mm.checkpoint_unpack(ckpt, st["dtype"])}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------- the definition, 64 bits
def _exact_checkpoint(x):
    """Codes (their values) and the values they stand for, group by group from the definition."""
    R, C = x.shape
    G = -(-C // GROUP)
    y = torch.nn.functional.pad(x.double(), (0, G * GROUP - C)).view(R, G, GROUP)
    amax = y.abs().amax(2)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140) / 448)) - 1
    for _ in range(3):                                      # the least e with amax <= 448 2^e
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = e.clamp(min=-126)[..., None]
    q = y / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)     # 3 bits behind the first
    q = torch.round(q / step) * step
    return (t.reshape(R, G * GROUP)[:, :C].contiguous() for t in (q, q * torch.exp2(e)))


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "norm":
        p = st["f"].double()
        out = {}
        if st["post"] is not None:
            var = p.square().mean(1) + EPS
            out["rstd_post"] = var.pow(-0.5)
            p = p / var.sqrt()[:, None] * st["post"].double()
        if st["gate"] is not None:
            p = st["gate"].double() * p
        out["r"] = r = p.add_(st["x"].double(), alpha=st["s"])
        if st["pre"] is not None:
            r = r.to(st["dtype"]).double()
            var = r.square().mean(1) + EPS
            out["rstd_pre"] = var.pow(-0.5)
            out["n"] = r / var.sqrt()[:, None] * st["pre"].double()
        return out
    if op == "norm_bwd":
        # the chain rule through unit-length rows: d(v / |v|) projects out the row's own direction
        def through(v, up, rstd):
            unit = v.double() * rstd.double()[:, None]
            return rstd.double()[:, None] * (up - unit * (up * unit).mean(1, keepdim=True)), unit
        out, D = {}, st["dr"].double()
        if st["pre"] is not None:
            dn = st["dn"].double()
            back, unit = through(st["r"], dn * st["pre"].double(), st["stats"]["rstd_pre"])
            out["d_pre_weight"] = (dn * unit).sum(0)
            D = D + back
        out["dx"] = D * st["s"]
        f, gate = st["f"].double(), st["gate"]
        q = D if gate is None else D * gate.double()
        p = f
        if st["post"] is not None:
            back, unit = through(st["f"], q * st["post"].double(), st["stats"]["rstd_post"])
            out["d_post_weight"] = (q * unit).sum(0)
            out["df"], p = back, unit * st["post"].double()
        else:
            out["df"] = q
        if gate is not None:
            out["d_gate"] = D * p if gate.dim() == 2 else (D * p).sum(0)
        return out
    if op == "permute":
        flat = st["idx"].reshape(-1).tolist()
        at, rows = 0, [-1] * st["R"]
        for e in range(st["E"]):
            mine = [a for a, x in enumerate(flat) if x == e]
            rows[at: at + len(mine)] = mine
            at += -(-len(mine) // st["align"]) * st["align"]
        src = torch.tensor(rows, device="cuda")
        token = src.clamp(min=0) // st["idx"].shape[1]
        return {"xs": st["x"].double()[token] * (src >= 0)[:, None], "offsets": None, "counts": None, "perm": None, "pos": None}
    if op in ("unpermute", "permute_bwd"):
        pos, w = st["plan"]["pos"], st["w"].double()
        y = torch.zeros(pos.shape[0], st["ys"].shape[1], dtype=torch.float64, device="cuda")
        for s in range(pos.shape[1]):
            at = (pos[:, s] >= 0).nonzero().flatten()
            rows = st["ys"][pos[at, s].long()].double()
            y[at] += rows * w[at, s, None] if op == "unpermute" else rows
        return y
    if op == "unpermute_bwd":
        pos, w, dy = st["plan"]["pos"], st["w"].double(), st["dy"].double()
        dys = torch.zeros(st["R"], dy.shape[1], dtype=torch.float64, device="cuda")
        dw = torch.zeros(pos.shape, dtype=torch.float64, device="cuda")
        for s in range(pos.shape[1]):
            at = (pos[:, s] >= 0).nonzero().flatten()
            to = pos[at, s].long()
            dys[to] = dy[at] * w[at, s, None]
            dw[at, s] = (dy[at] * st["ys"][to].double()).sum(1)
        return {"dys": dys, "dw": dw}
    if op == "act":
        R, I = case["R"], case["I"]
        g, u = st["gu"].double().split(I, dim=1)
        codes, _ = _exact_checkpoint(st["gu"].view(2 * R, I))
        return {"h": g * torch.sigmoid(g) * u, "codes": codes.view(R, 2 * I), "exps": None}
    if op == "act_bwd":
        R, I = case["R"], case["I"]
        exps = st["ckpt"]["exps"].view(2 * R, -1).double() - 127
        scale = torch.exp2(exps).repeat_interleave(GROUP, dim=1)[:, :I]
        g, u = (st["ckpt"]["codes"].view(2 * R, I).double() * scale).view(R, 2 * I).split(I, dim=1)
        dh, sig = st["dh"].double(), torch.sigmoid(g)
        return {"dgu": torch.cat([dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * g * sig], 1), "h": g * sig * u}
    codes, values = _exact_checkpoint(st["x"])
    return {"codes": codes, "exps": None, "x": values}
