"""Cases for the operators around the quantizer: the products that read FP4 codes (grouped by
expert, over ragged rows and over a ragged contraction; with low-rank adapters beside a shared
projection) and the norms before and after a block.

Plain forms (own = False) are elementary torch operations in fp32, rounded once at the end.
With own = True, run() makes the calls that a user makes of the library.
"""
import math
import random

import torch

own = False

EPS = 1e-6
NV, MX = "nvfp4", "mxfp4"


def listed():
    return [
        # One token at its 8 experts (decoding a single stream): latency and the weights' bytes.
        dict(name="experts_one_token", op="grouped", fmt=NV, tokens=1, topk=8, E=64, N=2048, K=4096),
        # A batch of 64 decoding requests, the down projection: a few rows per expert, some none.
        dict(name="experts_decode_batch", op="grouped", fmt=MX, tokens=64, topk=8, E=64, N=4096, K=2048),
        # Prompts of 4096 tokens in all at 8 experts each: large ragged groups.
        dict(name="experts_prompt", op="grouped", fmt=NV, tokens=4096, topk=8, E=64, N=2048, K=4096),
        # A small model with sizes that divide nothing: ragged rows, ragged N, a partial K block.
        dict(name="experts_ragged", op="grouped", fmt=MX, tokens=411, topk=3, E=12, N=1100, K=1056),
        # The weight gradients of a training micro-batch, both operands quantized along the tokens.
        dict(name="wgrad_experts", op="wgrad", fmt=NV, T=8192, E=16, N=2048, K=4096),
        # The same at sizes that divide nothing, experts without a token among them.
        dict(name="wgrad_ragged", op="wgrad", fmt=MX, T=1536, E=8, N=1100, K=1376),
        # 32 decoding requests, 24 adapters, beside a shared square projection.
        dict(name="adapters_decode", op="lora", fmt=NV, M=32, N=4096, K=4096, n=24, R=16, run=1),
        # Prompts of some 200 tokens each with their adapters.
        dict(name="adapters_prompt", op="lora", fmt=NV, M=4096, N=8192, K=4096, n=8, R=64, run=200),
        # One decoding token through the norms on both sides of a block.
        dict(name="norm_one_token", op="norm", M=1, D=4096, dtype="bf16", gate="channel", post=True, y=True),
        # A prompt or a training micro-batch.
        dict(name="norm_prompt", op="norm", M=16384, D=8192, dtype="bf16", gate="channel", post=True, y=True),
        # The gradients of a training micro-batch.
        dict(name="norm_grad", op="norm_bwd", M=8192, D=8192, dtype="bf16", gate="channel", post=True, y=True),
        # A narrow fp32 model, a gate per token, an odd number of rows.
        dict(name="norm_grad_ragged", op="norm_bwd", M=1021, D=1360, dtype="f32", gate="token", post=True, y=True),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(v / mult) * mult)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "lora", "norm", "norm_bwd"])
    fmt = rng.choice([NV, MX])
    if op == "grouped":
        E = _log(rng, 2, 128)
        topk = rng.randint(1, min(8, E))
        N, K = _log(rng, 64, 4096), _log(rng, 64, 8192, 32)
        most = min(6000, int(4096 * 8 * 2048 * 4096 / (N * K * topk)))
        return dict(op=op, fmt=fmt, tokens=_log(rng, 1, most), topk=topk, E=min(E, int(2 ** 29 / (N * K)) + topk), N=N, K=K)
    if op == "wgrad":
        return dict(op=op, fmt=fmt, T=_log(rng, 128, 8192, 128), E=_log(rng, 1, 16), N=_log(rng, 64, 2048), K=_log(rng, 64, 4096, 8))
    if op == "lora":
        N = _log(rng, 64, 8192)
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 4096), N=N, K=_log(rng, 64, 4096, 32), n=_log(rng, 1, 32),
                    R=rng.choice([8, 16, 24, 32, 64]), run=rng.choice([1, 3, 50, 300]))
    y = rng.random() < 0.85
    D = _log(rng, 64, 30000, 16)
    return dict(op=op, M=_log(rng, 1, max(2, min(40000, 32_000_000 // D))), D=D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                gate=rng.choice(["channel", "token", "full", "none"]) if y else "none",
                post=y and rng.random() < 0.7, y=y)


# ---- inputs -------------------------------------------------------------------------------


def _sizes(case, seed):
    """Rows per expert: every token takes its topk best of E skewed random scores."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    score = torch.randn(case["E"], generator=g) + torch.randn((case["tokens"], case["E"]), generator=g)
    return torch.bincount(score.topk(case["topk"], dim=1).indices.reshape(-1), minlength=case["E"])


def _lengths(case, seed):
    """Tokens per expert padded to 128 each, T in all; and how many of them are real."""
    r = random.Random(seed * 11 + 3)
    units = torch.bincount(torch.tensor([int(r.random() ** 1.6 * case["E"]) for _ in range(case["T"] // 128)]),
                           minlength=case["E"])
    real = torch.tensor([128 * int(u) - (r.randint(0, 127) if u else 0) for u in units])
    return 128 * units, real


def _codes(v, fmt):
    """Codes, scale bytes and the per-tensor scale of fp32 `v`, blocks along the last axis."""
    b = v.unflatten(-1, (-1, 16 if fmt == NV else 32))
    top = b.abs().amax(-1)
    if fmt == NV:
        sg = (v.abs().amax() / 2688).reshape(1)
        s = (top / 6 / sg).clamp(max=448).to(torch.float8_e4m3fn)
        step, s = s.float() * sg, s.view(torch.uint8)
    else:
        sg = None
        e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
        e = torch.where(top > 0, e, torch.full_like(e, -127))
        step, s = torch.ldexp(torch.ones_like(top), e), (e + 127).to(torch.uint8)
    q = b / torch.where(step == 0, torch.ones_like(step), step).unsqueeze(-1)
    m = q.abs()
    c = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    c = (c | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s.contiguous(), sg


def _tiles(s):
    """Scale bytes [.., rows, cols] in the tile layout of block-scaled products: tiles of 128 rows x 4
    columns, row r and column c of a tile at byte (r % 32) * 16 + (r // 32) * 4 + c."""
    rows, cols = s.shape[-2:]
    s = torch.nn.functional.pad(s, (0, -cols % 4, 0, -rows % 128))
    s = s.unflatten(-2, (-1, 4, 32)).unflatten(-1, (-1, 4))  # .., tile row, r // 32, r % 32, tile col, c
    return s.movedim(-2, -4).transpose(-3, -2).flatten(-5).contiguous()


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator("cuda").manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale)

    def acts(rows, cols):  # activations: a few channels far larger than the rest
        v = rand(rows, cols)
        v[:, torch.randint(cols, (max(1, cols // 100),), generator=g, device="cuda")] *= 8
        return v

    s = dict(case)
    if op == "grouped":
        E, N, K = case["E"], case["N"], case["K"]
        sizes = _sizes(case, seed)
        M = int(sizes.sum())
        s["xq"], s["xs"], s["x_sg"] = _codes(acts(M, K), case["fmt"])
        s["wq"], s["ws"], w_sg = _codes(rand(E, N, K, scale=K ** -0.5), case["fmt"])
        s["w_sg"] = None if w_sg is None else w_sg.expand(E) * (0.5 + torch.rand(E, generator=g, device="cuda"))
        s["ws_tiles"] = _tiles(s["ws"])
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = sizes.cumsum(0)
        s["offsets"] = off.cuda()
        # what the plain form indexes by: the experts that have rows, and where each row goes among them
        s["active"] = sizes.nonzero()[:, 0].cuda()
        place = (sizes > 0).cumsum(0) - 1
        s["row_expert"] = place.repeat_interleave(sizes).cuda()
        s["row_slot"] = (torch.arange(M) - off[:-1].repeat_interleave(sizes)).cuda()
        s["most"] = int(sizes.max())
    elif op == "wgrad":
        E, N, K = case["E"], case["N"], case["K"]
        padded, real = _lengths(case, seed)
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = padded.cumsum(0)
        T = int(off[-1])
        at = torch.arange(T) - off[:-1].repeat_interleave(padded)
        live = (at < real.repeat_interleave(padded)).cuda()
        s["gq"], s["gs"], s["g_sg"] = _codes(rand(N, T, scale=0.01) * live, case["fmt"])
        s["xq"], s["xs"], s["x_sg"] = _codes(acts(T, K).t().contiguous() * live, case["fmt"])
        s["gs_tiles"], s["xs_tiles"] = _tiles(s["gs"]), _tiles(s["xs"])
        s["offsets"] = off.cuda()
        most = max(1, int(padded.max()))
        cols = off[:-1, None] + torch.arange(most)
        s["cols"] = cols.clamp(max=T - 1).long().cuda()
        s["inside"] = (torch.arange(most) < padded[:, None]).cuda()
    elif op == "lora":
        M, N, K, n, R = (case[k] for k in "MNKnR")
        x = acts(M, K).to(torch.bfloat16)
        s["x"] = x
        s["xq"], s["xs"], s["x_sg"] = _codes(x.float(), case["fmt"])
        s["wq"], s["ws"], s["w_sg"] = _codes(rand(N, K, scale=K ** -0.5), case["fmt"])
        s["ws_tiles"] = _tiles(s["ws"])
        s["a"] = rand(n, R, K, scale=K ** -0.5).to(torch.bfloat16)
        s["b"] = rand(n, N, R, scale=R ** -0.5).to(torch.bfloat16)
        s["scaling"] = 0.25 + torch.rand(n, generator=g, device="cuda")
        # requests one after another, each of some tokens and with its adapter; one in ten without
        r = random.Random(seed * 13 + 5)
        ids = []
        while len(ids) < M:
            length = 1 if case["run"] == 1 else r.randint(1, 2 * case["run"])
            ids += [r.randrange(n) if r.random() < 0.9 else -1] * length
        s["ids"] = torch.tensor(ids[:M], dtype=torch.int32).cuda()
    else:
        M, D = case["M"], case["D"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["alpha"] = 0.75 if case["gate"] == "token" else 1.0
        s["h"] = (acts(M, D) * 2).to(dt)
        s["y"] = rand(M, D).to(dt) if case["y"] else None
        s["w_post"] = 1 + rand(D, scale=0.1) if case["post"] else None
        s["w_pre"] = 1 + rand(D, scale=0.1)
        shape = {"channel": (D,), "token": (M, 1), "full": (M, D)}.get(case["gate"])
        s["gate"] = None if shape is None else rand(*shape, scale=0.5)
        if case["gate"] == "full":
            s["gate"] = s["gate"].to(dt)
        if op == "norm_bwd":  # what the forward call kept: h after the block and the rows' reciprocal norms
            s["r_post"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS) if case["post"] else None
            s["r_pre"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dh_out"], s["dn"] = rand(M, D, scale=0.1).to(dt), rand(M, D, scale=0.1).to(dt)
    return s


# ---- the plain forms ------------------------------------------------------------------------


def _grid():
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    byte = torch.arange(256, device="cuda")
    return torch.stack([one[byte & 15], one[byte >> 4]], 1)


def _values(q, scales, sg, fmt):
    """The fp32 values that codes and scale bytes stand for."""
    if fmt == NV:
        s = scales.view(torch.float8_e4m3fn).float() * sg
    else:
        s = torch.ldexp(torch.ones((), device="cuda"), scales.int() - 127)
    v = _grid()[q.long()].flatten(-2)
    return (v.unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


def _plain_grouped(s):
    x = _values(s["xq"], s["xs"], s["x_sg"], s["fmt"])
    pick = s["active"]
    w_sg = None if s["w_sg"] is None else s["w_sg"][pick][:, None, None]
    w = _values(s["wq"][pick], s["ws"][pick], w_sg, s["fmt"])
    padded = torch.zeros((pick.numel(), s["most"], s["K"]), device="cuda")
    padded[s["row_expert"], s["row_slot"]] = x
    return (padded @ w.transpose(1, 2))[s["row_expert"], s["row_slot"]].to(torch.bfloat16)


def _plain_wgrad(s):
    g = _values(s["gq"], s["gs"], s["g_sg"], s["fmt"])[:, s["cols"]] * s["inside"]
    x = _values(s["xq"], s["xs"], s["x_sg"], s["fmt"])[:, s["cols"]] * s["inside"]
    return (g.transpose(0, 1) @ x.permute(1, 2, 0)).to(torch.bfloat16)


def _plain_lora(s):
    y = _values(s["xq"], s["xs"], s["x_sg"], s["fmt"]) @ _values(s["wq"], s["ws"], s["w_sg"], s["fmt"]).t()
    a, b = s["a"].float(), s["b"].float()
    t = (s["x"].float() @ a.flatten(0, 1).t()).unflatten(1, a.shape[:2])
    mine = s["ids"][:, None] == torch.arange(a.shape[0], device="cuda")
    t = t * (mine * s["scaling"])[:, :, None]
    return (y + t.flatten(1) @ b.transpose(1, 2).flatten(0, 1)).to(torch.bfloat16)


def _plain_norm(s):
    dt = s["h"].dtype
    t, out = s["h"].float(), {}
    if s["y"] is not None:
        u = s["y"].float()
        if s["post"]:
            out["r_post"] = torch.rsqrt(u.square().mean(1) + EPS)
            u = u * out["r_post"][:, None] * s["w_post"]
        if s["gate"] is not None:
            u = u * s["gate"].float()
        t = s["alpha"] * t + u
        out["h_out"] = t.to(dt)
    out["r_pre"] = torch.rsqrt(t.square().mean(1) + EPS)
    out["n"] = (t * out["r_pre"][:, None] * s["w_pre"]).to(dt)
    return out


def _plain_norm_bwd(s):
    dt = s["h"].dtype
    h, dn, r = s["h"].float(), s["dn"].float(), s["r_pre"][:, None]
    gn = dn * s["w_pre"]
    d = s["dh_out"].float() + r * gn - h * r ** 3 * (gn * h).mean(1, keepdim=True)
    out = {"dw_pre": (dn * h * r).sum(0)}
    if s["y"] is None:
        out["dh"] = d.to(dt)
        return out
    out["dh"] = (s["alpha"] * d).to(dt)
    y = s["y"].float()
    xhat = y * s["r_post"][:, None] if s["post"] else y
    u = xhat * s["w_post"] if s["post"] else y
    if s["gate_kind"] == "channel":
        out["dgate"] = (d * u).sum(0)
    elif s["gate_kind"] == "token":
        out["dgate"] = (d * u).sum(1, keepdim=True)
    elif s["gate_kind"] == "full":
        out["dgate"] = (d * u).to(dt)
    du = d if s["gate"] is None else d * s["gate"].float()
    if s["post"]:
        out["dw_post"] = (du * xhat).sum(0)
        gy, rp = du * s["w_post"], s["r_post"][:, None]
        du = rp * gy - y * rp ** 3 * (gy * y).mean(1, keepdim=True)
    out["dy"] = du.to(dt)
    return out


# ---- one pass -------------------------------------------------------------------------------


def run(s):
    op, nv = s["op"], s.get("fmt") == NV
    if op in ("norm", "norm_bwd"):
        s = dict(s, gate_kind="none" if s["gate"] is None else
                 "channel" if s["gate"].dim() == 1 else "token" if s["gate"].shape[1] == 1 else "full")
    if not own:
        return {"grouped": _plain_grouped, "wgrad": _plain_wgrad, "lora": _plain_lora, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd}[op](s)
    import hadamard_rotation_gb300 as hq
    if op == "grouped":
        if nv:
            return hq.hq_grouped_gemm_nvfp4(s["xq"], s["xs"], s["x_sg"], s["wq"], s["ws_tiles"], s["w_sg"], s["offsets"])
        return hq.hq_grouped_gemm_mxfp4(s["xq"], s["xs"], s["wq"], s["ws_tiles"], s["offsets"])
    if op == "wgrad":
        if nv:
            return hq.hq_grouped_wgrad_nvfp4(s["gq"], s["gs_tiles"], s["g_sg"], s["xq"], s["xs_tiles"], s["x_sg"], s["offsets"])
        return hq.hq_grouped_wgrad_mxfp4(s["gq"], s["gs_tiles"], s["xq"], s["xs_tiles"], s["offsets"])
    if op == "lora":
        if nv:
            return hq.hq_lora_gemm_nvfp4(s["xq"], s["xs"], s["x_sg"], s["wq"], s["ws_tiles"], s["w_sg"],
                                         s["x"], s["a"], s["b"], s["scaling"], s["ids"])
        return hq.hq_lora_gemm_mxfp4(s["xq"], s["xs"], s["wq"], s["ws_tiles"], s["x"], s["a"], s["b"], s["scaling"], s["ids"])
    if op == "norm":
        h_out, n, r_post, r_pre = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], alpha=s["alpha"],
                                                   eps=EPS, post_norm=s["post"])
        out = {"h_out": h_out if s["y"] is not None else None, "n": n, "r_post": r_post, "r_pre": r_pre}
    else:
        dh, dy, dw_post, dgate, dw_pre = hq.hq_block_norm_bwd(
            s["dh_out"], s["dn"], s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["r_post"], s["r_pre"],
            alpha=s["alpha"], post_norm=s["post"])
        out = {"dh": dh, "dy": dy, "dw_post": dw_post, "dgate": dgate, "dw_pre": dw_pre}
    return {k: v for k, v in out.items() if v is not None}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        es = 2 if case["dtype"] == "bf16" else 4
        M, D = case["M"], case["D"]
        full = {"full": M * D * es, "channel": 4 * D, "token": 4 * M, "none": 0}[case["gate"]]
        vec = 4 * D * (1 + case["post"]) + 4 * M * (1 + case["post"])
        if op == "norm":
            return {"bytes": M * D * es * (4 if case["y"] else 2) + full + vec, "flops": 12.0 * M * D}
        return {"bytes": M * D * es * (6 if case["y"] else 4) + 2 * full + 2 * vec, "flops": 30.0 * M * D}
    size = 0.5 + (1 / 16 if case["fmt"] == NV else 1 / 32)
    N, K = case["N"], case["K"]
    if op == "grouped":
        sizes = _sizes(case, 0)
        M, live = int(sizes.sum()), int((sizes > 0).sum())
        return {"bytes": size * (M * K + live * N * K) + 2 * M * N, "flops": 2.0 * M * N * K}
    if op == "wgrad":
        return {"bytes": size * case["T"] * (N + K) + 2 * case["E"] * N * K, "flops": 2.0 * case["T"] * N * K}
    M, n, R = case["M"], case["n"], case["R"]
    seen = min(n, M // case["run"] + 1)
    return {"bytes": size * (M * K + N * K) + 2 * M * K + 2 * M * N + 2 * seen * R * (N + K),
            "flops": 2.0 * M * N * K + 2.0 * M * R * (N + K)}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]

    def real(q, b, sg):
        """Codes by their sign, exponent and mantissa bits; scales by theirs."""
        c = torch.stack([q & 15, q >> 4], -1).flatten(-2).int()
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, m / 2, (2 + m) * torch.exp2(e.double() - 2))
        v = torch.where(c >= 8, -v, v)
        b = b.int()
        if case["fmt"] == NV:
            e, m = (b >> 3) & 15, (b & 7).double()
            t = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
            return v * (t * sg.double()).repeat_interleave(16, -1)
        return v * torch.exp2(b.double() - 127).repeat_interleave(32, -1)

    if op == "grouped":
        off = s["offsets"].tolist()
        out = torch.zeros((off[-1], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if b > a:
                x = real(s["xq"][a:b], s["xs"][a:b], s["x_sg"])
                w = real(s["wq"][e], s["ws"][e], None if s["w_sg"] is None else s["w_sg"][e])
                out[a:b] = x.mm(w.t())
        return out
    if op == "wgrad":
        off = s["offsets"].tolist()
        g, x = real(s["gq"], s["gs"], s["g_sg"]), real(s["xq"], s["xs"], s["x_sg"])
        return torch.stack([g[:, off[e]:off[e + 1]].mm(x[:, off[e]:off[e + 1]].t()) for e in range(case["E"])])
    if op == "lora":
        out = real(s["xq"], s["xs"], s["x_sg"]).mm(real(s["wq"], s["ws"], s["w_sg"]).t())
        for k in range(case["n"]):
            rows = (s["ids"] == k).nonzero()[:, 0]
            t = s["x"][rows].double().mm(s["a"][k].double().t())
            out[rows] += s["scaling"][k].double() * t.mm(s["b"][k].double().t())
        return out
    D = case["D"]
    d64 = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    h, y, gate, wq, wp = d64["h"], d64["y"], d64["gate"], d64["w_pre"], d64["w_post"]
    gate = torch.ones((), dtype=torch.float64, device="cuda") if gate is None else gate
    if op == "norm":
        out = {}
        if y is not None:
            if case["post"]:
                out["r_post"] = 1 / ((y * y).sum(1) / D + EPS).sqrt()
                y = y * out["r_post"].unsqueeze(1) * wp
            h = s["alpha"] * h + gate * y
            out["h_out"] = h
        out["r_pre"] = 1 / ((h * h).sum(1) / D + EPS).sqrt()
        out["n"] = wq * h * out["r_pre"].unsqueeze(1)
        return out
    # v_j = w_j x_j r and dr/dx_i = -r^3 x_i / D, so dx_i = r w_i dv_i - x_i r^3 / D sum_j w_j dv_j x_j
    r, dn = d64["r_pre"].unsqueeze(1), d64["dn"]
    d = d64["dh_out"] + r * wq * dn - h * r.pow(3) / D * (wq * dn * h).sum(1, keepdim=True)
    out = {"dw_pre": (dn * h * r).sum(0)}
    if y is None:
        return {**out, "dh": d}
    out["dh"] = s["alpha"] * d
    v = y * d64["r_post"].unsqueeze(1) if case["post"] else y
    u = v * wp if case["post"] else v
    if case["gate"] != "none":
        du = d * u
        out["dgate"] = du.sum(0) if case["gate"] == "channel" else du.sum(1, keepdim=True) if case["gate"] == "token" else du
    e = d * gate
    if case["post"]:
        out["dw_post"] = (e * v).sum(0)
        r = d64["r_post"].unsqueeze(1)
        e = r * wp * e - y * r.pow(3) / D * (wp * e * y).sum(1, keepdim=True)
    out["dy"] = e
    return out
