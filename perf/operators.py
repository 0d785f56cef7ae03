"""Cases of the FP8 projection path and of the pooled decode step of a Gated DeltaNet layer.

Operators (the "op" of a case):
  gemm    y = (aq as) (bq bs)^T, E4M3 codes with one fp32 scale per 128 values of a row of `a` and per 128 x 128 block of `b`
  encode  E4M3 codes and block scales of activations (1 x 128) or of a weight (128 x 128)
  tail    per head RMSNorm, times weight, times SiLU(z), as E4M3 codes and block scales
  decode  one token per row through the gated delta rule, states in a pool of slots, the tail's codes as output
  conv    one token per row through the causal short convolution + SiLU, histories in a pool of slots
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
TINY = 2.0 ** -126
DTYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one decoded token through the output projection of the 16/32-head layer: all latency and weight reads
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 2048, "K": 4096, "out": "bf16"},
        # the fused input projection (q, k, v, z, a, b: 12352 columns) of a batch of 256 decoded tokens
        {"name": "gemm_in_proj_256", "op": "gemm", "M": 256, "N": 12352, "K": 2048, "out": "bf16"},
        # a ragged chunk of tokens, partial blocks along every axis, fp32 result
        {"name": "gemm_ragged", "op": "gemm", "M": 1037, "N": 1040, "K": 2064, "out": "f32"},
        # the output projection of the long prefill
        {"name": "gemm_prefill", "op": "gemm", "M": 32768, "N": 2048, "K": 4096, "out": "bf16"},
        # hidden states of a decode batch on their way into the input projection
        {"name": "encode_act_256", "op": "encode", "what": "act", "M": 256, "K": 2048, "io": "bf16"},
        # the input projection's weight, encoded when a checkpoint is loaded
        {"name": "encode_weight", "op": "encode", "what": "weight", "M": 12352, "K": 2048, "io": "bf16"},
        # the gated tail of a ragged chunk of the 16-head layer with fp32 scan outputs
        {"name": "tail_ragged", "op": "tail", "M": 1037, "Hv": 16, "D": 128, "io": "f32"},
        # the gated tail of the long prefill
        {"name": "tail_prefill", "op": "tail", "M": 32768, "Hv": 32, "D": 128, "io": "bf16"},
        # three requests of the 16-head layer, one of the four rows padded
        {"name": "decode_3", "op": "decode", "B": 4, "Hk": 16, "Hv": 16, "slots": 9, "dead": 1, "packed": False},
        # a batch of 256 rows, 6 of them padded, straight from the input projection's output
        {"name": "decode_256", "op": "decode", "B": 256, "Hk": 16, "Hv": 32, "slots": 300, "dead": 6, "packed": True},
        # the convolutions in front of the two decode batches
        {"name": "conv_3", "op": "conv", "B": 4, "C": 6144, "K": 4, "slots": 9, "dead": 1, "row": 6144},
        {"name": "conv_256", "op": "conv", "B": 256, "C": 8192, "K": 4, "slots": 300, "dead": 6, "row": 12352},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "encode", "tail", "decode", "conv"])
    if op == "gemm":
        N, K = 16 * _log(rng, 1, 1024), 16 * _log(rng, 4, 512)
        most = min(32768, 32768 * 2048 * 4096 // (N * K))
        return {"op": op, "M": _log(rng, 1, most), "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "f32"])}
    if op == "encode":
        K = 16 * _log(rng, 1, 1024)
        return {"op": op, "what": rng.choice(["act", "weight"]), "M": _log(rng, 1, min(65536, (1 << 27) // K)), "K": K,
                "io": rng.choice(["bf16", "f32"])}
    if op == "tail":
        D, Hv = rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 5, 16, 32])
        return {"op": op, "M": _log(rng, 1, min(65536, (1 << 27) // (D * Hv))), "Hv": Hv, "D": D, "io": rng.choice(["bf16", "f32"])}
    B = _log(rng, 1, 256)
    slots, dead = B + rng.randrange(45), rng.randrange(B // 4 + 1)
    if op == "decode":
        Hk = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "B": B, "Hk": Hk, "Hv": Hk * rng.choice([1, 2]), "slots": slots, "dead": dead, "packed": rng.random() < 0.5}
    C = 8 * _log(rng, 8, 1024)
    return {"op": op, "B": B, "C": C, "K": rng.choice([2, 3, 4]), "slots": slots, "dead": dead, "row": C + 8 * rng.randrange(100)}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def _activations(g, M, K):
    """Rows of different sizes with a few large channels, as hidden states have them."""
    x = torch.randn(M, K, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=g))
    x *= 1 + 7 * (torch.rand(K, device="cuda", generator=g) < 0.01)
    return x


def _slots(g, case):
    """Distinct slots in any order; `dead` rows of the batch name none (-1)."""
    s = torch.randperm(case["slots"], device="cuda", generator=g)[: case["B"]].to(torch.int32)
    s[torch.randperm(case["B"], device="cuda", generator=g)[: case["dead"]]] = -1
    return s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["aq"], s["as"] = _encode_act(_activations(g, M, K))
        s["bq"], s["bs"] = _encode_weight(_randn(g, N, K) * 0.02)
        s["y"] = torch.empty(M, N, dtype=DTYPES[case["out"]], device="cuda")
    elif op == "encode":
        M, K = case["M"], case["K"]
        s["x"] = (_activations(g, M, K) if case["what"] == "act" else _randn(g, M, K) * 0.02).to(DTYPES[case["io"]])
        s["xq"] = torch.empty(M, K, dtype=E4M3, device="cuda")
        s["xs"] = torch.empty(M if case["what"] == "act" else -(-M // 128), -(-K // 128), device="cuda")
    elif op == "tail":
        M, Hv, D, dt = case["M"], case["Hv"], case["D"], DTYPES[case["io"]]
        s["o"], s["z"] = _randn(g, M, Hv, D, dtype=dt), _randn(g, M, Hv, D, dtype=dt)
        s["w"] = 0.5 + torch.rand(D, device="cuda", generator=g)
        s["xq"] = torch.empty(M, Hv * D, dtype=E4M3, device="cuda")
        s["xs"] = torch.empty(M, -(-Hv * D // 128), device="cuda")
    elif op == "decode":
        B, Hk, Hv, D = case["B"], case["Hk"], case["Hv"], 128
        s["q"], s["k"] = _randn(g, B, Hk, D, dtype=BF16), _randn(g, B, Hk, D, dtype=BF16)
        s["v"] = _randn(g, B, Hv, D, dtype=BF16)
        if case["packed"]:  # columns [.. | z | a | b] of the input projection's rows
            first = (2 * Hk + Hv) * D
            x = _randn(g, B, first + Hv * D + 2 * max(Hv, 4), dtype=BF16)
            s["z"] = x[:, first:first + Hv * D].unflatten(1, (Hv, D))
            s["a"] = x[:, first + Hv * D:][:, :Hv]
            s["b"] = x[:, first + Hv * D + max(Hv, 4):][:, :Hv]
        else:
            s["z"] = _randn(g, B, Hv, D, dtype=BF16)
            s["a"], s["b"] = _randn(g, B, Hv), _randn(g, B, Hv)
        s["A_log"] = torch.rand(Hv, device="cuda", generator=g) * math.log(16.0)
        s["dt_bias"] = torch.zeros(Hv, device="cuda")
        s["w"] = 0.5 + torch.rand(D, device="cuda", generator=g)
        s["pool"] = _randn(g, case["slots"], Hv, D, D) * 0.1
        s["slots"] = _slots(g, case)
        s["xq"] = torch.zeros(B, Hv * D, dtype=E4M3, device="cuda")
        s["xs"] = torch.zeros(B, Hv, device="cuda")
    else:
        B, C, K = case["B"], case["C"], case["K"]
        s["x"] = _randn(g, B, case["row"], dtype=BF16)[:, :C]
        s["w"] = _randn(g, C, K) * K ** -0.5
        s["pool"] = _randn(g, case["slots"], K - 1, C, dtype=BF16)
        s["slots"] = _slots(g, case)
        s["y"] = torch.zeros(B, C, dtype=BF16, device="cuda")
    return s


def _spread(scale, K, rows=1, N=None):
    """Block scales as a factor for each element: [.., blocks] -> [.., K], and each row `rows` times, N of them."""
    f = scale.repeat_interleave(128, dim=-1)[..., :K]
    return f if rows == 1 else f.repeat_interleave(rows, dim=0)[:N]


def _encode_act(x):
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128))
    s = (x.view(M, -1, 128).abs().amax(2) / 448).clamp_min(TINY)
    x = x.view(M, -1, 128) / s[:, :, None]
    return x.view(M, -1)[:, :K].clamp(-448, 448).to(E4M3).contiguous(), s


def _encode_weight(w):
    N, K = w.shape
    w = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    t = w.view(w.shape[0] // 128, 128, -1, 128)
    s = (t.abs().amax((1, 3)) / 448).clamp_min(TINY)
    t = (t / s[:, None, :, None]).view_as(w)
    return t[:N, :K].clamp(-448, 448).to(E4M3).contiguous(), s


def _tail(o, z, w):
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    return (o * r * w * (z * torch.sigmoid(z))).flatten(1)


def _delta(s, S, rows, t):
    """One step of the gated delta rule on the states S of the batch's `rows`, in the type `t`: (o, new S)."""
    c = s["case"]
    q, k, v = (s[n][rows].to(t) for n in ("q", "k", "v"))
    q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + EPS)
    k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + EPS)
    q, k = (x.repeat_interleave(c["Hv"] // c["Hk"], dim=1) for x in (q, k))
    x = s["a"][rows].to(t) + s["dt_bias"].to(t)
    alpha = torch.exp(-torch.exp(s["A_log"].to(t)) * torch.nn.functional.softplus(x))[:, :, None, None]
    beta = torch.sigmoid(s["b"][rows].to(t))[:, :, None]
    S = S * alpha
    u = beta * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    return (S * q[:, :, None, :]).sum(-1), S


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import gated_deltanet_03_b200 as gdn
        if op == "gemm":
            return gdn.fp8_gemm(s["aq"], s["as"], s["bq"], s["bs"], y=s["y"])
        if op == "encode":
            f = gdn.fp8_quantize_act if c["what"] == "act" else gdn.fp8_quantize_weight
            return f(s["x"], s["xq"], s["xs"])
        if op == "tail":
            return gdn.gdn_gated_rmsnorm_silu_fp8(s["o"], s["z"], s["w"], eps=EPS, xq=s["xq"], xs=s["xs"])
        if op == "decode":
            xq, xs, _ = gdn.gdn_decode_step_pooled_gated_fp8(s["q"], s["k"], s["v"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["pool"],
                                                             s["slots"], s["z"], s["w"], eps=EPS, xq=s["xq"], xs=s["xs"])
            return xq, xs, s["pool"]
        return gdn.gdn_short_conv1d_silu_decode_pooled(s["x"], s["w"], s["pool"], s["slots"], y=s["y"]), s["pool"]
    if op == "gemm":
        K, N = c["K"], c["N"]
        a = s["aq"].float() * _spread(s["as"], K)
        b = s["bq"].float() * _spread(s["bs"], K, 128, N)
        return torch.matmul(a, b.t()).to(DTYPES[c["out"]])
    if op == "encode":
        return (_encode_act if c["what"] == "act" else _encode_weight)(s["x"].float())
    if op == "tail":
        return _encode_act(_tail(s["o"].float(), s["z"].float(), s["w"]))
    rows = (s["slots"] >= 0).nonzero().squeeze(1)
    at = s["slots"][rows].long()
    if op == "decode":
        o, S = _delta(s, s["pool"][at], rows, F32)
        s["pool"][at] = S
        xq, xs = _encode_act(_tail(o, s["z"][rows].float(), s["w"]))
        s["xq"].view(torch.uint8)[rows] = xq.view(torch.uint8)
        s["xs"][rows] = xs
        return s["xq"], s["xs"], s["pool"]
    window = torch.cat([s["pool"][at], s["x"][rows][:, None]], 1)
    y = (window.float() * s["w"].t()).sum(1)
    s["y"][rows] = (y * torch.sigmoid(y)).to(BF16)
    s["pool"][at] = window[:, 1:]
    return s["y"], s["pool"]


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // 128)) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    if op == "encode":
        M, K = case["M"], case["K"]
        scales = -(-K // 128) * (M if case["what"] == "act" else -(-M // 128))
        return {"bytes": M * K * ((2 if case["io"] == "bf16" else 4) + 1) + 4 * scales, "flops": 3 * M * K}
    if op == "tail":
        n = case["M"] * case["Hv"] * case["D"]
        return {"bytes": n * (2 * (2 if case["io"] == "bf16" else 4) + 1) + 4 * case["M"] * -(-case["Hv"] * case["D"] // 128), "flops": 12 * n}
    live = case["B"] - case["dead"]
    if op == "decode":
        Hk, Hv = case["Hk"], case["Hv"]
        row = 2 * Hk * 256 + Hv * (256 + 256 + 128 + 4) + 2 * Hv * (2 if case["packed"] else 4)
        return {"bytes": live * (2 * Hv * 65536 + row), "flops": live * Hv * 8 * 16384}
    C, K = case["C"], case["K"]
    return {"bytes": live * C * 2 * (2 + 2 * (K - 1)) + C * K * 4, "flops": live * C * (2 * K + 4)}


def _exact_blocks(x, rows):
    """Values over their block scale (unrounded), and the scales, of blocks of `rows` x 128."""
    M, K = x.shape
    p = x.new_zeros(-(-M // rows) * rows, -(-K // 128) * 128)
    p[:M, :K] = x
    blocks = p.reshape(p.shape[0] // rows, rows, p.shape[1] // 128, 128).permute(0, 2, 1, 3)
    scale = torch.maximum(blocks.abs().flatten(2).max(2).values / 448.0, torch.tensor(TINY, dtype=F64, device=x.device))
    q = (blocks / scale[..., None, None]).permute(0, 2, 1, 3).reshape(p.shape)
    return q[:M, :K], scale


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = torch.arange(K, device="cuda") // 128
        a = s["aq"].to(F64) * s["as"].to(F64)[:, kb]
        b = s["bq"].to(F64) * s["bs"].to(F64)[torch.arange(N, device="cuda") // 128][:, kb]
        return torch.einsum("mk,nk->mn", a, b)
    if op == "encode":
        return _exact_blocks(s["x"].to(F64), 1 if case["what"] == "act" else 128)
    if op == "tail":
        o, z = s["o"].to(F64), s["z"].to(F64)
        y = o / torch.sqrt((o * o).sum(2, keepdim=True) / case["D"] + EPS) * s["w"].to(F64) * z / (1 + torch.exp(-z))
        return _exact_blocks(y.reshape(case["M"], -1), 1)
    live = [(i, t) for i, t in enumerate(s["slots"].tolist()) if t >= 0]
    rows, at = (torch.tensor([p[j] for p in live], device="cuda", dtype=torch.long) for j in (0, 1))
    if op == "decode":
        Hv = case["Hv"]
        head = torch.arange(Hv, device="cuda") // (Hv // case["Hk"])
        pool = s["pool"].to(F64)
        q, k = (s[n][rows].to(F64)[:, head] for n in ("q", "k"))
        v, z, b = (s[n][rows].to(F64) for n in ("v", "z", "b"))
        q = q / torch.sqrt((q * q).sum(2, keepdim=True) + EPS)
        k = k / torch.sqrt((k * k).sum(2, keepdim=True) + EPS)
        g = -torch.exp(s["A_log"].to(F64)) * torch.log1p(torch.exp(s["a"][rows].to(F64) + s["dt_bias"].to(F64)))
        alpha, beta = torch.exp(g), 1 / (1 + torch.exp(-b))
        S = pool[at]
        write = torch.einsum("bhij,bhj->bhi", S, k) * alpha[..., None]
        S = alpha[..., None, None] * S + torch.einsum("bhi,bhj->bhij", beta[..., None] * (v - write), k)
        pool[at] = S
        o = torch.einsum("bhij,bhj->bhi", S, q)
        y = o / torch.sqrt((o * o).sum(2, keepdim=True) / 128 + EPS) * s["w"].to(F64) * z / (1 + torch.exp(-z))
        codes, scales = _exact_blocks(y.reshape(len(live), -1), 1)
        xq, xs = torch.zeros(case["B"], Hv * 128, dtype=F64, device="cuda"), torch.zeros(case["B"], Hv, dtype=F64, device="cuda")
        xq[rows], xs[rows] = codes, scales
        return xq, xs, pool
    K = case["K"]
    pool, x, w = s["pool"].to(F64), s["x"][rows].to(F64), s["w"].to(F64)
    old = pool[at]
    pre = x * w[:, K - 1] + sum(old[:, j] * w[:, j] for j in range(K - 1))
    y = torch.zeros(case["B"], case["C"], dtype=F64, device="cuda")
    y[rows] = pre / (1 + torch.exp(-pre))
    pool[at] = torch.stack([old[:, j + 1] if j + 1 < K - 1 else x for j in range(K - 1)], 1)
    return y, pool
