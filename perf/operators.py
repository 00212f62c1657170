"""The layer norm and 8-bit product operators: their cases, plain forms and definitions in 64 bits.

`listed()` and `draw()` give cases, `prepare()` what a program holds before a call, `run()`
one pass through an operator (the plain form, or the library's kernels where `own` is true),
`work()` the bytes and operations that pass cannot do without, and `exact()` its results
computed in 64 bits.

Operators (`case["op"]`):
  ln_fwd      y = LN(x) with the row statistics the backward pass needs
  ln_bwd      dx, dgamma, dbeta of a layer norm on a residual branch (dx includes the
              residual stream's own gradient)
  linear      y = act(x W^T + b) with the weights held in 8 bits and x quantised in the call
  linear_step forward and backward of a linear layer in a training step: both operands of
              each of the three products quantised in the call, in the direction it reduces
  mlp         y = x + MLP(LN(x)) with both products in 8 bits

8-bit values are e4m3 with one power-of-two scale per 128 consecutive values along the
reduction: scale 2^e, e the least integer (at least -127) with max |x| <= 448 * 2^e.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the final norm of 16 CLS rows (a batch of UMT-L clips): latency only
        {"name": "ln_fwd_cls16", "op": "ln_fwd", "M": 16, "C": 1024, "dtype": "bf16"},
        # UMT-L, first stage: 16 clips of 1569 tokens
        {"name": "ln_fwd_umt_l", "op": "ln_fwd", "M": 25104, "C": 1024, "dtype": "bf16"},
        # DeiT-T, two images, trained in fp32: the smallest gradient
        {"name": "ln_bwd_tiny", "op": "ln_bwd", "M": 394, "C": 192, "dtype": "fp32"},
        # rows left by pruning (an odd count) of an odd width in fp16: no 16-byte rows
        {"name": "ln_bwd_odd", "op": "ln_bwd", "M": 8577, "C": 1001, "dtype": "fp16"},
        # DeiT-B, 256 images: the largest gradient
        {"name": "ln_bwd_deit_b", "op": "ln_bwd", "M": 50432, "C": 768, "dtype": "bf16"},
        # one token through UMT-L's fc1 (serving one row: latency, weights streamed once)
        {"name": "linear_1", "op": "linear", "M": 1, "K": 1024, "N": 4096, "gelu": True},
        # 16 rows through the widest weights the library takes
        {"name": "linear_16_wide", "op": "linear", "M": 16, "K": 2048, "N": 8192, "gelu": False},
        # DeiT-S fc1, 256 images
        {"name": "linear_deit_s", "op": "linear", "M": 50432, "K": 384, "N": 1536, "gelu": True},
        # a small ragged training step: rows, width and outputs that end inside a block
        {"name": "step_ragged", "op": "linear_step", "M": 395, "K": 200, "N": 776},
        # UMT-L fc1 after the second pruning: 16 clips of 768 tokens, a training step
        {"name": "step_umt_l", "op": "linear_step", "M": 12288, "K": 1024, "N": 4096},
        # DeiT-T, two images: the whole sublayer at its smallest
        {"name": "mlp_tiny", "op": "mlp", "M": 394, "C": 192, "H": 768},
        # UMT-L, first stage: the largest
        {"name": "mlp_umt_l", "op": "mlp", "M": 25104, "C": 1024, "H": 4096},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "linear", "linear_step", "mlp"])
    if op in ("ln_fwd", "ln_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        C = _log_int(rng, 48, 4096)
        if rng.random() < 0.7:
            C = max(8, C // 8 * 8)
        top = 38_000_000 // (2 if dtype == "fp32" else 1) // C
        return {"op": op, "M": _log_int(rng, 1, min(60000, top)), "C": C, "dtype": dtype}
    if op in ("linear", "linear_step"):
        K, N = _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
        if op == "linear":
            top = min(50000, 30_000_000_000 // (K * N))
            return {"op": op, "M": _log_int(rng, 1, top), "K": K, "N": N,
                    "gelu": rng.random() < 0.5}
        top = min(30000, 50_000_000_000 // (K * N))
        return {"op": op, "M": _log_int(rng, 2, top), "K": K, "N": N}
    C = 64 * rng.randint(1, 16)
    H = 64 * rng.randint(1, 64)
    top = min(50000, 100_000_000_000 // (C * H))
    return {"op": op, "M": _log_int(rng, 1, top), "C": C, "H": H}


# ------------------------------------------------------------------ inputs
def _rows(g, M, C, dtype, dev):
    """Token rows as the residual stream holds them: a fifth of the rows three times as
    large (foreground), a few columns far larger than the rest."""
    x = torch.randn(M, C, generator=g, device=dev)
    x *= torch.where(torch.rand(M, 1, generator=g, device=dev) < 0.2, 3.0, 1.0)
    x *= torch.where(torch.rand(1, C, generator=g, device=dev) < 0.01, 12.0, 1.0)
    return (x + 0.1).to(dtype)


def _weight(g, N, K, dev):
    return (torch.randn(N, K, generator=g, device=dev) * 0.02).clamp_(-0.04, 0.04).bfloat16()


def _bias(g, n, std, dev):
    return (torch.randn(n, generator=g, device=dev) * std).bfloat16()


def _stored(w):
    """A weight [N, K] as a checkpoint in 8 bits keeps it: the values, each row padded to a
    multiple of 16 bytes, and the scale bytes (e + 127) in tiles of 128 rows x 4 blocks, the
    byte of row r and block j at 16 (r % 32) + 4 (r / 32 % 4) + j % 4 of its tile."""
    N, K = w.shape
    KB, KQ, NT = -(-K // 128), -(-K // 512), -(-N // 128)
    p = torch.zeros(N, KB * 128, device=w.device)
    p[:, :K] = w.float()
    p = p.view(N, KB, 128)
    m, k = torch.frexp(p.abs().amax(-1))
    e = torch.where(m > 0, k - 9 + (m > 0.875), -127).clamp_(min=-127)
    q = torch.ldexp(p, -e[..., None].float()).view(N, KB * 128)
    q = q[:, : -(-K // 16) * 16].to(torch.float8_e4m3fn).contiguous()
    s = torch.zeros(NT * 128, KQ * 4, dtype=torch.uint8, device=w.device)
    s[:N, :KB] = (e + 127).to(torch.uint8)
    s = s.view(NT, 4, 32, KQ, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op, M = case["op"], case["M"]
    s = {"op": op}
    if op in ("ln_fwd", "ln_bwd"):
        C, dt = case["C"], DTYPES[case["dtype"]]
        s["x"] = _rows(g, M, C, dt, dev)
        s["gamma"] = (1.0 + 0.05 * torch.randn(C, generator=g, device=dev)).to(dt)
        s["beta"] = (0.02 * torch.randn(C, generator=g, device=dev)).to(dt)
        if op == "ln_bwd":
            x = s["x"].double()
            mean = x.mean(1, keepdim=True)
            rstd = 1.0 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
            s["stats"] = torch.cat([mean, rstd], 1).float()
            s["dy"] = (torch.randn(M, C, generator=g, device=dev) * 0.1).to(dt)
            s["dres"] = (torch.randn(M, C, generator=g, device=dev) * 0.1).to(dt)
    elif op == "linear":
        K, N = case["K"], case["N"]
        s["x"] = _rows(g, M, K, torch.bfloat16, dev)
        s["wq"], s["ws"] = _stored(_weight(g, N, K, dev))
        s["b"] = _bias(g, N, 0.01, dev)
        s["N"], s["gelu"] = N, case["gelu"]
    elif op == "linear_step":
        K, N = case["K"], case["N"]
        s["x"] = _rows(g, M, K, torch.bfloat16, dev)
        s["w"] = _weight(g, N, K, dev)
        s["b"] = _bias(g, N, 0.01, dev)
        s["dy"] = (torch.randn(M, N, generator=g, device=dev) * 1e-3).bfloat16()
    else:
        C, H = case["C"], case["H"]
        s["x"] = _rows(g, M, C, torch.bfloat16, dev)
        s["w1q"], s["w1s"] = _stored(_weight(g, H, C, dev))
        s["w2q"], s["w2s"] = _stored(_weight(g, C, H, dev))
        s["b1"], s["b2"] = _bias(g, H, 0.01, dev), _bias(g, C, 0.01, dev)
        s["gamma"] = (1.0 + 0.05 * torch.randn(C, generator=g, device=dev)).bfloat16()
        s["beta"] = (0.02 * torch.randn(C, generator=g, device=dev)).bfloat16()
        s["C"], s["H"] = C, H
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _norm(x):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    return (x - mean) * rstd, mean, rstd


def _q(x):
    """The values [R, K] takes in 8 bits, blocks of 128 along the last axis."""
    R, K = x.shape
    KB = -(-K // 128)
    p = torch.zeros(R, KB * 128, device=x.device)
    p[:, :K] = x
    p = p.view(R, KB, 128)
    m, k = torch.frexp(p.abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, k - 9 + (m > 0.875), -127).clamp(min=-127).float()
    v = torch.ldexp(p, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(v, e).view(R, KB * 128)[:, :K]


def _unstored(q, s, N, K):
    KB, KQ, NT = -(-K // 128), -(-K // 512), -(-N // 128)
    e = s.view(NT, KQ, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(NT * 128, KQ * 4)[:N, :KB]
    e = (e.float() - 127.0).repeat_interleave(128, 1)[:, :K]
    return torch.ldexp(q.float()[:, :K], e)


def _gelu(z):
    return 0.5 * z * (1.0 + torch.erf(z * (1.0 / math.sqrt(2.0))))


def _run_plain(s):
    op = s["op"]
    if op == "ln_fwd":
        xh, mean, rstd = _norm(s["x"])
        y = xh * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["x"].dtype), "stats": torch.cat([mean, rstd], 1)}
    if op == "ln_bwd":
        mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
        xh = (s["x"].float() - mean) * rstd
        dy = s["dy"].float()
        w = dy * s["gamma"].float()
        dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
        dx = dx + s["dres"].float()
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    if op == "linear":
        w = _unstored(s["wq"], s["ws"], s["N"], s["x"].shape[1])
        z = _q(s["x"].float()) @ w.T + s["b"].float()
        return (_gelu(z) if s["gelu"] else z).bfloat16()
    if op == "linear_step":
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        y = _q(x) @ _q(w).T + s["b"].float()
        dx = _q(dy) @ _q(w.T).T
        dw = _q(dy.T) @ _q(x.T).T
        return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw.bfloat16(), "db": dy.sum(0)}
    x = s["x"].float()
    w1 = _unstored(s["w1q"], s["w1s"], s["H"], s["C"])
    w2 = _unstored(s["w2q"], s["w2s"], s["C"], s["H"])
    u = _norm(s["x"])[0] * s["gamma"].float() + s["beta"].float()
    a = _gelu(_q(u) @ w1.T + s["b1"].float())
    return (x + (_q(a) @ w2.T + s["b2"].float())).bfloat16()


def _run_own(s):
    import free_vit_token_b200 as rs

    op = s["op"]
    if op == "ln_fwd":
        y, stats = rs.rs_ln_forward(s["x"], s["gamma"], s["beta"], eps=EPS)
        return {"y": y, "stats": stats}
    if op == "ln_bwd":
        dx, dg, db = rs.rs_ln_backward(s["dy"], s["x"], s["stats"], s["gamma"], dres=s["dres"])
        return {"dx": dx, "dgamma": dg, "dbeta": db}
    if op == "linear":
        w = rs.Fp8(s["wq"], s["ws"], s["N"], s["x"].shape[1])
        return rs.rs_fp8_linear(s["x"], w, bias=s["b"], gelu=s["gelu"])
    if op == "linear_step":
        wq, wtq, _ = rs.rs_fp8_quantize(s["w"], rows=True, cols=True)
        xq, xtq, _ = rs.rs_fp8_quantize(s["x"], rows=True, cols=True)
        y = rs.rs_fp8_gemm(xq, wq, bias=s["b"])
        dx, dw, db = rs.rs_fp8_linear_backward(s["dy"], xtq, wtq, bias=True)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    w1 = rs.Fp8(s["w1q"], s["w1s"], s["H"], s["C"])
    w2 = rs.Fp8(s["w2q"], s["w2s"], s["C"], s["H"])
    return rs.rs_mlp_forward_fp8(s["x"], w1, s["b1"], w2, s["b2"], s["gamma"], s["beta"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, M = case["op"], case["M"]
    if op in ("ln_fwd", "ln_bwd"):
        C, e = case["C"], 4 if case["dtype"] == "fp32" else 2
        if op == "ln_fwd":
            return {"bytes": 2 * e * M * C + 2 * e * C + 8 * M, "flops": 8 * M * C}
        return {"bytes": 4 * e * M * C + e * C + 8 * C + 8 * M, "flops": 14 * M * C}
    if op == "mlp":
        C, H = case["C"], case["H"]
        weights = 2 * C * H + 2 * C * H // 128
        return {"bytes": 4 * M * C + weights + 2 * H + 6 * C, "flops": 4 * M * C * H}
    K, N = case["K"], case["N"]
    if op == "linear":
        return {"bytes": 2 * M * K + N * K + N * K // 128 + 2 * N + 2 * M * N,
                "flops": 2 * M * N * K}
    return {"bytes": 2 * (M * K + N * K + M * N + N) + 2 * (M * N + M * K + N * K) + 4 * N,
            "flops": 6 * M * N * K}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_64(v):
    """Nearest e4m3 value, ties to the even mantissa, of |v| <= 448."""
    lo = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    lo = torch.where(torch.exp2(lo) > v.abs().clamp(min=2.0 ** -6), lo - 1, lo)
    lo = torch.where(torch.exp2(lo + 1) <= v.abs(), lo + 1, lo)
    step = torch.exp2(lo - 3)
    return torch.round(v / step) * step


def _q64(x):
    """Each 128 consecutive values of a row rounded to e4m3 at their own power of two."""
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], 128):
        c = x[:, j:j + 128]
        top = c.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448.0))
        e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
        e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)
        f = torch.exp2(e.clamp(min=-127))
        out[:, j:j + 128] = _e4m3_64(c / f) * f
    return out


def _weights_64(q, s, N, K):
    r = torch.arange(N, device=q.device)[:, None]
    j = torch.arange(K, device=q.device)[None, :] // 128
    at = (r // 128 * (-(-K // 512)) + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4
    return q[:, :K].double() * torch.exp2(s[at].double() - 127.0)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.dtype in
         (torch.bfloat16, torch.float16, torch.float32)}
    op = s["op"]

    def layer_norm():
        c = d["x"] - d["x"].sum(1, keepdim=True) / d["x"].shape[1]
        r = ((c * c).sum(1, keepdim=True) / c.shape[1] + EPS).rsqrt()
        return c * r * d["gamma"] + d["beta"], r

    def cdf(z):
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))

    if op == "ln_fwd":
        y, r = layer_norm()
        return {"y": y, "stats": torch.stack([d["x"].mean(1), r[:, 0]], 1)}
    if op == "ln_bwd":
        mu, r = d["stats"].split(1, 1)
        xh = (d["x"] - mu) * r
        w = d["dy"] * d["gamma"]
        C = w.shape[1]
        dx = w * r - r / C * (w.sum(1, keepdim=True) + xh * (w * xh).sum(1, keepdim=True))
        return {"dx": dx + d["dres"], "dgamma": torch.einsum("rc,rc->c", d["dy"], xh),
                "dbeta": d["dy"].sum(0)}
    if op == "linear":
        z = torch.addmm(d["b"], _q64(d["x"]), _weights_64(s["wq"], s["ws"], s["N"],
                                                          case["K"]).T)
        return z * cdf(z) if s["gelu"] else z
    if op == "linear_step":
        qt = lambda t: _q64(t.T.contiguous())  # noqa: E731
        return {"y": torch.addmm(d["b"], _q64(d["x"]), _q64(d["w"]).T),
                "dx": _q64(d["dy"]) @ qt(d["w"]).T, "dw": qt(d["dy"]) @ qt(d["x"]).T,
                "db": d["dy"].sum(0)}
    u, _ = layer_norm()
    z = torch.addmm(d["b1"], _q64(u), _weights_64(s["w1q"], s["w1s"], s["H"], s["C"]).T)
    del u
    h = torch.addmm(d["b2"], _q64(z * cdf(z)), _weights_64(s["w2q"], s["w2s"], s["C"], s["H"]).T)
    return d["x"] + h
