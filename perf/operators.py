"""The training operators of the BitLinear library, as cases to measure.

Five kinds of pass:

  step         a BitLinear training step that keeps its activations as 8-bit
               codes: (norm,) quantise, ternary matmul, rescale, and from the
               codes and the output's gradient the gradients of the input and
               of the latent weights
  grad_input   dX = gamma * dY C, C the ternary matrix in its packed storage
  grad_weight  dW (+)= dY^T X^, X^ = q / s from the 8-bit codes of the forward
  norm_fwd     LayerNorm / RMSNorm of bf16 rows, with its statistics
  norm_bwd     its gradients: of the rows, of the weight and of the bias

The quantisers' rounding and clamping are passed straight through, scales are
constants, so with the forward Y = (q C^T) * (gamma / s):
  dX = gamma * dY C          dW = dY^T (q / s)
and behind a norm (no affine parameters) with xh = q / s read from the codes:
  r = sqrt(stat + eps)   dx = (g - mean(g) - xh mean(g xh)) / r   (LayerNorm; RMSNorm has no mean(g))
"""

import math

import torch

own = False

EPS = 1e-5
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's LayerNorm before the output head: all latency
        {"name": "norm_fwd_one_token", "op": "norm_fwd", "norm": "layer", "affine": True, "M": 1, "K": 2560},
        # the RMSNorm of a 2B-class hidden state, 4096 tokens
        {"name": "norm_fwd_2b", "op": "norm_fwd", "norm": "rms", "affine": True, "M": 4096, "K": 2560},
        # the backward of a 2B-class block's LayerNorm: 4096 rows to reduce for the weight and bias
        {"name": "norm_bwd_2b", "op": "norm_bwd", "norm": "layer", "affine": True, "M": 4096, "K": 2560},
        # few long rows: a 70B-class width, an odd number of tokens
        {"name": "norm_bwd_70b_m257", "op": "norm_bwd", "norm": "rms", "affine": True, "M": 257, "K": 8192},
        # the down projection of the 2B-class feed-forward block
        {"name": "grad_input_2b_down", "op": "grad_input", "M": 4096, "K": 6912, "N": 2560},
        # a 70B-class layer with few tokens: few output tiles, a long sum
        {"name": "grad_input_70b_m128", "op": "grad_input", "M": 128, "K": 8192, "N": 28672},
        # the up projection of the 2B-class block: fp32 gradient of the latent weights
        {"name": "grad_weight_2b_up", "op": "grad_weight", "M": 4096, "K": 2560, "N": 6912, "bits": 8,
         "out": "fp32", "accumulate": False},
        # the 4-bit-activation layer, gradient in bf16
        {"name": "grad_weight_a48_bf16", "op": "grad_weight", "M": 2048, "K": 4096, "N": 11008, "bits": 4,
         "out": "bf16", "accumulate": False},
        # a ragged micro-batch added to what earlier ones left (rows of dY that are not 16-byte aligned)
        {"name": "grad_weight_ragged_acc", "op": "grad_weight", "M": 257, "K": 1344, "N": 1003, "bits": 8,
         "out": "fp32", "accumulate": True},
        # the smallest whole step: launches and hand-overs count
        {"name": "step_tiny", "op": "step", "norm": "layer", "M": 16, "K": 256, "N": 512, "bits": 8},
        # the up projection of the 2B-class block behind its SubLN, 4096 tokens
        {"name": "step_2b_up", "op": "step", "norm": "rms", "M": 4096, "K": 2560, "N": 6912, "bits": 8},
        # the largest: a 70B-class layer, 2048 tokens
        {"name": "step_70b", "op": "step", "norm": "none", "M": 2048, "K": 8192, "N": 28672, "bits": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "grad_input", "grad_weight", "norm_fwd", "norm_bwd"])
    case = {"op": op, "M": _log_int(rng, 1, 8192), "K": 64 * _log_int(rng, 1, 256)}
    if op in ("norm_fwd", "norm_bwd"):
        case.update(norm=rng.choice(["layer", "rms"]), affine=rng.random() < 0.75)
        return case
    case["N"] = _log_int(rng, 64, 16384)
    while case["M"] * case["K"] * case["N"] > 2048 * 8192 * 28672:
        case["M"] = (case["M"] + 1) // 2
    if op != "grad_input":
        case["bits"] = rng.choice([8, 8, 4])
    if op == "grad_weight":
        case.update(out=rng.choice(["fp32", "bf16"]), accumulate=rng.random() < 0.5)
    if op == "step":
        case["norm"] = rng.choice(["none", "rms", "layer"])
    return case


def work(case):
    M, K, N, op = case["M"], case["K"], case.get("N", 0), case["op"]
    if op == "norm_fwd":
        par = (4 if case["norm"] == "layer" else 2) * K if case["affine"] else 0
        stats = (8 if case["norm"] == "layer" else 4) * M
        return {"bytes": 4 * M * K + par + stats, "flops": 8 * M * K}
    if op == "norm_bwd":
        par = ((2 + 8) if case["norm"] == "layer" else (2 + 4)) * K if case["affine"] else 0
        stats = (8 if case["norm"] == "layer" else 4) * M
        return {"bytes": 6 * M * K + par + stats, "flops": 14 * M * K}
    if op == "grad_input":
        return {"bytes": 2 * M * N + N * K // 4 + 2 * M * K + 4, "flops": 2 * M * N * K}
    if op == "grad_weight":
        dw = (4 if case["out"] == "fp32" else 2) * N * K
        return {"bytes": 2 * M * N + M * K + 4 * M + (2 if case["accumulate"] else 1) * dw, "flops": 2 * M * N * K}
    return {"bytes": 4 * M * N + 4 * M * K + N * K // 4 + 4 * N * K + 4, "flops": 6 * M * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(M, K, g):
    """Hidden states: Gaussian with one channel in a hundred ten times larger."""
    x = torch.randn(M, K, generator=g, device=DEVICE)
    ch = torch.randperm(K, generator=g, device=DEVICE)[: max(1, K // 100)]
    x[:, ch] *= 10.0
    return x.to(torch.bfloat16)


def _grads(M, N, g):
    """Gradients: small, and of very different size from token to token."""
    scale = 1e-3 * torch.exp(torch.randn(M, 1, generator=g, device=DEVICE))
    return (torch.randn(M, N, generator=g, device=DEVICE) * scale).to(torch.bfloat16)


def _packed(N, K, g):
    """Ternary codes in the library's 2-bit storage: byte b of the 32-bit word
    of weights 16w..16w+15 holds weights 16w + 4j + b (j = 0..3) as code + 1 in
    bits 2j, 2j+1.  31% zeros, as Gaussian weights give."""
    p = torch.zeros(N, K // 4, dtype=torch.uint8, device=DEVICE)
    for j in range(4):
        u = torch.rand(N, K // 4, generator=g, device=DEVICE)
        p += ((u > 0.345).to(torch.uint8) + (u > 0.655).to(torch.uint8)) << (2 * j)
    return p


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    M, K, op = case["M"], case["K"], case["op"]
    st = {"case": dict(case)}
    if op in ("norm_fwd", "norm_bwd"):
        st["X"] = _rows(M, K, g) + 0.25
        st["weight"] = st["bias"] = None
        if case["affine"]:
            st["weight"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=DEVICE)).to(torch.bfloat16)
            if case["norm"] == "layer":
                st["bias"] = (0.1 * torch.randn(K, generator=g, device=DEVICE)).to(torch.bfloat16)
        if op == "norm_bwd":
            st["dY"] = _grads(M, K, g)
            x = st["X"].double()
            st["mean"] = x.mean(1).float() if case["norm"] == "layer" else None
            stat = x.var(1, unbiased=False) if case["norm"] == "layer" else x.square().mean(1)
            st["stat"] = stat.float()
        return st
    N = case["N"]
    st["dY"] = _grads(M, N, g)
    if op in ("step", "grad_input"):
        st["Wp"] = _packed(N, K, g)
        st["gamma"] = (0.01 + 0.01 * torch.rand(1, generator=g, device=DEVICE)).float()
    if op == "step":
        st["X"] = _rows(M, K, g)
    if op == "grad_weight":
        # what the forward kept: codes and scales of its input
        st["Xq"], st["scale"] = _codes(_rows(M, K, g), case["bits"])
        if case["accumulate"]:
            st["dW"] = 1e-2 * torch.randn(N, K, generator=g, device=DEVICE)
            if case["out"] == "bf16":
                st["dW"] = st["dW"].to(torch.bfloat16)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _codes(x, bits):
    """Per token s = Q / max(max|x|, 1e-5) in fp32, q = round_half_even(fp32(x s))."""
    x = x.float()
    a = x.abs().amax(1).clamp_min(1e-5)
    s = torch.full_like(a, 127.0 if bits == 8 else 7.0) / a   # a division: number / tensor takes a reciprocal
    return torch.round(x * s[:, None]).to(torch.int8), s


def _ternary(Wp, K):
    """[N, K] fp32 codes of the packed storage."""
    sh = torch.arange(0, 8, 2, device=Wp.device, dtype=torch.uint8).view(1, 1, 4, 1)
    w = Wp.view(-1, K // 16, 1, 4)
    return (((w >> sh) & 3).to(torch.float32) - 1.0).reshape(-1, K)


def _norm_stats(x, norm):
    """Mean and biased variance (or mean of squares) of each row: formed in 64
    bits, since they decide codes, and rounded once."""
    x = x.double()
    if norm == "layer":
        mu = x.mean(1)
        return mu.float(), (x - mu[:, None]).square().mean(1).float()
    return None, x.square().mean(1).float()


def _normed(x, norm):
    """The norm ahead of the quantiser, with the roundings its definition names."""
    mu, stat = _norm_stats(x, norm)
    r = torch.sqrt(stat + EPS)
    x = x.float() - (mu[:, None] if mu is not None else 0.0)
    return (x / r[:, None]).to(torch.bfloat16), stat


def _norm_dx(g, xh, stat, norm):
    r = torch.sqrt(stat + EPS)[:, None]
    c = (g * xh).mean(1, keepdim=True)
    d = g - xh * c
    if norm == "layer":
        d = d - g.mean(1, keepdim=True)
    return d / r


def _plain_step(st):
    c = st["case"]
    K, norm = c["K"], c["norm"]
    x, stat = st["X"], None
    if norm != "none":
        x, stat = _normed(x, norm)
    q, s = _codes(x, c["bits"])
    t = _ternary(st["Wp"], K)
    qf = q.float()
    Y = ((qf @ t.t()) * (st["gamma"] / s)[:, None]).to(torch.bfloat16)   # the sum is a whole number below 2^24
    dy = st["dY"].float()
    xh = qf / s[:, None]
    dX = (dy @ t) * st["gamma"]
    dW = dy.t() @ xh
    if norm != "none":
        dX = _norm_dx(dX, xh, stat, norm)
    return {"Y": Y, "dX": dX.to(torch.bfloat16), "dW": dW}


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "step":
        return _plain_step(st)
    if op == "grad_input":
        return {"dX": ((st["dY"].float() @ _ternary(st["Wp"], c["K"])) * st["gamma"]).to(torch.bfloat16)}
    if op == "grad_weight":
        dW = st["dY"].float().t() @ (st["Xq"].float() / st["scale"][:, None])
        if c["accumulate"]:
            st["dW"].copy_(st["dW"].float() + dW)
            return {"dW": st["dW"]}
        return {"dW": dW if c["out"] == "fp32" else dW.to(torch.bfloat16)}
    x = st["X"].float()
    w = st["weight"].float() if st["weight"] is not None else None
    if op == "norm_fwd":
        if c["norm"] == "layer":
            mu = x.mean(1)
            xc = x - mu[:, None]
            stat = xc.square().mean(1)
        else:
            mu, xc, stat = None, x, x.square().mean(1)
        y = xc / torch.sqrt(stat + EPS)[:, None]
        if w is not None:
            y = y * w
        if st["bias"] is not None:
            y = y + st["bias"].float()
        out = {"Y": y.to(torch.bfloat16), "stat": stat}
        if mu is not None:
            out["mean"] = mu
        return out
    dy = st["dY"].float()
    xc = x - st["mean"][:, None] if st["mean"] is not None else x
    xh = xc / torch.sqrt(st["stat"] + EPS)[:, None]
    out = {"dX": _norm_dx(dy * w if w is not None else dy, xh, st["stat"], c["norm"]).to(torch.bfloat16)}
    if w is not None:
        out["dweight"] = (dy * xh).sum(0)
        if c["norm"] == "layer":
            out["dbias"] = dy.sum(0)
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _library(st):
    from bitlinear_bl_forward_b200 import bl

    c = st["case"]
    op = c["op"]
    norm = {"rms": bl.BL_NORM_RMS, "layer": bl.BL_NORM_LAYER}.get(c.get("norm"))
    if op == "step":
        Y, Xq, scale, stat = bl.bl_forward_checkpoint(st["X"], st["Wp"], st["gamma"], c["N"], c["bits"],
                                                      norm=norm, eps=EPS)
        dX = bl.bl_backward_input(st["dY"], st["Wp"], st["gamma"], c["K"])
        dW = bl.bl_backward_weight(st["dY"], Xq, scale)
        if norm is not None:
            dX = bl.bl_norm_backward_checkpoint(dX, Xq, scale, norm, stat, eps=EPS)
        return {"Y": Y, "dX": dX, "dW": dW}
    if op == "grad_input":
        return {"dX": bl.bl_backward_input(st["dY"], st["Wp"], st["gamma"], c["K"])}
    if op == "grad_weight":
        if c["accumulate"]:
            return {"dW": bl.bl_backward_weight(st["dY"], st["Xq"], st["scale"], out=st["dW"], accumulate=True)}
        dtype = torch.float32 if c["out"] == "fp32" else torch.bfloat16
        return {"dW": bl.bl_backward_weight(st["dY"], st["Xq"], st["scale"], dtype=dtype)}
    if op == "norm_fwd":
        Y, mean, stat = bl.bl_norm_forward(st["X"], norm, weight=st["weight"], bias=st["bias"], eps=EPS)
        out = {"Y": Y, "stat": stat}
        if mean is not None:
            out["mean"] = mean
        return out
    dX, dweight, dbias = bl.bl_norm_backward(st["dY"], st["X"], norm, st["stat"], mean=st["mean"],
                                             weight=st["weight"], need_bias=st["bias"] is not None, eps=EPS)
    out = {"dX": dX}
    if dweight is not None:
        out["dweight"] = dweight
    if dbias is not None:
        out["dbias"] = dbias
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_codes(x64, bits):
    """The codes are defined through fp32 roundings of exact 64-bit products and quotients."""
    Q = torch.tensor(127.0 if bits == 8 else 7.0, dtype=torch.float64, device=x64.device)
    floor = torch.tensor(1e-5, dtype=torch.float32).double().item()
    s = torch.true_divide(Q, torch.clamp(torch.max(torch.abs(x64), dim=1).values, min=floor)).float().double()
    return torch.round((x64 * s.unsqueeze(1)).float().double()), s


def _exact_weights(Wp, K):
    """Codes by looking every byte up: 256 bytes, four fields each."""
    table = torch.tensor([[float((b >> (2 * j)) & 3) - 1.0 for j in range(4)] for b in range(256)],
                         dtype=torch.float64, device=Wp.device)
    N = Wp.shape[0]
    return table[Wp.long()].view(N, K // 16, 4, 4).transpose(2, 3).reshape(N, K)


def _exact_norm_dx(g, xh, stat, norm):
    K = g.shape[1]
    out = g - xh * (torch.einsum("mk,mk->m", g, xh) / K).unsqueeze(1)
    if norm == "layer":
        out -= (g.sum(dim=1) / K).unsqueeze(1)
    return out * (stat.double() + EPS).rsqrt().unsqueeze(1)


def exact(case, seed):
    st = prepare(case, seed)
    op, K, norm = case["op"], case["K"], case.get("norm")
    f64 = torch.float64
    if op == "step":
        x = st["X"].to(f64)
        var = None
        if norm != "none":
            mu = x.sum(dim=1) / K if norm == "layer" else torch.zeros_like(x[:, 0])
            var = (torch.einsum("mk,mk->m", x - mu.unsqueeze(1), x - mu.unsqueeze(1)) / K).float()
            r = torch.sqrt((var + torch.tensor(EPS, dtype=torch.float32, device=var.device)).double()).float()
            diff = (x - mu.float().double().unsqueeze(1)).float().double()
            x = (diff / r.double().unsqueeze(1)).float().to(torch.bfloat16).to(f64)
        q, s = _exact_codes(x, case["bits"])
        W = _exact_weights(st["Wp"], K) * st["gamma"].to(f64)
        xh = q / s.unsqueeze(1)
        dy = st["dY"].to(f64)
        Y = xh @ W.T
        dX = dy @ W
        if norm != "none":
            dX = _exact_norm_dx(dX, xh, var, norm)
        del W
        return {"Y": Y, "dX": dX, "dW": dy.T @ xh}
    dy = st["dY"].to(f64) if "dY" in st else None
    if op == "grad_input":
        return {"dX": dy @ (_exact_weights(st["Wp"], K) * st["gamma"].to(f64))}
    if op == "grad_weight":
        dW = dy.T @ (st["Xq"].to(f64) / st["scale"].to(f64).unsqueeze(1))
        return {"dW": dW + st["dW"].to(f64) if case["accumulate"] else dW}
    x = st["X"].to(f64)
    w = st["weight"].to(f64) if case["affine"] else 1.0
    if op == "norm_fwd":
        mu = x.sum(dim=1) / K if norm == "layer" else None
        d = x - mu.unsqueeze(1) if norm == "layer" else x
        stat = torch.einsum("mk,mk->m", d, d) / K
        y = d * (stat + EPS).rsqrt().unsqueeze(1) * w
        if st["bias"] is not None:
            y = y + st["bias"].to(f64)
        out = {"Y": y, "stat": stat}
        if norm == "layer":
            out["mean"] = mu
        return out
    d = x - st["mean"].to(f64).unsqueeze(1) if norm == "layer" else x
    xh = d * (st["stat"].to(f64) + EPS).rsqrt().unsqueeze(1)
    out = {"dX": _exact_norm_dx(dy * w, xh, st["stat"], norm)}
    if case["affine"]:
        out["dweight"] = torch.einsum("mk,mk->k", dy, xh)
        if norm == "layer":
            out["dbias"] = dy.sum(dim=0)
    return out
