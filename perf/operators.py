"""Cases of the feed-forward operators: what a gated feed-forward block runs
in training (16-bit) and in serving (8-bit integers).

    quant_i8      rows -> 8-bit integers and one scale a row
    gemm_i8       product of 8-bit integers, one scale a token and a channel, bias
    gemm_glu      H = act(X Wg^T) * (X Wu^T), optionally with both pre-activations
    gemm_glu_i8   the same from 8-bit integers with scales
    gemm_glu_bwd  dX, dWg, dWu from dH and the saved pre-activations

`run` computes a case in its plain form (elementary torch operations in
float32, rounded once), or with this package's kernels where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # activations of a small decode batch, before an integer product
        dict(name="quant_decode_16", op="quant_i8", m=16, k=7168, dtype="bf16"),
        # activations of a long prefill: bandwidth
        dict(name="quant_prefill_16k", op="quant_i8", m=16384, k=7168, dtype="f16"),
        # down projection for one token: latency, and the weights' bytes
        dict(name="i8_token_1", op="gemm_i8", m=1, n=7168, k=2048, out="bf16", bias=False),
        # a decode batch of odd size, with bias
        dict(name="i8_batch_67", op="gemm_i8", m=67, n=4096, k=7168, out="f16", bias=True),
        # a large prefill: the matrix cores
        dict(name="i8_prefill_8k", op="gemm_i8", m=8192, n=8192, k=8192, out="bf16", bias=False),
        # gated up projection of a decode batch from integers
        dict(name="glu_i8_batch_8", op="gemm_glu_i8", m=8, n=2048, k=7168, out="bf16", act="silu"),
        # and of a ragged prefill
        dict(name="glu_i8_prefill_4001", op="gemm_glu_i8", m=4001, n=8192, k=4096, out="f16", act="gelu_tanh"),
        # gated up projection for one token, 16-bit weights
        dict(name="glu_token_1", op="gemm_glu", m=1, n=2048, k=7168, dtype="bf16", act="silu", save=False),
        # a short prompt of odd length
        dict(name="glu_prompt_509", op="gemm_glu", m=509, n=2048, k=7168, dtype="f16", act="gelu_tanh", save=False),
        # a training step's forward pass, pre-activations kept
        dict(name="glu_train_8k", op="gemm_glu", m=8192, n=8192, k=4096, dtype="bf16", act="silu", save=True),
        # backward of a narrow block on a ragged number of tokens
        dict(name="glu_bwd_1003", op="gemm_glu_bwd", m=1003, n=1408, k=2048, dtype="f16", act="relu"),
        # backward of a training step
        dict(name="glu_bwd_8k", op="gemm_glu_bwd", m=8192, n=8192, k=4096, dtype="bf16", act="silu"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, step * max(1, round(v / step))))


def draw(rng):
    op = rng.choice(["quant_i8", "gemm_i8", "gemm_glu_i8", "gemm_glu", "gemm_glu_bwd"])
    act = rng.choice(["silu", "gelu_tanh", "relu"])
    if op == "quant_i8":
        return dict(op=op, m=_log(rng, 1, 16384), k=_log(rng, 256, 7168, 16), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "gemm_i8":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 256, 8192, 8), k=_log(rng, 256, 8192, 16),
                    out=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.5)
    if op == "gemm_glu_i8":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 256, 8192, 8), k=_log(rng, 256, 4096, 16),
                    out=rng.choice(["bf16", "f16"]), act=act)
    if op == "gemm_glu":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 256, 8192, 8), k=_log(rng, 256, 4096, 8),
                    dtype=rng.choice(["bf16", "f16"]), act=act, save=rng.random() < 0.5)
    return dict(op=op, m=_log(rng, 128, 8192), n=_log(rng, 256, 8192, 8), k=_log(rng, 256, 4096, 8),
                dtype=rng.choice(["bf16", "f16"]), act=act)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _codes(gen, rows, cols, std):
    """Normal rows as a model's quantiser leaves them: codes and a scale a row."""
    x = torch.randn(rows, cols, generator=gen, device=DEV, dtype=torch.float32)
    top = x.abs().amax(1, keepdim=True).clamp_min_(1e-6)
    s = top.mul(std / 127.0)
    return x.mul_(127.0).div_(top).round_().to(torch.int8), s.reshape(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]
    s = dict(case=case, workspace=None)

    def normal(rows, cols, std, dt):
        return torch.randn(rows, cols, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dt)

    if op == "quant_i8":
        x = torch.randn(m, k, generator=gen, device=DEV, dtype=torch.float32)
        # tokens differ in size, and a few channels stand out
        x.mul_(torch.rand(m, 1, generator=gen, device=DEV).mul_(4).exp_())
        x[:, :: max(1, k // 7)] *= 20
        s["x"] = x.to(DT[case["dtype"]])
        s["q"] = torch.empty(m, k, dtype=torch.int8, device=DEV)
        s["scale"] = torch.empty(m, dtype=torch.float32, device=DEV)
        return s
    n = case["n"]
    # weights of variance 1/k: products are of the size of their inputs
    std = k ** -0.5
    if op in ("gemm_i8", "gemm_glu_i8"):
        s["a"], s["a_scale"] = _codes(gen, m, k, 1.0)
        if op == "gemm_i8":
            s["b"], s["b_scale"] = _codes(gen, n, k, std)
            s["bias"] = normal(1, n, 0.1, DT[case["out"]]).reshape(-1) if case["bias"] else None
        else:
            s["wg"], s["g_scale"] = _codes(gen, n, k, std)
            s["wu"], s["u_scale"] = _codes(gen, n, k, std)
        s["out"] = torch.empty(m, n, dtype=DT[case["out"]], device=DEV)
        return s
    dt = DT[case["dtype"]]
    s["x"] = normal(m, k, 1.0, dt)
    s["wg"], s["wu"] = normal(n, k, std, dt), normal(n, k, std, dt)
    if op == "gemm_glu":
        s["h"] = torch.empty(m, n, dtype=dt, device=DEV)
        s["g"] = torch.empty_like(s["h"]) if case["save"] else None
        s["u"] = torch.empty_like(s["h"]) if case["save"] else None
        return s
    s["g"], s["u"], s["dh"] = normal(m, n, 1.0, dt), normal(m, n, 1.0, dt), normal(m, n, 0.5, dt)
    s["dx"] = torch.empty(m, k, dtype=dt, device=DEV)
    s["dwg"], s["dwu"] = torch.empty(n, k, dtype=dt, device=DEV), torch.empty(n, k, dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "relu":
        return torch.clamp_min(x, 0.0)
    return 0.5 * x * (1.0 + torch.tanh(GELU_C * (x + GELU_A * x * x * x)))


def _act_grad(x, kind):
    if kind == "silu":
        p = torch.sigmoid(x)
        return p * (1.0 + x * (1.0 - p))
    if kind == "relu":
        return (x > 0).to(x.dtype)
    t = torch.tanh(GELU_C * (x + GELU_A * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * x * x)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "quant_i8":
        x = s["x"].float()
        top = x.abs().amax(1).clamp_min(2.0 ** -100)
        inv = torch.true_divide(torch.full_like(top, 127.0), top)
        q = torch.round(x * inv[:, None]).clamp(-127, 127).to(torch.int8)
        return {"q": q, "scale": top / 127.0}
    if op == "gemm_i8":
        y = s["a"].float() @ s["b"].float().t()
        y = y * s["a_scale"][:, None] * s["b_scale"][None, :]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(DT[c["out"]])
    if op == "gemm_glu_i8":
        a = s["a"].float()
        g = (a @ s["wg"].float().t()) * s["a_scale"][:, None] * s["g_scale"][None, :]
        u = (a @ s["wu"].float().t()) * s["a_scale"][:, None] * s["u_scale"][None, :]
        return (_act(g, c["act"]) * u).to(DT[c["out"]])
    dt = DT[c["dtype"]]
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    if op == "gemm_glu":
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(g, c["act"]) * u).to(dt)
        return {"h": h, "g": g.to(dt), "u": u.to(dt)} if c["save"] else {"h": h}
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    dg, du = dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])
    return {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt)}


def _kernels(s):
    import block_scaled_gemm_02_amd as bsg

    c, op, m, k = s["case"], s["case"]["op"], s["case"]["m"], s["case"]["k"]
    if op == "quant_i8":
        bsg.quant_i8(s["x"], s["q"], s["scale"], m, k)
        return {"q": s["q"], "scale": s["scale"]}
    n = c["n"]
    if s["workspace"] is None:      # scratch that a program keeps beside its layer
        s["workspace"] = torch.empty(bsg.workspace_bytes(op, m, n, k), dtype=torch.uint8, device=DEV)
    ws = s["workspace"]
    if op == "gemm_i8":
        bsg.gemm_i8(s["a"], s["b"], s["a_scale"], s["b_scale"], s["bias"], s["out"], m, n, k, workspace=ws)
        return s["out"]
    if op == "gemm_glu_i8":
        bsg.gemm_glu_i8(s["a"], s["wg"], s["wu"], s["a_scale"], s["g_scale"], s["u_scale"], s["out"], m, n, k,
                        act=c["act"], workspace=ws)
        return s["out"]
    if op == "gemm_glu":
        bsg.gemm_glu(s["x"], s["wg"], s["wu"], s["h"], s["g"], s["u"], m, n, k, act=c["act"], workspace=ws)
        return {"h": s["h"], "g": s["g"], "u": s["u"]} if c["save"] else {"h": s["h"]}
    bsg.gemm_glu_bwd(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], s["dx"], s["dwg"], s["dwu"], m, n, k,
                     act=c["act"], workspace=ws)
    return {"dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quant_i8":
        return {"bytes": m * k * (SIZE[case["dtype"]] + 1) + 4 * m, "flops": 2 * m * k}
    n = case["n"]
    if op == "gemm_i8":
        o = SIZE[case["out"]]
        return {"bytes": m * k + n * k + o * m * n + 4 * (m + n) + (o * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "gemm_glu_i8":
        return {"bytes": m * k + 2 * n * k + SIZE[case["out"]] * m * n + 4 * (m + 2 * n), "flops": 4 * m * n * k}
    if op == "gemm_glu":
        return {"bytes": 2 * (m * k + 2 * n * k + m * n * (3 if case["save"] else 1)), "flops": 4 * m * n * k}
    # dh, g, u, x, both weights in; dx and both weight gradients out
    return {"bytes": 2 * (3 * m * n + 2 * m * k + 4 * n * k), "flops": 8 * m * n * k}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _glu64(g, u, kind):
    """(value, d value / d g, d value / d u) of act(g) * u."""
    if kind == "relu":
        on = g.gt(0).double()
        return on * g * u, on * u, on * g
    if kind == "silu":
        e = torch.exp(-g.abs())
        sig = torch.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        val, der = g * sig, sig + g * sig * (1.0 - sig)
    else:
        z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        # 1 + tanh z = 2 sigmoid(2 z)
        sig = torch.sigmoid(2.0 * z)
        val = g * sig
        der = sig + g * 2.0 * sig * (1.0 - sig) * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * g ** 2)
    return val * u, der * u, val


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant_i8":
        x = s["x"].double()
        top = x.abs().max(dim=1).values.clamp(min=2.0 ** -100)
        return {"q": None, "scale": top / 127.0}
    if op == "gemm_i8":
        a = s["a"].double().mul_(s["a_scale"].double().unsqueeze(1))
        b = s["b"].double().mul_(s["b_scale"].double().unsqueeze(1))
        y = torch.mm(a, b.t())
        return y if s["bias"] is None else y.add_(s["bias"].double())
    if op == "gemm_glu_i8":
        a = s["a"].double().mul_(s["a_scale"].double().unsqueeze(1))
        g = torch.mm(a, s["wg"].double().mul_(s["g_scale"].double().unsqueeze(1)).t())
        u = torch.mm(a, s["wu"].double().mul_(s["u_scale"].double().unsqueeze(1)).t())
        return _glu64(g, u, case["act"])[0]
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    if op == "gemm_glu":
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        h = _glu64(g, u, case["act"])[0]
        return {"h": h, "g": g, "u": u} if case["save"] else {"h": h}
    dh = s["dh"].double()
    _, to_g, to_u = _glu64(s["g"].double(), s["u"].double(), case["act"])
    dg, du = dh * to_g, dh * to_u
    return {"dx": torch.mm(dg, wg) + torch.mm(du, wu), "dwg": torch.mm(dg.t(), x), "dwu": torch.mm(du.t(), x)}
