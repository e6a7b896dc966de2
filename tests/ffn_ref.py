"""Plain 64-bit implementation of the feed-forward operators and the error
bounds their kernels have to keep, for tests/test_gpu_ffn.py.

Bounds, with e = 2^-24 (one fp32 rounding) and r the rounding of the output
type, half a step of its significand: 2^-p with p = 8 bits for bf16, 11 for fp16
and 24 for fp32, the leading one included (plus half its smallest step):
  * an fp32 sum of K products of exactly represented factors is off by at most
    (K + 1) e sum|products|, whatever its order;
  * an activation is evaluated with relative error at most 2^-20 (1 + |t|), t
    being the exponential's argument: its rounding gives |t| 2^-22, exp2 and
    rcp one ulp each;
  * |act'| <= 1.13 for all three activations, |act''| <= 1.6 (tanh-form GELU
    has the largest: 2 phi(0) = 0.8 at 0, doubled).
"""
import math

import torch

E = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
ACTS = ["silu", "gelu_tanh", "relu"]
C = math.sqrt(2.0 / math.pi)


def act64(g, kind):
    """(act, act', |exponential argument|) in float64."""
    if kind == "relu":
        return g.clamp(min=0.0), (g > 0).double(), torch.zeros_like(g)
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g), g.abs()
    t = 2 * C * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(t)
    return g * s, s + g * s * torch.sigmoid(-t) * 2 * C * (1 + 3 * 0.044715 * g ** 2), t.abs()


def out_bound(ref, err, dt):
    """An fp32 value within err of ref, rounded to dt."""
    return err + (ref.abs() + err) * ROUND[dt] + STEP[dt]


def glu64(x, wg, wu, kind):
    """(h, g, u) in float64 and the fp32 error bounds of each."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    k = x.shape[1]
    eg = (k + 1) * E * (x.abs() @ wg.abs().t())
    eu = (k + 1) * E * (x.abs() @ wu.abs().t())
    return (*_gate(g, u, eg, eu, kind), g, u, eg, eu)


def _gate(g, u, eg, eu, kind):
    a, _, t = act64(g, kind)
    ea = 1.13 * eg + 2.0 ** -20 * (1 + t) * a.abs()
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2 * E * (a * u).abs()


def i8_64(a, b, sa, sb):
    """Scaled integer product in float64 and its fp32 error bound: the exact
    int32 sum is converted and multiplied twice (three roundings)."""
    y = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :]
    return y, 4 * E * y.abs()


def glu_bwd64(dh, x, wg, wu, g, u, kind, dt):
    """(dx, dwg, dwu) in float64 and their bounds before the output rounding:
    dG and dU carry the activation's error and one rounding to dt."""
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, g, u))
    a, d, t = act64(g, kind)
    dg, du = dh * u * d, dh * a
    # act' is a sum of two terms of the activation's accuracy: |g s (1-s) ...| <= 1.6 |g| bounds the second
    ed = 0.0 if kind == "relu" else 2.0 ** -20 * (1 + t) * (d.abs() + 1.13)
    eg = (dh * u).abs() * ed + 3 * E * dg.abs()
    eu = dh.abs() * 2.0 ** -20 * (1 + t) * a.abs() + 2 * E * du.abs()
    eg, eu = out_bound(dg, eg, dt), out_bound(du, eu, dt)
    m, n = g.shape
    mag = (dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs()
    dx, ex = dg @ wg + du @ wu, eg @ wg.abs() + eu @ wu.abs() + (2 * n + 1) * E * mag
    out = [(dx, ex)]
    for z, ez in ((dg, eg), (du, eu)):
        out.append((z.t() @ x, ez.t() @ x.abs() + (m + 1) * E * ((z.abs() + ez).t() @ x.abs())))
    return out


def check(name, got, ref, err, dt):
    """got (dtype dt) within its bound of ref, element by element."""
    assert got.dtype == dt and tuple(got.shape) == tuple(ref.shape)
    bound = out_bound(ref, err, dt)
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} past their bound, first {i}: "
                             f"{float(got[i])} for {float(ref[i])} +- {float(bound[i])}")
