"""Plain 64-bit forms of the grouped products, the gated block with an 8-bit
checkpoint and the 4-bit decode, with a bound on the error of each output that
follows from the roundings the kernels make.

Every function takes float64 tensors (any device) and returns values and
elementwise bounds.  The roundings counted:
  * an fp32 sum of K terms: each of at most K + 8 additions rounds by 2^-24 of
    a partial sum, which sum |a||b| bounds (products of bf16 are exact in
    fp32); twice that, since a matrix instruction adds its terms in an order
    and at alignments of its own;
  * an activation: at most 16 fp32 operations on values of at most 1 + |z|
    (2^-24 each: 2^-20 (1 + |z|)), and the argument's own error times the
    slope, at most 1.13 (gelu), and 0.8 for the derivative (gelu'');
  * bf16 rounds by at most 2^-8 of the value, and by 2^-134 (half of the least
    subnormal) near zero.
"""
import math

import torch

ACTS = ("none", "gelu_erf", "gelu_tanh", "relu", "silu")
BF = 2.0 ** -8
F32 = 2.0 ** -24
C = math.sqrt(2 / math.pi)


def act64(z, act):
    """act(z) and its derivative"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu_erf":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(C * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)


def mm(a, b, ea=None, eb=None):
    """a [M, K] b [K, N] and its error, for operands that are off by ea and eb"""
    aa, ab = a.abs(), b.abs()
    e = 2 * (a.shape[1] + 8) * F32 * (aa @ ab)
    if ea is not None:
        e = e + ea @ ab
    if eb is not None:
        e = e + (aa if ea is None else aa + ea) @ eb
    return a @ b, e


def act_err(z, ez, act):
    """errors of act(z) and of act'(z) in fp32 for z off by ez"""
    if act == "none":
        return ez, torch.zeros_like(z)
    f = 2.0 ** -20 * (1 + z.abs())
    if act == "relu":
        return ez, (z.abs() <= ez).to(z.dtype)   # the step: either side of zero
    return 1.13 * ez + f, 0.8 * ez + f


def rounded(v, e):
    """error of v, known to e, once it is rounded to bf16"""
    return e + BF * (v.abs() + e) + 2.0 ** -134


def prod(a, ea, b, eb):
    """a b and its error (one fp32 rounding)"""
    v = a * b
    return v, a.abs() * eb + b.abs() * ea + ea * eb + F32 * v.abs()


def linear(x, W, b, act):
    z, ez = mm(x, W.t())
    if b is not None:
        z = z + b
        ez = ez + F32 * z.abs()
    return z, ez


def grouped(x, off, W, b, act):
    """y [R, N] (rows outside the groups NaN) and its bound"""
    y = torch.full((x.shape[0], W.shape[1]), float("nan"), dtype=torch.float64, device=x.device)
    e = y.clone()
    for g in range(len(off) - 1):
        r = slice(off[g], off[g + 1])
        z, ez = linear(x[r], W[g], None if b is None else b[g], act)
        y[r] = act64(z, act)[0]
        e[r] = rounded(y[r], act_err(z, ez, act)[0])
    return y, e


def grouped_bwd(x, off, W, b, act, dy):
    """(dx, dW, db) and their bounds"""
    dx = torch.full_like(x, float("nan"))
    edx = dx.clone()
    dW, db = torch.zeros_like(W), torch.zeros(W.shape[:2], dtype=torch.float64, device=x.device)
    edW, edb = torch.zeros_like(W), torch.zeros_like(db)
    for g in range(len(off) - 1):
        r = slice(off[g], off[g + 1])
        dz, e = dy[r], torch.zeros_like(dy[r])
        if act != "none":
            z, ez = linear(x[r], W[g], None if b is None else b[g], act)
            da = act64(z, act)[1]
            dz, e = prod(dy[r], torch.zeros_like(dz), da, act_err(z, ez, act)[1])
            e = rounded(dz, e)
        dx[r], t = mm(dz, W[g], e)
        edx[r] = rounded(dx[r], t)
        dW[g], t = mm(dz.t(), x[r], e.t())
        edW[g] = rounded(dW[g], t)
        db[g], t = dz.sum(0), e.sum(0) + 2 * (dz.shape[0] + 72) * F32 * dz.abs().sum(0)
        edb[g] = rounded(db[g], t)
    return (dx, dW, db), (edx, edW, edb)


def glu(x, Wg, Wu, Wd, act):
    """The gated block and its bound"""
    (g, eg), (u, eu) = mm(x, Wg.t()), mm(x, Wu.t())
    m, em = prod(act64(g, act)[0], act_err(g, eg, act)[0], u, eu)
    y, e = mm(m, Wd.t(), rounded(m, em))
    return y, rounded(y, e)


def glu_bwd_at(g, u, x, Wg, Wu, Wd, act, dy):
    """The gated block's gradients at given g and u, and their bounds"""
    z = torch.zeros_like(g)
    a, da = act64(g, act)
    ea, eda = act_err(g, z, act)
    m, em = prod(a, ea, u, z)
    em = rounded(m, em)
    dm, edm = mm(dy, Wd)
    t, et = prod(dm, edm, u, z)
    dg, edg = prod(t, et, da, eda)
    edg = rounded(dg, edg)
    du, edu = prod(dm, edm, a, ea)
    edu = rounded(du, edu)
    dx, edx = mm(torch.cat((dg, du), 1), torch.cat((Wg, Wu)), torch.cat((edg, edu), 1))
    outs = [(dx, edx), mm(dg.t(), x, edg.t()), mm(du.t(), x, edu.t()), mm(dy.t(), m, None, em)]
    return [v for v, _ in outs], [rounded(v, e) for v, e in outs]


def e4m3_table():
    """the values of the 256 E4M3 codes"""
    out = []
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        out.append(math.nan if e == 15 and m == 7 else s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)))
    return torch.tensor(out, dtype=torch.float64)


def ckpt_values(codes, scales):
    """g, u [M, H] that a checkpoint stands for"""
    H = codes.shape[1] // 2
    v = e4m3_table().to(codes.device)[codes.long()]
    col = torch.arange(H, device=codes.device) // 32
    s = torch.exp2(scales.double() - 127)
    return v[:, :H] * s[:, col], v[:, H:] * s[:, scales.shape[1] // 2 + col]


def check(name, got, want, bound):
    """Every element of got (any type) is within bound of want; NaN in want means "not looked at"."""
    got = got.double().to(want.device)
    look = ~torch.isnan(want)
    assert bool(torch.isfinite(got[look]).all()), f"{name}: not finite"
    off = torch.where(look, (got - want).abs() - bound, torch.full_like(want, -1.0))
    worst = float(off.max()) if off.numel() else -1.0
    if look.any():
        rel = float((got - want)[look].norm() / want[look].norm().clamp(min=1e-300))
        print(f"  {name}: rel {rel:.2e}, of its bound {float(((got - want).abs() / bound)[look].max()):.3f}", flush=True)
    assert worst <= 0, f"{name}: {int((off > 0).sum())} values outside their bound, worst by {worst:.3e}"


def w4_dense(q, s, z):
    """W, and |s| code and |s| |z|, which its two sums run over"""
    c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1).double()
    per = c.shape[1] // s.shape[1]
    z = torch.full_like(s, 8.0).double() if z is None else z.double()
    z, s = z.repeat_interleave(per, 1), s.double().repeat_interleave(per, 1)
    return s * (c - z), s.abs() * c, s.abs() * z.abs()


def w4_linear(x, ex, q, s, z):
    """x W^T for x known to ex (or None), and its error:
      * x as two E4M3 values under the power of two 2^e that brings the largest of its 128 k into (224, 448]: hi leaves at
        most 16 of the scaled 448, lo holds that to half of 2^-9 in units of 2^(e-4), so x is kept to 2^-10 2^(e-4) <=
        2^-14 / 224 of the largest, below 2^-21, and exactly where its last bit (2^-7 of its binade) is at least 2^-9
        of that unit: down to 2^-13 of the largest;
      * products of x and codes, aligned to 13 bits below a neighbour: 2^-13 each, twice that for two steps;
      * fp32 sums of x code and of -x z, and one scale each."""
    W, code, zero = w4_dense(q, s, z)
    K = x.shape[1]
    top = torch.nn.functional.pad(x.abs(), (0, -K % 128)).view(x.shape[0], -1, 128).amax(-1).repeat_interleave(128, 1)[:, :K]
    kept = torch.where(x.abs() >= 2.0 ** -13 * top, torch.zeros_like(x), 2.0 ** -21 * top)
    e = 2.0 ** -12 * (x.abs() @ code.t()) + kept @ code.t() + 2 * (K + 16) * F32 * (x.abs() @ (code + zero).t())
    return x @ W.t(), e if ex is None else e + ex @ W.abs().t()


def w4_glu(x, wg, wu, wd, act):
    (g, eg), (u, eu) = w4_linear(x, None, *wg), w4_linear(x, None, *wu)
    a = act64(g, act)[0]
    m, em = prod(a, act_err(g, eg, act)[0], u, eu)
    y, e = w4_linear(m, rounded(m, em), *wd)
    return y, rounded(y, e)
