"""The feed-forward operators beyond one dense bf16 block, in their plain form and as the library's kernels.

Three families, each reached through the public binding where ``own`` is true:

  grouped   y[r] = act(x[r] W[e]^T + b[e]) for the rows r of expert e (rows sorted by expert, ragged), and its gradients
  ckpt      the gated block that keeps its gate and up projections in 8 bits for the backward pass, and that backward pass
  w4        decode with 4-bit weights, a scale (and a zero point) for each group of k: one Linear, and the gated block

A case is a dict of plain values; ``kind`` names the call.
"""
import math

import torch

own = False

# The expert layer of a routed block (8 experts of 4096 -> 14336, 4096 tokens of two choices each), the 8192 -> 28672
# block, the 4096 square of a decode layer; the others are generic sizes, odd on purpose.
_LISTED = [
    # one projection of a routed layer over a training batch
    dict(name="experts_8192rows_8x4096-14336", kind="grouped_fwd", R=8192, E=8, K=4096, N=14336, act="none", bias=False),
    # many small experts and few rows, some experts without one: serving, and the tail of a batch
    dict(name="experts_200rows_64x1024-1536", kind="grouped_fwd", R=200, E=64, K=1024, N=1536, act="silu", bias=True),
    # that projection's gradients: input, and every expert's weight
    dict(name="experts_grad_8192rows_8x4096-14336", kind="grouped_bwd", R=8192, E=8, K=4096, N=14336, act="none", bias=False),
    # gradients with an activation and a bias, ragged in every size
    dict(name="experts_grad_3001rows_16x1032-1528", kind="grouped_bwd", R=3001, E=16, K=1032, N=1528, act="gelu_tanh", bias=True),
    # a training step of one gated block, forward and backward
    dict(name="ckpt_step_4096tok_4096-14336", kind="ckpt_step", M=4096, D=4096, H=14336, act="silu"),
    # a small model's step on an odd number of tokens
    dict(name="ckpt_step_1001tok_768-2056", kind="ckpt_step", M=1001, D=768, H=2056, act="gelu_tanh"),
    # the backward pass of the largest block, its checkpoint made earlier
    dict(name="ckpt_grad_4096tok_8192-28672", kind="ckpt_bwd", M=4096, D=8192, H=28672, act="gelu_tanh"),
    # the same on a middle-sized block
    dict(name="ckpt_grad_2047tok_2048-5640", kind="ckpt_bwd", M=2047, D=2048, H=5640, act="silu"),
    # one token through one square layer: latency
    dict(name="w4_linear_1tok_4096-4096", kind="w4_linear", M=1, K=4096, N=4096, G=128, zeros=False, bias=False, act="none"),
    # a full decode batch through a wide layer, fine groups with zero points
    dict(name="w4_linear_16tok_8192-28672", kind="w4_linear", M=16, K=8192, N=28672, G=32, zeros=True, bias=True, act="gelu_erf"),
    # one token through the largest gated block: bound by the weights
    dict(name="w4_block_1tok_8192-28672", kind="w4_glu", M=1, D=8192, H=28672, G=128, zeros=False, act="silu"),
    # a handful of tokens through a middle-sized gated block
    dict(name="w4_block_5tok_4096-14336", kind="w4_glu", M=5, D=4096, H=14336, G=64, zeros=True, act="gelu_tanh"),
]
_ACTS = ("none", "gelu_erf", "gelu_tanh", "relu", "silu")
_BLOCK = 32   # hidden units that share a checkpoint scale


def listed():
    return [dict(c) for c in _LISTED]


def _spread(rng, lo, hi, step):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    kind = rng.choice(("grouped_fwd", "grouped_bwd", "ckpt_step", "ckpt_bwd", "w4_linear", "w4_glu"))
    most = max((work(c) for c in _LISTED if c["kind"] == kind), key=lambda w: w["flops"])
    while True:
        act = rng.choice(_ACTS)
        if kind.startswith("grouped"):
            c = dict(kind=kind, R=_spread(rng, 1, 16384, 1), E=_spread(rng, 1, 128, 1), K=_spread(rng, 64, 8192, 8),
                     N=_spread(rng, 64, 16384, 8), act=act, bias=rng.random() < 0.5)
        elif kind.startswith("ckpt"):
            c = dict(kind=kind, M=_spread(rng, 1, 16384, 1), D=_spread(rng, 64, 8192, 8), H=_spread(rng, 64, 28672, 8), act=act)
        else:
            g = rng.choice((32, 64, 128))
            c = dict(kind=kind, M=rng.randint(1, 16), G=g, zeros=rng.random() < 0.5, act=act)
            if kind == "w4_linear":
                c.update(K=_spread(rng, 256, 28672, g), N=_spread(rng, 64, 32768, 8), bias=rng.random() < 0.5)
            else:
                c.update(D=_spread(rng, 256, 8192, 128), H=_spread(rng, 256, 28672, 128))
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.bfloat16)


def _uniform(g, bound, *shape, dtype=torch.bfloat16):
    return (torch.rand(*shape, device="cuda", generator=g, dtype=torch.float32) * (2 * bound) - bound).to(dtype)


def _sizes(seed, R, E):
    """Rows of each expert: uneven, about one expert in eight without any (as a router leaves them)."""
    g = torch.Generator().manual_seed(seed ^ 0x5EED)
    p = torch.rand(E, generator=g) + 0.25
    p[torch.rand(E, generator=g) < 0.125] = 0
    if not bool((p > 0).any()):
        p[0] = 1
    return torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)


def _w4_weight(g, N, K, G, zeros):
    bound = 1 / math.sqrt(K)
    q = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)   # codes 2j (low) and 2j + 1
    s = (torch.rand(N, K // G, device="cuda", generator=g) * 0.5 + 0.75).mul_(bound / 8).to(torch.bfloat16)
    z = torch.randint(5, 12, (N, K // G), device="cuda", generator=g).to(torch.bfloat16) if zeros else None
    return q, s, z


def prepare(case, seed):
    g = _gen(seed)
    k = case["kind"]
    st = dict(case)
    if k.startswith("grouped"):
        R, E, K, N = (case[n] for n in ("R", "E", "K", "N"))
        sizes = _sizes(seed, R, E)
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = torch.cumsum(sizes, 0)
        st.update(x=_normal(g, R, K), W=_uniform(g, 1 / math.sqrt(K), E, N, K), off=off.cuda(), longest=int(sizes.max()),
                  b=_uniform(g, 1 / math.sqrt(K), E, N) if case["bias"] else None)
        if k == "grouped_bwd":
            st["dy"] = _normal(g, R, N)
    elif k.startswith("ckpt"):
        M, D, H = (case[n] for n in ("M", "D", "H"))
        st.update(x=_normal(g, M, D), Wg=_uniform(g, 1 / math.sqrt(D), H, D), Wu=_uniform(g, 1 / math.sqrt(D), H, D),
                  Wd=_uniform(g, 1 / math.sqrt(H), D, H), dy=_normal(g, M, D))
        if k == "ckpt_bwd":   # a checkpoint of gate and up values of the size that these weights give (sd 1 / sqrt(3))
            st["codes"], st["scales"] = _checkpoint(_normal(g, M, H).float() * 0.577, _normal(g, M, H).float() * 0.577)
    elif k == "w4_linear":
        M, K, N = (case[n] for n in ("M", "K", "N"))
        st["x"] = _normal(g, M, K)
        st["q"], st["s"], st["z"] = _w4_weight(g, N, K, case["G"], case["zeros"])
        st["b"] = _uniform(g, 1 / math.sqrt(K), N) if case["bias"] else None
    else:
        M, D, H = (case[n] for n in ("M", "D", "H"))
        st["x"] = _normal(g, M, D)
        for n, (rows, cols) in (("g", (H, D)), ("u", (H, D)), ("d", (D, H))):
            st["q" + n], st["s" + n], st["z" + n] = _w4_weight(g, rows, cols, case["G"], case["zeros"])
    return st


# ---------------------------------------------------------------------------
# the plain form, in 32 bits
# ---------------------------------------------------------------------------
_C0, _C1 = math.sqrt(2 / math.pi), 0.044715


def _act(z, act):
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_C0 * (z + _C1 * z * z * z)))
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "gelu_erf":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * (_C0 * (1 + 3 * _C1 * z * z))
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _checkpoint(g, u):
    """g, u [M, H] fp32 -> E4M3 codes [M, 2H] and, for each row and 32 hidden units, the exponent (+ 127) of the least
    power of two that brings the block's largest magnitude to 448 or less."""
    M, H = g.shape
    nb = -(-H // _BLOCK)
    v = torch.nn.functional.pad(torch.stack((g, u), 1), (0, nb * _BLOCK - H)).view(M, 2, nb, _BLOCK)
    mant, ex = torch.frexp(v.abs().amax(-1, keepdim=True))   # mant in [0.5, 1)
    e = (ex - 9 + (mant > 0.875)).clamp(min=-126)
    codes = torch.ldexp(v, -e).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(M, 2, nb * _BLOCK)[:, :, :H].reshape(M, 2 * H).contiguous(), (e + 127).to(torch.uint8).reshape(M, 2 * nb)


def _values(codes, scales):
    M, H = codes.shape[0], codes.shape[1] // 2
    nb = scales.shape[1] // 2
    v = codes.view(torch.float8_e4m3fn).float().view(M, 2, H)
    s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127).view(M, 2, nb, 1)
    v = v * s.expand(M, 2, nb, _BLOCK).reshape(M, 2, nb * _BLOCK)[:, :, :H]
    return v[:, 0], v[:, 1]


def _ckpt_grads(st, g, u):
    x, dy, act = st["x"].float(), st["dy"].float(), st["act"]
    a = _act(g, act)
    dWd = dy.t() @ (a * u)
    dm = dy @ st["Wd"].float()
    dg, du = dm * u * _dact(g, act), dm * a
    dx = dg @ st["Wg"].float() + du @ st["Wu"].float()
    return tuple(t.bfloat16() for t in (dx, dg.t() @ x, du.t() @ x, dWd))


def _plain_ckpt_step(st):
    x = st["x"].float()
    g, u = x @ st["Wg"].float().t(), x @ st["Wu"].float().t()
    y = (_act(g, st["act"]) * u) @ st["Wd"].float().t()
    return (y.bfloat16(),) + _ckpt_grads(st, *_values(*_checkpoint(g, u)))


def _padded(st):
    """Rows of every expert side by side, [E, longest] indexes into the rows, and which of them exist."""
    off = st["off"].long()
    i = torch.arange(st["longest"], device=off.device) + off[:-1, None]
    there = i < off[1:, None]
    return torch.where(there, i, torch.zeros_like(i)), there


def _plain_grouped(st):
    i, there = _padded(st)
    x = st["x"].float()[i] * there[..., None]
    W = st["W"].float()
    back = i[there]

    def rows(t, cols):
        return torch.zeros(st["R"], cols, device=t.device).index_copy_(0, back, t[there]).bfloat16()

    if st["kind"] == "grouped_fwd":
        z = torch.bmm(x, W.transpose(1, 2))
        if st["b"] is not None:
            z = z + st["b"].float()[:, None]
        return rows(_act(z, st["act"]), st["N"])
    dz = st["dy"].float()[i] * there[..., None]
    if st["act"] != "none":
        z = torch.bmm(x, W.transpose(1, 2))
        if st["b"] is not None:
            z = z + st["b"].float()[:, None]
        dz = dz * _dact(z, st["act"])
    out = (rows(torch.bmm(dz, W), st["K"]), torch.bmm(dz.transpose(1, 2), x).bfloat16())
    return out + (dz.sum(1).bfloat16(),) if st["b"] is not None else out


def _w4_dense(q, s, z, dtype):
    N, Kh = q.shape
    c = torch.stack((q & 15, q >> 4), -1).view(N, s.shape[1], -1).to(dtype)
    return ((c - (8 if z is None else z.to(dtype)[..., None])) * s.to(dtype)[..., None]).view(N, 2 * Kh)


def _plain_w4(st):
    x = st["x"].float()
    if st["kind"] == "w4_linear":
        y = x @ _w4_dense(st["q"], st["s"], st["z"], torch.float32).t()
        if st["b"] is not None:
            y = y + st["b"].float()
        return _act(y, st["act"]).bfloat16()
    g, u = (x @ _w4_dense(st["q" + n], st["s" + n], st["z" + n], torch.float32).t() for n in "gu")
    return ((_act(g, st["act"]) * u) @ _w4_dense(st["qd"], st["sd"], st["zd"], torch.float32).t()).bfloat16()


# ---------------------------------------------------------------------------
def _kernels(st):
    import gemm_epilogue_bf16_amd as F

    k = st["kind"]
    if k == "grouped_fwd":
        return F.fmlp_grouped_linear(st["x"], st["off"], st["W"], st["b"], st["act"])
    if k == "grouped_bwd":
        dx, dW, db = F.fmlp_grouped_linear_bwd(st["x"], st["off"], st["W"], st["b"], st["act"], st["dy"])
        return (dx, dW, db) if db is not None else (dx, dW)
    if k == "ckpt_step":
        y, codes, scales = F.fmlp_glu_ckpt(st["x"], st["Wg"], st["Wu"], st["Wd"], st["act"])
        return (y,) + tuple(F.fmlp_glu_ckpt_bwd(st["x"], codes, scales, st["Wg"], st["Wu"], st["Wd"], st["act"], st["dy"]))
    if k == "ckpt_bwd":
        return tuple(F.fmlp_glu_ckpt_bwd(st["x"], st["codes"], st["scales"], st["Wg"], st["Wu"], st["Wd"], st["act"], st["dy"]))
    if k == "w4_linear":
        return F.fmlp_linear_w4(st["x"], st["q"], st["s"], st["z"], st["b"], st["act"])
    return F.fmlp_glu_w4(st["x"], st["qg"], st["sg"], st["zg"], st["qu"], st["su"], st["zu"], st["qd"], st["sd"], st["zd"], st["act"])


def run(st):
    if own:
        return _kernels(st)
    k = st["kind"]
    if k.startswith("grouped"):
        return _plain_grouped(st)
    if k == "ckpt_step":
        return _plain_ckpt_step(st)
    if k == "ckpt_bwd":
        return _ckpt_grads(st, *_values(st["codes"], st["scales"]))
    return _plain_w4(st)


def work(case):
    k = case["kind"]
    if k.startswith("grouped"):
        R, E, K, N = (case[n] for n in ("R", "E", "K", "N"))
        W, b, gemm = E * N * K * 2, E * N * 2 * case["bias"], 2 * R * K * N
        if k == "grouped_fwd":
            return {"bytes": R * K * 2 + W + b + R * N * 2 + 4 * (E + 1), "flops": gemm}
        return {"bytes": 2 * (R * K * 2 + W + b) + R * N * 2 + 4 * (E + 1), "flops": (2 + (case["act"] != "none")) * gemm}
    if k.startswith("ckpt"):
        M, D, H = (case[n] for n in ("M", "D", "H"))
        W, gemm = 3 * D * H * 2, 2 * M * D * H
        saved = 2 * M * H + 2 * M * -(-H // _BLOCK)
        back = {"bytes": M * D * 6 + 2 * W + saved, "flops": 6 * gemm}
        if k == "ckpt_bwd":
            return back
        return {"bytes": back["bytes"] + M * D * 2, "flops": 9 * gemm}
    M, G = case["M"], case["G"]
    per = 0.5 + (4 if case["zeros"] else 2) / G   # bytes of a weight
    if k == "w4_linear":
        K, N = case["K"], case["N"]
        return {"bytes": int(N * K * per) + 2 * (M * K + M * N + N * case["bias"]), "flops": 2 * M * K * N}
    D, H = case["D"], case["H"]
    return {"bytes": int(3 * D * H * per) + 4 * M * D, "flops": 6 * M * D * H}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _act64(z, act):
    """(act(z), its derivative)"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).double()
        return z * on, on
    if act == "silu":
        s = torch.special.expit(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu_erf":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))   # (1 + tanh) / 2
    return z * s, s + 2 * z * s * (1 - s) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)


def _e4m3(v):
    """The nearest E4M3 value, ties to even; |v| is at most 448."""
    ex = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), ex.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _kept(v):
    """What a checkpoint of v [M, H] stands for."""
    out = torch.empty_like(v)
    for at in range(0, v.shape[1], _BLOCK):
        b = v[:, at:at + _BLOCK]
        top = b.abs().amax(1, keepdim=True)
        s = torch.exp2(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -126))))
        out[:, at:at + _BLOCK] = _e4m3(b / s) * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    k, act = case["kind"], case["act"]
    if k.startswith("grouped"):
        off = st["off"].tolist()
        x, b = st["x"].double(), st["b"]
        y = torch.zeros(case["R"], case["N"], device="cuda", dtype=torch.float64)
        dx, dW, db = torch.zeros_like(x), [], []
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            We = st["W"][e].double()
            z = torch.addmm(torch.zeros(case["N"], device="cuda", dtype=torch.float64) if b is None else b[e].double(), x[lo:hi], We.t())
            a, da = _act64(z, act)
            y[lo:hi] = a
            if k == "grouped_bwd":
                dz = st["dy"][lo:hi].double() * da
                dx[lo:hi] = dz @ We
                dW.append((dz.t() @ x[lo:hi]).float())   # a rounding to 24 bits, far below what is compared, for the memory
                db.append(dz.sum(0))
        if k == "grouped_fwd":
            return y
        return (dx, torch.stack(dW)) + ((torch.stack(db),) if b is not None else ())
    if k.startswith("ckpt"):
        x, dy = st["x"].double(), st["dy"].double()
        Wg, Wu, Wd = (st[n].double() for n in ("Wg", "Wu", "Wd"))
        first = ()
        if k == "ckpt_step":
            g, u = x @ Wg.t(), x @ Wu.t()
            first = ((_act64(g, act)[0] * u) @ Wd.t(),)
            g, u = _kept(g), _kept(u)
        else:
            H = case["H"]
            v, s = st["codes"].int(), st["scales"].double()
            mag = torch.where((v & 0x78) == 0, (v & 7) * 2.0 ** -9, (8 + (v & 7)) * torch.exp2(((v >> 3) & 15).double() - 10))
            v = torch.where(v > 127, -mag, mag)
            col = torch.arange(H, device="cuda") // _BLOCK
            s = torch.exp2(s - 127)
            g, u = v[:, :H] * s[:, col], v[:, H:] * s[:, col + s.shape[1] // 2]
        a, da = _act64(g, act)
        dWd = dy.t() @ (a * u)
        dm = dy @ Wd
        du = dm * a
        dg = dm * u * da
        return first + (dg @ Wg + du @ Wu, dg.t() @ x, du.t() @ x, dWd)
    x = st["x"].double()
    if k == "w4_linear":
        z = x @ _dense64(st["q"], st["s"], st["z"]).t()
        return _act64(z if st["b"] is None else z + st["b"].double(), act)[0]
    g = x @ _dense64(st["qg"], st["sg"], st["zg"]).t()
    u = x @ _dense64(st["qu"], st["su"], st["zu"]).t()
    return (_act64(g, act)[0] * u) @ _dense64(st["qd"], st["sd"], st["zd"]).t()


def _dense64(q, s, z):
    """Weights of packed codes: code k of a row is the low (k even) or the high half of byte k // 2."""
    W = torch.empty(q.shape[0], 2 * q.shape[1], device=q.device, dtype=torch.float64)
    W[:, 0::2] = (q % 16).double()
    W[:, 1::2] = (q // 16).double()
    per = W.shape[1] // s.shape[1]
    W -= 8.0 if z is None else z.double().repeat_interleave(per, 1)
    return W.mul_(s.double().repeat_interleave(per, 1))
