"""The gated block with an 8-bit checkpoint on the GPU, against the plain 64-bit
form with the bounds of ffn64.py."""
import pytest
import torch

import ffn64

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8, 8), (3, 72, 40), (17, 64, 32), (130, 96, 264), (257, 520, 136), (700, 256, 1032), (1500, 264, 2056)]


def make(M, D, H, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    t = dict(x=rnd(M, D), Wg=rnd(H, D) / D ** 0.5, Wu=rnd(H, D) / D ** 0.5, Wd=rnd(D, H) / H ** 0.5, dy=rnd(M, D))
    return {k: v.bfloat16() for k, v in t.items()}


def blocks(v):
    """largest finite magnitude of each row's blocks of 32"""
    nb = -(-v.shape[1] // 32)
    v = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    return torch.nn.functional.pad(v, (0, nb * 32 - v.shape[1])).view(v.shape[0], nb, 32).amax(-1)


def exponents(top):
    """the least e >= -126 with top <= 448 * 2^e"""
    mant, ex = torch.frexp(top)
    return torch.where(top > 0, (ex - 9 + (mant > 0.875)).clamp(min=-126), torch.full_like(ex, -126))


def check_stored(v, ev, codes, scales):
    """A half of a checkpoint against the values v (known to ev) it should hold."""
    top = blocks(v)
    e = scales.int() - 127
    # the maximum of values known to ev is known to the largest ev of the block
    etop = blocks(ev)
    assert bool(((e >= exponents(top - etop)) & (e <= exponents(top + etop))).all())
    unit = torch.exp2(e.double()).repeat_interleave(32, 1)[:, :v.shape[1]]
    kept = ffn64.e4m3_table().cuda()[codes.long()] * unit
    # half a step: 2^-4 of the value, or half of the least subnormal (2^-10) in the scaled unit
    ffn64.check("stored", kept, v, ev + torch.maximum(2.0 ** -4 * (v.abs() + ev), 2.0 ** -10 * unit))
    # and no code but the nearest, where the value is not at a border between two codes
    table = ffn64.e4m3_table()[:127].cuda()
    mids = (table[1:] + table[:-1]) / 2
    s = (v / unit).abs()
    near = (s.reshape(-1, 1) - mids).abs().amin(1).reshape(s.shape) > ev / unit + 1e-12
    want = table[torch.bucketize(s, mids)]
    assert torch.equal(want[near], (kept / unit).abs()[near])


@pytest.mark.parametrize("M,D,H", SHAPES)
@pytest.mark.parametrize("act", ffn64.ACTS)
def test_step(M, D, H, act):
    import gemm_epilogue_bf16_amd as F

    t = make(M, D, H)
    d = {k: v.double() for k, v in t.items()}
    y, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], act)
    assert codes.shape == (M, 2 * H) and scales.shape == (M, 2 * (-(-H // 32)))
    want, bound = ffn64.glu(d["x"], d["Wg"], d["Wu"], d["Wd"], act)
    ffn64.check("y", y, want, bound)
    nb = scales.shape[1] // 2
    for i, W in enumerate((d["Wg"], d["Wu"])):
        v, ev = ffn64.mm(d["x"], W.t())
        check_stored(v, ev, codes[:, i * H:(i + 1) * H], scales[:, i * nb:(i + 1) * nb])
    got = F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], act, t["dy"])
    want, bound = ffn64.glu_bwd_at(*ffn64.ckpt_values(codes, scales), d["x"], d["Wg"], d["Wu"], d["Wd"], act, d["dy"])
    for n, a, w, e in zip(("dx", "dWg", "dWu", "dWd"), got, want, bound):
        ffn64.check(n, a, w, e)
    again = F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], act, t["dy"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_large_tiles_and_split_products():
    """256-row tiles in every product: the weights read k-major"""
    import gemm_epilogue_bf16_amd as F

    M, D, H = 4100, 1032, 4104
    t = make(M, D, H, seed=1)
    d = {k: v.double() for k, v in t.items()}
    y, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], "gelu_tanh")
    want, bound = ffn64.glu(d["x"], d["Wg"], d["Wu"], d["Wd"], "gelu_tanh")
    ffn64.check("y", y, want, bound)
    nb = scales.shape[1] // 2
    v, ev = ffn64.mm(d["x"][:300], d["Wu"].t())
    check_stored(v, ev, codes[:300, H:], scales[:300, nb:])
    got = F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], "gelu_tanh", t["dy"])
    want, bound = ffn64.glu_bwd_at(*ffn64.ckpt_values(codes, scales), d["x"], d["Wg"], d["Wu"], d["Wd"], "gelu_tanh", d["dy"])
    for n, a, w, e in zip(("dx", "dWg", "dWu", "dWd"), got, want, bound):
        ffn64.check(n, a, w, e)


# the weight gradients in one launch, with either tile, in two, and in three
@pytest.mark.parametrize("M,D,H", [(300, 512, 1000), (601, 776, 3080), (600, 1032, 5128), (2100, 2056, 5128)])
def test_weight_gradients_of_every_form(M, D, H):
    gradients_at(M, D, H, "relu")


def test_operands_past_31_bits():
    """dg and du together span 2^31 bytes: their products read rewritten copies"""
    gradients_at(65536 + 8, 8, 8192, "silu")


def test_forward_past_32_bits():
    """2^32 codes and more: the rows at the end"""
    import gemm_epilogue_bf16_amd as F

    M, D, H = (1 << 19) + 200, 16, 4096
    t = make(M, D, H, seed=10)
    y, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], "silu")
    r = slice(M - 300, M)
    d = {k: v.double() for k, v in t.items() if k != "dy"}
    want, bound = ffn64.glu(d["x"][r], d["Wg"], d["Wu"], d["Wd"], "silu")
    ffn64.check("y", y[r], want, bound)
    nb = scales.shape[1] // 2
    for i, W in enumerate((d["Wg"], d["Wu"])):
        v, ev = ffn64.mm(d["x"][r], W.t())
        check_stored(v, ev, codes[r, i * H:(i + 1) * H], scales[r, i * nb:(i + 1) * nb])


def gradients_at(M, D, H, act):
    import gemm_epilogue_bf16_amd as F

    t = make(M, D, H, seed=9)
    d = {k: v.double() for k, v in t.items()}
    _, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], act)
    got = F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], act, t["dy"])
    want, bound = ffn64.glu_bwd_at(*ffn64.ckpt_values(codes, scales), d["x"], d["Wg"], d["Wu"], d["Wd"], act, d["dy"])
    for n, a, w, e in zip(("dx", "dWg", "dWu", "dWd"), got, want, bound):
        ffn64.check(n, a, w, e)


def test_codes_of_every_value():
    """The backward reads every finite code and scales over their range: g takes all 254 finite codes, at scales from
    2^-20 to 2^3, with u = 1.  dm = dy Wd is then seen through du = dm act(g) (act none: g itself) exactly."""
    import gemm_epilogue_bf16_amd as F

    H, D = 256, 8
    M = 24
    finite = [c for c in range(256) if c & 127 != 127]
    row = torch.tensor((finite + finite)[:H], dtype=torch.uint8)
    codes = torch.empty(M, 2 * H, dtype=torch.uint8)
    codes[:, :H] = row
    codes[:, H:] = 0x38   # 1.0
    scales = torch.full((M, 2 * (H // 32)), 127, dtype=torch.uint8)
    scales[:, :H // 32] = (torch.arange(M) + 107).to(torch.uint8)[:, None]
    x = torch.zeros(M, D, dtype=torch.bfloat16)
    x[:, 0] = 1
    dy = torch.zeros(M, D, dtype=torch.bfloat16)
    dy[0, 0] = 1   # only token 0 has a gradient: dWu's column 0 is du of token 0
    Wd = torch.zeros(D, H, dtype=torch.bfloat16)
    Wd[0] = 1
    W = torch.zeros(H, D, dtype=torch.bfloat16)
    a = [t.cuda() for t in (x, codes, scales, W, W, Wd)]
    for m in range(M):
        dy.zero_()
        dy[m, 0] = 1
        _, dWg, dWu, dWd = F.fmlp_glu_ckpt_bwd(*a, "none", dy.cuda())
        g = ffn64.e4m3_table()[row.long()] * 2.0 ** (m + 107 - 127)
        assert torch.equal(dWu[:, 0].double().cpu(), g)          # 4 significant bits: exact in bf16
        assert torch.equal(dWd[0].double().cpu(), g)             # m = g * 1
        assert bool((dWg[:, 0] == 1).all())


def test_zero_rows_and_wide_ranges():
    import gemm_epilogue_bf16_amd as F

    t = make(64, 64, 96, seed=2)
    x = t["x"]
    x[0] = 0
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -60
    x[3] = x[3] * 2.0 ** -126   # subnormal products
    y, codes, scales = F.fmlp_glu_ckpt(x, t["Wg"], t["Wu"], t["Wd"], "none")
    assert not codes[0].any() and bool((scales[0] == 1).all())
    for i, n in enumerate(("Wg", "Wu")):
        v, ev = ffn64.mm(x[:3].double(), t[n].double().t())
        check_stored(v, ev, codes[:3, i * 96:(i + 1) * 96], scales[:3, i * 3:(i + 1) * 3])
    assert bool((scales[3] <= 12).all()) and bool((scales[3] >= 1).all())


def test_not_finite():
    """An infinity or NaN in a row of x: its g and u are stored as NaN, other rows are untouched; a non-finite single g
    does not reach its block's scale."""
    import gemm_epilogue_bf16_amd as F

    t = make(40, 64, 96, seed=3)
    clean = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], "silu")
    x = t["x"].clone()
    x[5, 3] = float("inf")
    x[9, 7] = float("nan")
    y, codes, scales = F.fmlp_glu_ckpt(x, t["Wg"], t["Wu"], t["Wd"], "silu")
    others = torch.ones(40, dtype=torch.bool, device="cuda")
    others[[5, 9]] = False
    for a, b in ((y, clean[0]), (codes, clean[1]), (scales, clean[2])):
        assert torch.equal(a[others], b[others])
    assert bool(((codes[[5, 9]] & 127) == 127).all())
    # one weight row gives an infinite g: only that unit is NaN, and the block keeps the others' scale
    Wg = t["Wg"].clone()
    Wg[33] = float("inf")
    y, codes, scales = F.fmlp_glu_ckpt(t["x"], Wg, t["Wu"], t["Wd"], "silu")
    assert bool(((codes[:, 33] & 127) == 127).all())
    keep = torch.arange(96, device="cuda") != 33
    g = ffn64.mm(t["x"].double(), t["Wg"].double().t())
    v = g[0].clone()
    v[:, 33] = 0
    kept, _ = ffn64.ckpt_values(codes, scales)
    assert bool((torch.abs(kept - g[0])[:, keep] <= 2.0 ** -4 * v.abs().amax(1, keepdim=True)).all())


def test_gradients_near_those_of_the_full_values():
    """Eight bits keep each g and u to 2^-4, so the gradients stay near those of the unrounded block: a sum of many terms
    whose errors are independent.  Checked as what it is, a bound on the terms: |dx - dx_full| <= 2^-4 (L |g| + |u|) sums."""
    import gemm_epilogue_bf16_amd as F

    t = make(256, 128, 320, seed=4)
    d = {k: v.double() for k, v in t.items()}
    _, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"], "silu")
    got = F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], "silu", t["dy"])
    g, u = d["x"] @ d["Wg"].t(), d["x"] @ d["Wu"].t()
    full, own = ffn64.glu_bwd_at(g, u, d["x"], d["Wg"], d["Wu"], d["Wd"], "silu", d["dy"])
    # stored values are off by at most 2^-4 of themselves plus 2^-10 of the scaled unit, which is at most 2^-8 of the
    # block's maximum; silu' is at most 1.1 and its slope at most 0.5
    top = lambda v: blocks(v).repeat_interleave(32, 1)[:, :v.shape[1]]   # noqa: E731
    eg, eu = 2.0 ** -4 * g.abs() + 2.0 ** -17 * top(g), 2.0 ** -4 * u.abs() + 2.0 ** -17 * top(u)
    dm = (d["dy"] @ d["Wd"]).abs()
    a, da = ffn64.act64(g, "silu")
    em = 1.1 * eg * (u.abs() + eu) + a.abs() * eu
    edg = dm * (0.5 * eg * (u.abs() + eu) + da.abs() * eu)
    edu = dm * 1.1 * eg
    extra = (edg @ d["Wg"].abs() + edu @ d["Wu"].abs(), edg.t() @ d["x"].abs(), edu.t() @ d["x"].abs(), d["dy"].abs().t() @ em)
    for n, a_, w, e, x in zip(("dx", "dWg", "dWu", "dWd"), got, full, own, extra):
        ffn64.check(n, a_, w, 1.01 * (e + x))


def test_gradient_agrees_with_differences():
    """against central differences of the 64-bit block, at a g and u that the checkpoint holds exactly"""
    import gemm_epilogue_bf16_amd as F

    M = D = 64
    H = 96
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.eye(M, device="cuda", dtype=torch.float64)   # g and u are then the weights' columns: 4 significant bits
    grid = lambda *s: torch.randint(-15, 16, s, generator=g, device="cuda").double() / 8   # noqa: E731
    Wg, Wu = grid(H, D), grid(H, D)
    Wd = torch.randn(D, H, generator=g, device="cuda").bfloat16().double() / 8
    dy = torch.randn(M, D, generator=g, device="cuda").bfloat16().double()
    t = [v.bfloat16() for v in (x, Wg, Wu, Wd)]
    y, codes, scales = F.fmlp_glu_ckpt(*t, "gelu_tanh")
    gg, uu = ffn64.ckpt_values(codes, scales)
    assert torch.equal(gg, Wg.t()) and torch.equal(uu, Wu.t())
    grads = F.fmlp_glu_ckpt_bwd(t[0], codes, scales, *t[1:], "gelu_tanh", dy.bfloat16())
    _, bound = ffn64.glu_bwd_at(gg, uu, x, Wg, Wu, Wd, "gelu_tanh", dy)
    p = dict(x=x, Wg=Wg, Wu=Wu, Wd=Wd)
    h = 1e-5
    for n, grad, e in zip(("x", "Wg", "Wu", "Wd"), grads, bound):
        v = torch.randn(p[n].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(s):
            q = dict(p)
            q[n] = p[n] + s * v
            return float((((ffn64.act64(q["x"] @ q["Wg"].t(), "gelu_tanh")[0] * (q["x"] @ q["Wu"].t())) @ q["Wd"].t()) * dy).sum())

        quotient = (loss(h) - loss(-h)) / (2 * h)
        assert abs(quotient - float((grad.double() * v).sum())) <= float((e * v.abs()).sum()) + 1e-4


def test_no_tokens_and_leading_dims():
    import gemm_epilogue_bf16_amd as F

    t = make(6, 64, 96, seed=5)
    x = t["x"].view(2, 3, 64)
    y, codes, scales = F.fmlp_glu_ckpt(x, t["Wg"], t["Wu"], t["Wd"])
    assert y.shape == x.shape
    dx, *_ = F.fmlp_glu_ckpt_bwd(x, codes, scales, t["Wg"], t["Wu"], t["Wd"], "silu", t["dy"].view(2, 3, 64))
    assert dx.shape == x.shape
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, codes, scales = F.fmlp_glu_ckpt(e, t["Wg"], t["Wu"], t["Wd"])
    assert y.shape == (0, 64) and codes.shape == (0, 192)
    dx, *dW = F.fmlp_glu_ckpt_bwd(e, codes, scales, t["Wg"], t["Wu"], t["Wd"], "silu", e)
    assert not any(w.any() for w in dW)


def test_under_graph_capture():
    import gemm_epilogue_bf16_amd as F

    t = make(300, 128, 264, seed=6)

    def step():
        y, codes, scales = F.fmlp_glu_ckpt(t["x"], t["Wg"], t["Wu"], t["Wd"])
        return (y, codes, scales) + F.fmlp_glu_ckpt_bwd(t["x"], codes, scales, t["Wg"], t["Wu"], t["Wd"], "silu", t["dy"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        t["x"].copy_(torch.randn(300, 128, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


def test_refusals():
    import gemm_epilogue_bf16_amd as F

    t = make(8, 64, 96)
    x, Wg, Wu, Wd, dy = (t[k] for k in ("x", "Wg", "Wu", "Wd", "dy"))
    y, codes, scales = F.fmlp_glu_ckpt(x, Wg, Wu, Wd)
    for call, err in ((lambda: F.fmlp_glu_ckpt(x.float(), Wg, Wu, Wd), TypeError),
                      (lambda: F.fmlp_glu_ckpt(x, Wg, Wu, Wd.t()), ValueError),
                      (lambda: F.fmlp_glu_ckpt(x, Wg[:64], Wu, Wd), ValueError),
                      (lambda: F.fmlp_glu_ckpt(x, Wg, Wu, Wd, "swish"), KeyError),
                      (lambda: F.fmlp_glu_ckpt(x, Wg, Wu, Wd, out=(y, codes[:4], scales)), ValueError),
                      (lambda: F.fmlp_glu_ckpt_bwd(x, codes[:, :96].contiguous(), scales, Wg, Wu, Wd, "silu", dy), ValueError),
                      (lambda: F.fmlp_glu_ckpt_bwd(x, codes, scales.float(), Wg, Wu, Wd, "silu", dy), TypeError),
                      (lambda: F.fmlp_glu_ckpt_bwd(x, codes, scales[:4], Wg, Wu, Wd, "silu", dy), ValueError),
                      (lambda: F.fmlp_glu_ckpt_bwd(x, codes, scales, Wg, Wu, Wd, "silu", dy[:4]), ValueError),
                      (lambda: F.fmlp_glu_ckpt_bwd(x, codes, scales, Wg, Wu, Wd, "silu", dy,
                                                   workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), F.FmlpError)):
        with pytest.raises(err):
            call()
