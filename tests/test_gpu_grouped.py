"""Products grouped by expert and their gradients on the GPU, against the plain
64-bit form with the bounds of ffn64.py."""
import pytest
import torch

import ffn64

pytestmark = pytest.mark.gpu

# (rows of each group, rows before the first and after the last group, K, N)
SHAPES = [
    ([1], 0, 0, 8, 8),                                   # the smallest call
    ([5, 0, 3], 0, 0, 72, 40),                           # an empty group, ragged sizes
    ([0, 0, 17, 0], 2, 3, 264, 136),                     # rows that belong to nobody on both sides
    ([130, 1, 128, 127, 129], 0, 1, 96, 200),            # around a row tile
    ([300, 0, 513, 64, 65, 63], 1, 0, 256, 520),         # around the k stages of dW
    ([0, 0], 0, 7, 64, 64),                              # no group has rows
    ([2000, 1500, 600], 0, 0, 520, 776),                 # 256-row tiles, split weight gradient
    ([900, 1100, 950, 1146], 0, 0, 1032, 4104),          # 256-row tiles in every product
]


def make(rows, before, after, K, N, bias, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    R = before + sum(rows) + after
    off = [before]
    for n in rows:
        off.append(off[-1] + n)
    t = dict(x=torch.randn(R, K, generator=g, device=dev), W=torch.randn(len(rows), N, K, generator=g, device=dev) / K ** 0.5,
             b=torch.randn(len(rows), N, generator=g, device=dev) if bias else None,
             dy=torch.randn(R, N, generator=g, device=dev))
    t = {k: None if v is None else v.bfloat16() for k, v in t.items()}
    return t, off, torch.tensor(off, dtype=torch.int32, device=dev)


def dbl(t):
    return {k: None if v is None else v.double() for k, v in t.items()}


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[3]}-{s[4]}r{sum(s[0])}")
@pytest.mark.parametrize("act,bias", [("none", False), ("gelu_erf", True), ("gelu_tanh", True), ("relu", False), ("silu", True)])
def test_forward_and_gradients(shape, act, bias):
    import gemm_epilogue_bf16_amd as F

    rows, before, after, K, N = shape
    t, off, offs = make(rows, before, after, K, N, bias)
    d = dbl(t)
    R = t["x"].shape[0]
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], act, out=y)
    want, bound = ffn64.grouped(d["x"], off, d["W"], d["b"], act)
    ffn64.check("y", y, want, bound)
    outside = torch.ones(R, dtype=torch.bool)
    outside[off[0]:off[-1]] = False
    assert bool((y[outside.cuda()] == 7.0).all())

    dx = torch.full((R, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dW, db = torch.empty_like(t["W"]), torch.empty(len(rows), N, dtype=torch.bfloat16, device="cuda")
    F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], t["b"], act, t["dy"], out=(dx, dW, db))
    want, bound = ffn64.grouped_bwd(d["x"], off, d["W"], d["b"], act, d["dy"])
    for n, got, w, e in zip(("dx", "dW", "db"), (dx, dW, db), want, bound):
        ffn64.check(n, got, w, e)
    assert bool((dx[outside.cuda()] == 7.0).all())
    # the same call again gives the same bits
    again = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], t["b"], act, t["dy"])
    inside = ~outside.cuda()
    assert torch.equal(again[0][inside], dx[inside]) and torch.equal(again[1], dW)
    assert again[2] is None if not bias else torch.equal(again[2], db)


# few tiles over a long contraction, in up to 32 parts, a ragged last part, a group of one row and an empty one
@pytest.mark.parametrize("rows,K,N", [([200], 8200, 1032), ([1, 0, 90, 300], 4104, 264), ([257], 6152, 520), ([3], 9000, 8)])
@pytest.mark.parametrize("act", ffn64.ACTS)
def test_split_contraction(rows, K, N, act):
    import gemm_epilogue_bf16_amd as F

    t, off, offs = make(rows, 1, 2, K, N, act != "relu", seed=7)
    d = dbl(t)
    y = torch.full(t["dy"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], act, out=y)
    want, bound = ffn64.grouped(d["x"], off, d["W"], d["b"], act)
    ffn64.check("y", y, want, bound)
    assert bool((y[:1] == 7.0).all()) and bool((y[-2:] == 7.0).all())
    assert torch.equal(F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], act)[1:-2], y[1:-2])
    got = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], t["b"], act, t["dy"])
    want, bound = ffn64.grouped_bwd(d["x"], off, d["W"], d["b"], act, d["dy"])
    for n, a, w, e in zip(("dx", "dW", "db"), got, want, bound):
        if a is not None:
            ffn64.check(n, a, w, e)


def test_split_contraction_without_rows_and_under_capture():
    """The tables are the device's: a replayed graph follows them, down to groups without rows."""
    import gemm_epilogue_bf16_amd as F

    t, off, offs = make([120, 80], 0, 0, 4104, 264, True, seed=8)
    call = lambda: F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], "silu", out=y)   # noqa: E731
    y = torch.zeros_like(t["dy"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cut in ((0, 120, 200), (0, 0, 200), (5, 5, 5), (0, 200, 200)):
        offs.copy_(torch.tensor(cut, dtype=torch.int32))
        y.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.fill_(3.0)
        call()
        assert torch.equal(got, y), cut
        assert cut != (5, 5, 5) or bool((y == 3.0).all())


# dx's last tiles in 2 and 4 parts of a long contraction, whole rounds before them and none; rows of nobody
@pytest.mark.parametrize("rows,K,N", [([1000, 1100, 950, 1146, 900, 1096, 1000, 1000], 2056, 4104), ([0, 8000, 0, 31], 2056, 4104),
                                      ([1024, 1024, 1024, 1024], 1032, 4104), ([13, 4200, 1], 1032, 4168)])
def test_split_last_round(rows, K, N):
    import gemm_epilogue_bf16_amd as F

    t, off, offs = make(rows, 3, 2, K, N, False, seed=6)
    d = dbl(t)
    dx = torch.full(t["x"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    dW = torch.empty_like(t["W"])
    F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], None, "none", t["dy"], out=(dx, dW, None))
    want, bound = ffn64.grouped_bwd(d["x"], off, d["W"], None, "none", d["dy"])
    ffn64.check("dx", dx, want[0], bound[0])
    ffn64.check("dW", dW, want[1], bound[1])
    assert bool((dx[:3] == 7.0).all()) and bool((dx[-2:] == 7.0).all())
    again = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], None, "none", t["dy"])
    assert torch.equal(again[0][3:-2], dx[3:-2])


def test_gradient_agrees_with_differences():
    """The GPU's gradients against central differences of the 64-bit forward along random directions.  The difference
    quotient is off by h^2/6 of the third derivative and by rounding / h; what remains is the gradient's own bound."""
    import gemm_epilogue_bf16_amd as F

    rows = [20, 0, 33]
    t, off, offs = make(rows, 0, 0, 48, 64, True, seed=3)
    d = dbl(t)
    (dx, dW, db) = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], t["b"], "gelu_tanh", t["dy"])
    _, bound = ffn64.grouped_bwd(d["x"], off, d["W"], d["b"], "gelu_tanh", d["dy"])
    g = torch.Generator(device="cuda").manual_seed(5)
    h = 1e-5
    for name, grad, e in (("x", dx, bound[0]), ("W", dW, bound[1]), ("b", db, bound[2])):
        v = torch.randn(d[name].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(s):
            p = dict(d)
            p[name] = d[name] + s * v
            return float((ffn64.grouped(p["x"], off, p["W"], p["b"], "gelu_tanh")[0] * d["dy"]).sum())

        quotient = (loss(h) - loss(-h)) / (2 * h)
        assert abs(quotient - float((grad.double() * v).sum())) <= float((e * v.abs()).sum()) + 1e-4


def test_single_and_many_groups_agree_with_the_dense_call():
    """One group is a Linear; the same weight for every group too, whatever the cuts."""
    import gemm_epilogue_bf16_amd as F

    t, off, offs = make([700], 0, 0, 256, 512, True, seed=1)
    y = F.fmlp_linear(t["x"], t["W"][0], t["b"][0], "silu")
    assert torch.equal(F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], "silu"), y)
    cuts = torch.tensor([0, 3, 3, 259, 400, 700], dtype=torch.int32, device="cuda")
    W, b = t["W"].expand(5, -1, -1).contiguous(), t["b"].expand(5, -1).contiguous()
    assert torch.equal(F.fmlp_grouped_linear(t["x"], cuts, W, b, "silu"), y)


def test_many_groups():
    """the most groups a call takes, most of them with one row or none"""
    import gemm_epilogue_bf16_amd as F

    rows = [(i * 7) % 3 for i in range(1024)]
    t, off, offs = make(rows, 1, 2, 64, 72, True, seed=2)
    d = dbl(t)
    want, bound = ffn64.grouped(d["x"], off, d["W"], d["b"], "gelu_tanh")
    ffn64.check("y", F.fmlp_grouped_linear(t["x"], offs, t["W"], t["b"], "gelu_tanh"), want, bound)
    want, bound = ffn64.grouped_bwd(d["x"], off, d["W"], d["b"], "gelu_tanh", d["dy"])
    got = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], t["b"], "gelu_tanh", t["dy"])
    for n, a, w, e in zip(("dx", "dW", "db"), got, want, bound):
        ffn64.check(n, a, w, e)


def test_offsets_past_32_bits():
    """2^32 output elements and more: the rows at the end"""
    import gemm_epilogue_bf16_amd as F

    K, N, R = 32, 4096, (1 << 20) + 300
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(R, K, generator=g, device="cuda").bfloat16()
    W = (torch.randn(3, N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    off = torch.tensor([0, 100, R - 257, R], dtype=torch.int32, device="cuda")
    y = F.fmlp_grouped_linear(x, off, W, None, "silu")
    for r, e in ((slice(0, 100), 0), (slice(R - 600, R - 257), 1), (slice(R - 257, R), 2)):
        want, bound = ffn64.grouped(x[r].double(), [0, r.stop - r.start], W[e:e + 1].double(), None, "silu")
        ffn64.check(f"group {e}", y[r], want, bound)


def test_infinities_stay_in_their_group():
    import gemm_epilogue_bf16_amd as F

    rows = [40, 30, 50]
    t, off, offs = make(rows, 0, 0, 64, 64, False, seed=4)
    clean = F.fmlp_grouped_linear(t["x"], offs, t["W"])
    cb = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], None, "none", t["dy"])
    for bad in (float("inf"), float("nan")):
        x, dy = t["x"].clone(), t["dy"].clone()
        x[off[1]:off[2]] = bad
        dy[off[1]:off[2]] = bad
        y = F.fmlp_grouped_linear(x, offs, t["W"])
        dx, dW, _ = F.fmlp_grouped_linear_bwd(x, offs, t["W"], None, "none", dy)
        for got, want in ((y, clean), (dx, cb[0])):
            assert torch.equal(got[:off[1]], want[:off[1]]) and torch.equal(got[off[2]:], want[off[2]:])
            assert not bool(torch.isfinite(got[off[1]:off[2]]).any())
        assert torch.equal(dW[0], cb[1][0]) and torch.equal(dW[2], cb[1][2])


def test_offsets_out_of_order_or_range_stay_in_the_buffers():
    """A bad table gives unspecified rows; it reads and writes nothing outside the buffers (guard rows around them keep
    their values), and the groups before the bad entry are right.  The table is clamped on the device before any kernel
    uses it, so nothing out of range is ever addressed."""
    import gemm_epilogue_bf16_amd as F

    t, off, _ = make([40, 40, 40], 0, 0, 64, 64, False, seed=6)
    want = F.fmlp_grouped_linear(t["x"], torch.tensor(off, dtype=torch.int32, device="cuda"), t["W"])
    for table in ([0, 40, 30, 120], [0, 40, 2 ** 31 - 1, 120], [-5, 40, 90, 400], [0, 40, -2 ** 31, 80]):
        big = torch.full((120 + 2 * 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        y = big[64:184]
        offs = torch.tensor(table, dtype=torch.int64).to(torch.int32).cuda()
        F.fmlp_grouped_linear(t["x"], offs, t["W"], out=y)
        dx, dW, _ = F.fmlp_grouped_linear_bwd(t["x"], offs, t["W"], None, "none", t["dy"])
        torch.cuda.synchronize()
        assert bool((big[:64] == 7.0).all()) and bool((big[184:] == 7.0).all())
        assert torch.equal(y[:40], want[:40])


def test_no_rows():
    import gemm_epilogue_bf16_amd as F

    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.randn(3, 40, 64, device="cuda").bfloat16()
    b = torch.zeros(3, 40, device="cuda").bfloat16()
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert F.fmlp_grouped_linear(x, offs, W, b).shape == (0, 40)
    dx, dW, db = F.fmlp_grouped_linear_bwd(x, offs, W, b, "silu", torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"))
    assert dx.shape == (0, 64) and not dW.any() and not db.any()


def test_sizes_from_the_router_under_graph_capture():
    """Offsets made on the device by work of the same graph; every replay against the eager result, with eager work and
    synchronisation in between, on other inputs each time."""
    import gemm_epilogue_bf16_amd as F

    E, K, N, R = 8, 64, 96, 500
    t, _, _ = make([R] + [0] * (E - 1), 0, 0, K, N, True, seed=7)
    ids = torch.empty(R, dtype=torch.int64, device="cuda")
    grid = torch.arange(E + 1, device="cuda")

    def step():
        s, order = torch.sort(ids, stable=True)
        offs = torch.searchsorted(s, grid).to(torch.int32)
        xs = t["x"][order]
        y = F.fmlp_grouped_linear(xs, offs, t["W"], t["b"], "silu")
        return (y,) + F.fmlp_grouped_linear_bwd(xs, offs, t["W"], t["b"], "silu", t["dy"])

    gen = torch.Generator(device="cuda").manual_seed(0)
    ids.copy_(torch.randint(0, E, (R,), generator=gen, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        ids.copy_(torch.randint(0, E if i else 2, (R,), generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    import gemm_epilogue_bf16_amd as F

    a, _, oa = make([300, 200], 0, 0, 256, 512, True, seed=8)
    b, _, ob = make([100, 400], 0, 0, 256, 512, True, seed=9)
    want = [F.fmlp_grouped_linear_bwd(t["x"], o, t["W"], t["b"], "silu", t["dy"]) for t, o in ((a, oa), (b, ob))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, (t, o) in enumerate(((a, oa), (b, ob))):
            with torch.cuda.stream(streams[i]):
                got[i].append(F.fmlp_grouped_linear_bwd(t["x"], o, t["W"], t["b"], "silu", t["dy"]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for x, w in zip(g, want[i]):
                assert torch.equal(x, w)


def test_expert_layer_of_grouped_products_equals_the_fused_one():
    """The route, the gate, up and down products and the combine as separate calls, against fmlp_moe_glu on the same
    routes: both round the hidden values to bf16 once more here (gate and up stored), so they agree to that."""
    import gemm_epilogue_bf16_amd as F

    T, D, H, E, k = 300, 128, 192, 4, 2
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = rnd(T, D).bfloat16()
    Wr = rnd(E, D).bfloat16()
    Wg, Wu = ((rnd(E, H, D) / D ** 0.5).bfloat16() for _ in range(2))
    Wd = (rnd(E, D, H) / H ** 0.5).bfloat16()
    ids, gw = F.fmlp_moe_route(x, Wr, k)
    want = F.fmlp_moe_glu(x, ids, gw, Wg, Wu, Wd, "silu")
    order = torch.argsort(ids.reshape(-1), stable=True)
    offs = torch.searchsorted(ids.reshape(-1)[order].contiguous(), torch.arange(E + 1, dtype=torch.int32, device="cuda")).to(torch.int32)
    xs = x[order // k]
    gate = F.fmlp_grouped_linear(xs, offs, Wg, None, "silu")
    up = F.fmlp_grouped_linear(xs, offs, Wu)
    m = gate * up
    down = F.fmlp_grouped_linear(m, offs, Wd)
    y = torch.zeros(T, D, device="cuda").index_add_(0, order // k, down.float() * gw.reshape(-1)[order][:, None])
    # 64-bit reference; each of gate, up, m, down carries one bf16 rounding (2^-8), so does the fused form's m and y
    d = lambda t: t.double()   # noqa: E731
    ref = torch.zeros(T, D, device="cuda", dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        mm = ffn64.act64(d(xs[r]) @ d(Wg[e]).t(), "silu")[0] * (d(xs[r]) @ d(Wu[e]).t())
        w = d(gw).reshape(-1)[order][r][:, None]
        ref.index_add_(0, (order // k)[r], (mm @ d(Wd[e]).t()) * w)
        mag.index_add_(0, (order // k)[r], (mm.abs() @ d(Wd[e]).abs().t()) * w)
    # three roundings on the way to m (gate, up, their product), one of down and one of y: 5 * 2^-8 of the magnitudes,
    # and the fp32 sums (below 2^-12 of them here) within the slack of 1.2
    ffn64.check("separate", y, ref, 1.2 * 5 * ffn64.BF * mag)
    ffn64.check("fused", want, ref, 1.2 * 2 * ffn64.BF * mag)


def test_refusals():
    import gemm_epilogue_bf16_amd as F

    t, _, offs = make([8, 8], 0, 0, 64, 64, True)
    x, W, b, dy = t["x"], t["W"], t["b"], t["dy"]
    for call, err in ((lambda: F.fmlp_grouped_linear(x.float(), offs, W), TypeError),
                      (lambda: F.fmlp_grouped_linear(x, offs.long(), W), TypeError),
                      (lambda: F.fmlp_grouped_linear(x, offs[:2].contiguous(), W), ValueError),
                      (lambda: F.fmlp_grouped_linear(x, offs.cpu(), W), ValueError),
                      (lambda: F.fmlp_grouped_linear(x.t(), offs, W), ValueError),
                      (lambda: F.fmlp_grouped_linear(x, offs, W[0]), ValueError),
                      (lambda: F.fmlp_grouped_linear(x, offs, W, b[0]), ValueError),
                      (lambda: F.fmlp_grouped_linear(x, offs, W, out=dy[:4]), ValueError),
                      (lambda: F.fmlp_grouped_linear(x, offs, W, b, "tanh"), KeyError),
                      (lambda: F.fmlp_grouped_linear_bwd(x, offs, W, b, "silu", dy,
                                                         workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), F.FmlpError),
                      (lambda: F.fmlp_grouped_linear_bwd(x, offs, W, b, "none", dy[:4]), ValueError),
                      (lambda: F.fmlp_grouped_linear_bwd(x, offs, W, b, "none", dy.float()), TypeError)):
        with pytest.raises(err):
            call()
