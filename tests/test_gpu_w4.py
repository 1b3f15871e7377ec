"""Decode with 4-bit weights and group scales on the GPU, against the plain
64-bit form with the bounds of ffn64.py."""
import pytest
import torch

import ffn64

pytestmark = pytest.mark.gpu


def weight(g, N, K, G, zeros):
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(N, K // G, generator=g, device="cuda") + 0.5).mul_(0.25 / K ** 0.5).bfloat16()
    z = (torch.rand(N, K // G, generator=g, device="cuda") * 15).bfloat16() if zeros else None
    return q, s, z


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# K over group and chunk borders, one and many batches, odd numbers of groups; N around tiles
LINEAR = [(1, 32, 8, 32), (1, 128, 16, 128), (2, 96, 24, 32), (3, 192, 40, 64), (16, 384, 72, 128), (5, 160, 16, 32),
          (1, 4096, 48, 128), (4, 4128, 32, 32), (16, 4096, 80, 64), (7, 5248, 40, 128), (16, 2080, 56, 32),
          (1, 28672, 24, 128), (9, 14336, 40, 64), (16, 8192, 264, 32), (13, 8256, 136, 64), (1, 32768, 8, 32)]


@pytest.mark.parametrize("M,K,N,G", LINEAR)
@pytest.mark.parametrize("zeros", [False, True])
def test_linear(M, K, N, G, zeros):
    import gemm_epilogue_bf16_amd as F

    g = gen(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = weight(g, N, K, G, zeros)
    b = torch.randn(N, generator=g, device="cuda").bfloat16()
    z, e = ffn64.w4_linear(x.double(), None, *w)
    for act in ffn64.ACTS:
        bias = b if act in ("gelu_erf", "silu") else None
        zz = z if bias is None else z + b.double()
        ez = e if bias is None else e + ffn64.F32 * zz.abs()
        want = ffn64.act64(zz, act)[0]
        ffn64.check(act, F.fmlp_linear_w4(x, *w, bias, act), want, ffn64.rounded(want, ffn64.act_err(zz, ez, act)[0]))


@pytest.mark.parametrize("M,K,N,G", [(1, 262144, 24, 64), (16, 65536, 40, 32), (9, 1048576, 8, 128)])
def test_long_rows_in_many_slices(M, K, N, G):
    import gemm_epilogue_bf16_amd as F

    g = gen(K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = weight(g, N, K, G, True)
    want, e = ffn64.w4_linear(x.double(), None, *w)
    ffn64.check("y", F.fmlp_linear_w4(x, *w), want, ffn64.rounded(want, e))


@pytest.mark.parametrize("M,D,H,G", [(1, 32, 64, 32), (2, 96, 160, 32), (16, 128, 256, 128), (5, 320, 448, 64),
                                     (1, 4096, 1024, 128), (16, 4096, 1152, 128), (3, 1056, 4128, 32), (16, 2112, 4160, 64)])
@pytest.mark.parametrize("zeros", [(False, False), (True, True), (True, False), (False, True)])
def test_gated_block(M, D, H, G, zeros):
    import gemm_epilogue_bf16_amd as F

    g = gen(D + H)
    x = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    wg, wu, wd = weight(g, H, D, G, zeros[0]), weight(g, H, D, G, zeros[0]), weight(g, D, H, G, zeros[1])
    for act in ffn64.ACTS:
        want, bound = ffn64.w4_glu(x.double(), wg, wu, wd, act)
        y = F.fmlp_glu_w4(x, *wg, *wu, *wd, act)
        ffn64.check(act, y, want, bound)
        assert torch.equal(y, F.fmlp_glu_w4(x, *wg, *wu, *wd, act))   # the same bits again


@pytest.mark.parametrize("M", range(1, 17))
def test_every_token_count(M):
    import gemm_epilogue_bf16_amd as F

    g = gen(M)
    for K in (1024, 2592, 4096):
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        w = weight(g, 40, K, 32, M % 2 == 0)
        want, e = ffn64.w4_linear(x.double(), None, *w)
        out = torch.full((18, 40), 7.0, dtype=torch.bfloat16, device="cuda")
        F.fmlp_linear_w4(x, *w, out=out[1:1 + M])
        ffn64.check(f"K={K}", out[1:1 + M], want, ffn64.rounded(want, e))
        assert bool((out[0] == 7).all()) and bool((out[1 + M:] == 7).all())


@pytest.mark.parametrize("G", [32, 64, 128])
def test_every_code_exactly(G):
    """One token with a single 1: y is one column of W, and s (code - z) of small integers is exact."""
    import gemm_epilogue_bf16_amd as F

    K, N = 256, 16
    codes = (torch.arange(N).view(-1, 1) + torch.arange(K).view(1, -1)) % 16
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8).cuda()
    s = torch.full((N, K // G), 0.5, dtype=torch.bfloat16, device="cuda")
    for z in (None, torch.arange(K // G, device="cuda").bfloat16().repeat(N, 1)):
        W = 0.5 * (codes - (8 if z is None else z.cpu().long().repeat_interleave(G, 1))).double()
        for k0 in range(0, K, 16):
            y = F.fmlp_linear_w4(torch.eye(K, device="cuda").bfloat16()[k0:k0 + 16].contiguous(), q, s, z)
            assert torch.equal(y.double().cpu(), W[:, k0:k0 + 16].t())


def test_not_finite_tokens_stay_apart():
    import gemm_epilogue_bf16_amd as F

    g = gen(3)
    for K in (512, 8192):   # staged activations, and read beside the weights
        x = torch.randn(8, K, generator=g, device="cuda").bfloat16()
        w = weight(g, 40, K, 64, True)
        clean = F.fmlp_linear_w4(x, *w)
        x[2, 17] = float("inf")
        x[5, K - 1] = float("nan")
        y = F.fmlp_linear_w4(x, *w)
        keep = [0, 1, 3, 4, 6, 7]
        assert torch.equal(y[keep], clean[keep])
        assert not bool(torch.isfinite(y[[2, 5]]).any())


def test_large_values_and_zero_scales():
    import gemm_epilogue_bf16_amd as F

    g = gen(4)
    x = (torch.randn(3, 256, generator=g, device="cuda") * 1e15).bfloat16()
    q, s, z = weight(g, 24, 256, 32, True)
    s[:, 1] = 0
    s[3] *= 2.0 ** 40
    s[4] *= -1
    want, e = ffn64.w4_linear(x.double(), None, q, s, z)
    ffn64.check("y", F.fmlp_linear_w4(x, q, s, z), want, ffn64.rounded(want, e))


def test_offsets_and_leading_dims():
    """views into larger buffers, 16-byte aligned; x with leading dimensions"""
    import gemm_epilogue_bf16_amd as F

    g = gen(5)
    xs = torch.randn(3, 4, 128, generator=g, device="cuda").bfloat16()
    q, s, z = weight(g, 64, 128, 32, True)
    want = F.fmlp_linear_w4(xs[1], q[16:48].contiguous(), s[16:48].contiguous(), z[16:48].contiguous())
    assert torch.equal(F.fmlp_linear_w4(xs[1].view(2, 2, 128), q[16:48], s[16:48], z[16:48]).view(4, 32), want)


def test_no_tokens():
    import gemm_epilogue_bf16_amd as F

    g = gen(6)
    w = weight(g, 64, 64, 32, False)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert F.fmlp_linear_w4(x, *w).shape == (0, 64)
    assert F.fmlp_glu_w4(x, *w, *w, *w).shape == (0, 64)


def test_captured_on_two_streams():
    """Two captured graphs replayed at once on two streams, eager work in between; every replay against the eager result."""
    import gemm_epilogue_bf16_amd as F

    g = gen(7)
    G, D, H = 64, 256, 512
    w = [weight(g, H, D, G, True), weight(g, H, D, G, True), weight(g, D, H, G, True)]
    xs = [torch.randn(m, D, generator=g, device="cuda").bfloat16() for m in (1, 9)]

    def step(x):
        return F.fmlp_glu_w4(F.fmlp_glu_w4(x, *w[0], *w[1], *w[2]), *w[0], *w[1], *w[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in xs:
            step(x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(x))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            assert torch.equal(o.clone(), step(x)), i


def test_trained_block_served_in_four_bits():
    """A training step of the block with its checkpoint, then the updated weights rounded to 4 bits by group and served:
    the decode output is the gated block of those weights."""
    import gemm_epilogue_bf16_amd as F

    g = gen(8)
    D, H, G = 128, 256, 32
    p = [(torch.randn(*s, generator=g, device="cuda") / s[1] ** 0.5).bfloat16() for s in ((H, D), (H, D), (D, H))]
    x, dy = (torch.randn(64, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    _, codes, scales = F.fmlp_glu_ckpt(x, *p, "silu")
    _, *grads = F.fmlp_glu_ckpt_bwd(x, codes, scales, *p, "silu", dy)
    p = [(w.float() - 0.01 * d.float()).bfloat16() for w, d in zip(p, grads)]
    packed = []
    for w in p:
        v = w.float().view(w.shape[0], -1, G)
        lo, hi = v.amin(-1), v.amax(-1)
        s = ((hi - lo) / 15).bfloat16()
        z = (-lo / s.float()).round().bfloat16()
        c = (v / s.float()[..., None] + z.float()[..., None]).round().clamp(0, 15).to(torch.uint8).view(w.shape)
        packed += [(c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), s, z]
    t = torch.randn(4, D, generator=g, device="cuda").bfloat16()
    want, bound = ffn64.w4_glu(t.double(), packed[:3], packed[3:6], packed[6:], "silu")
    ffn64.check("served", F.fmlp_glu_w4(t, *packed, "silu"), want, bound)


def test_refusals():
    import gemm_epilogue_bf16_amd as F

    g = gen(9)
    x = torch.randn(4, 64, generator=g, device="cuda").bfloat16()
    q, s, z = weight(g, 64, 64, 32, True)
    for call, err in ((lambda: F.fmlp_linear_w4(x.float(), q, s), TypeError),
                      (lambda: F.fmlp_linear_w4(x, q.to(torch.int8), s), TypeError),
                      (lambda: F.fmlp_linear_w4(x, q, s.float()), TypeError),
                      (lambda: F.fmlp_linear_w4(x, q[:, :16].contiguous(), s), ValueError),
                      (lambda: F.fmlp_linear_w4(x, q, s[:32]), ValueError),
                      (lambda: F.fmlp_linear_w4(x, q, s, z[:, :1].contiguous()), ValueError),
                      (lambda: F.fmlp_linear_w4(x, q, s.cpu()), ValueError),
                      (lambda: F.fmlp_linear_w4(x, q, s, None, z[0]), ValueError),
                      (lambda: F.fmlp_linear_w4(x, q, torch.cat((s, s), 1)), F.FmlpError),      # group 16
                      (lambda: F.fmlp_linear_w4(x, q, s[:, :1].contiguous()), None),             # group 64 is one
                      (lambda: F.fmlp_linear_w4(x.repeat(5, 1), q, s), F.FmlpError),             # 20 tokens
                      (lambda: F.fmlp_linear_w4(x, q, s, act="swish"), KeyError),
                      (lambda: F.fmlp_glu_w4(x, q, s, z, q, s, None, q, s, z), F.FmlpError),
                      (lambda: F.fmlp_glu_w4(x, q, s, z, q, s[:, :1].contiguous(), z[:, :1].contiguous(), q, s, z), ValueError)):
        if err is None:
            call()
            continue
        with pytest.raises(err):
            call()
