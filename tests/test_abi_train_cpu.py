"""The C ABI of the grouped products and of the gated block with an 8-bit
checkpoint on the CPU: sizes, and every refusal before a device is touched."""
import os

import pytest

OK, E_NULL, E_SHAPE, E_ALIGN, E_ARG, E_WS = range(6)
X, W, B, Y, WS, O, Q, S = (0x10000 * i for i in range(1, 9))   # fake, aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import gemm_epilogue_bf16_amd as F

    if not os.path.exists(F.library_path()):
        from gemm_epilogue_bf16_amd.build import build

        build()
    return F.lib()


def _err(L):
    return L.fmlp_last_error().decode()


def grouped(L, x=X, off=O, w=W, b=B, act=1, R=40, K=64, N=72, E=4, y=Y, ws=WS, nb=BIG):
    return L.fmlp_grouped_linear(x, off, w, b, act, R, K, N, E, y, ws, nb, None)


def grouped_bwd(L, x=X, off=O, w=W, b=B, act=1, dy=Y, R=40, K=64, N=72, E=4, dx=Y, dW=Y, db=B, ws=WS, nb=BIG):
    return L.fmlp_grouped_linear_bwd(x, off, w, b, act, dy, R, K, N, E, dx, dW, db, ws, nb, None)


COMMON = [
    (dict(K=60), E_ALIGN, "K=60"), (dict(N=20), E_ALIGN, "N=20"), (dict(K=0), E_SHAPE, "K=0"),
    (dict(N=1 << 22), E_SHAPE, "N=4194304"), (dict(R=-1), E_SHAPE, "R=-1"), (dict(R=1 << 31), E_SHAPE, "R=2147483648"),
    (dict(E=0), E_ARG, "E=0"), (dict(E=1025), E_ARG, "E=1025"), (dict(act=5), E_ARG, "act=5"),
    (dict(x=None), E_NULL, "x is NULL"), (dict(off=None), E_NULL, "group_off is NULL"), (dict(w=None), E_NULL, "W is NULL"),
    (dict(x=X + 2), E_ALIGN, "x is not"), (dict(off=O + 2), E_ALIGN, "group_off is not 4-byte"),
    (dict(b=B + 8), E_ALIGN, "b is not"),
]


LONG = dict(R=200, K=8192, N=1024, E=1)   # few tiles over a long contraction: split, with a workspace


@pytest.mark.parametrize("kw,status,msg", COMMON + [
    (dict(y=None), E_NULL, "y is NULL"), (dict(LONG, ws=None, nb=0), E_WS, "NULL"), (dict(LONG, nb=16), E_WS, "needs"),
    (dict(LONG, ws=WS + 8), E_ALIGN, "workspace"),
])
def test_grouped_validation(L, kw, status, msg):
    assert grouped(L, **kw) == status and msg in _err(L)


@pytest.mark.parametrize("kw,status,msg", COMMON + [
    (dict(dy=None), E_NULL, "dy is NULL"), (dict(dx=None), E_NULL, "dx is NULL"), (dict(dW=None), E_NULL, "dW is NULL"),
    (dict(db=B + 4), E_ALIGN, "db is not"), (dict(ws=None, nb=0), E_WS, "NULL"), (dict(nb=16), E_WS, "needs"),
    (dict(ws=WS + 8), E_ALIGN, "workspace"),
    (dict(R=1 << 20, K=1024), E_SHAPE, "2^30"), (dict(R=1 << 24, N=64), E_SHAPE, "2^30"),
    (dict(K=32768, N=32768), E_SHAPE, "N*K=1073741824"),
])
def test_grouped_bwd_validation(L, kw, status, msg):
    assert grouped_bwd(L, **kw) == status and msg in _err(L)


def test_grouped_no_rows_is_a_noop(L):
    assert grouped(L, x=None, R=0, y=None) == OK
    assert grouped(L, x=None, R=0, y=None, ws=None, nb=0) == OK
    assert grouped(L, x=None, R=0, y=None, w=None) == E_NULL


def test_grouped_sizes(L):
    assert L.fmlp_grouped_linear_workspace_size(40, 64, 72, 4) == 0
    assert L.fmlp_grouped_linear_workspace_size(0, 8192, 1024, 1) == 0
    assert L.fmlp_grouped_linear_workspace_size(*(LONG[k] for k in "RKNE")) == 8192 + 256 * 256 * 256 * 4
    assert L.fmlp_grouped_linear_bwd_workspace_size(40, 64, 72, 4, 0) == 8192
    assert L.fmlp_grouped_linear_bwd_workspace_size(40, 64, 72, 4, 1) == 8192 + 40 * 72 * 2 + 128   # dz
    # 4 groups of one tile each over about 8192 rows: split, a multiple of the gradient's fp32 size
    parts = L.fmlp_grouped_linear_bwd_workspace_size(32768, 64, 72, 4, 0) - 8192
    assert parts % (4 * 64 * 72 * 4) == 0 and 2 <= parts // (4 * 64 * 72 * 4) <= 8
    assert L.fmlp_grouped_linear_bwd_workspace_size(-1, 64, 72, 4, 0) == 0


def ckpt(L, x=X, wg=W, wu=W, wd=W, act=4, M=20, D=64, H=72, y=Y, codes=Q, scales=S, ws=WS, nb=BIG):
    return L.fmlp_glu_ckpt(x, wg, wu, wd, act, M, D, H, y, codes, scales, ws, nb, None)


def ckpt_bwd(L, x=X, wg=W, wu=W, wd=W, act=4, M=20, D=64, H=72, codes=Q, scales=S, dy=Y, dx=Y, dWg=Y, dWu=Y, dWd=Y, ws=WS, nb=BIG):
    return L.fmlp_glu_ckpt_bwd(x, codes, scales, wg, wu, wd, act, dy, M, D, H, dx, dWg, dWu, dWd, ws, nb, None)


BLOCK = [
    (dict(D=60), E_ALIGN, "D=60"), (dict(H=12), E_ALIGN, "H=12"), (dict(D=0), E_SHAPE, "D=0"), (dict(H=1 << 22), E_SHAPE, "H="),
    (dict(M=-1), E_SHAPE, "M=-1"), (dict(act=9), E_ARG, "gate_act=9"), (dict(x=None), E_NULL, "x is NULL"),
    (dict(wg=None), E_NULL, "Wg is NULL"), (dict(wu=None), E_NULL, "Wu is NULL"), (dict(wd=None), E_NULL, "Wd is NULL"),
    (dict(codes=None), E_NULL, "codes is NULL"), (dict(scales=None), E_NULL, "scales is NULL"),
    (dict(codes=Q + 8), E_ALIGN, "codes is not"), (dict(scales=S + 1), E_ALIGN, "scales is not"),
    (dict(ws=None, nb=0), E_WS, "NULL"), (dict(nb=8192), E_WS, "needs"),
]


@pytest.mark.parametrize("kw,status,msg", BLOCK + [(dict(y=None), E_NULL, "y is NULL")])
def test_ckpt_validation(L, kw, status, msg):
    assert ckpt(L, **kw) == status and msg in _err(L)


@pytest.mark.parametrize("kw,status,msg", BLOCK + [
    (dict(dy=None), E_NULL, "dy is NULL"), (dict(dx=None), E_NULL, "dx is NULL"), (dict(dWg=None), E_NULL, "dWg is NULL"),
    (dict(dWu=None), E_NULL, "dWu is NULL"), (dict(dWd=None), E_NULL, "dWd is NULL"),
    (dict(M=1 << 22), E_SHAPE, "2^22"), (dict(H=1 << 21), E_SHAPE, "2H must"),
])
def test_ckpt_bwd_validation(L, kw, status, msg):
    assert ckpt_bwd(L, **kw) == status and msg in _err(L)


def test_ckpt_sizes_and_no_tokens(L):
    assert L.fmlp_glu_ckpt_codes_size(20, 72) == 20 * 144
    assert L.fmlp_glu_ckpt_scales_size(20, 72) == 20 * 2 * 3
    assert L.fmlp_glu_ckpt_workspace_size(20, 64, 72) == 8192 + 3072
    assert L.fmlp_glu_ckpt_bwd_workspace_size(0, 64, 72) == 8192
    assert L.fmlp_glu_ckpt_codes_size(-1, 72) == 0 and L.fmlp_glu_ckpt_workspace_size(1, 0, 72) == 0
    assert ckpt(L, M=0, x=None, y=None, codes=None, scales=None) == OK
    # a checkpoint that is smaller than the recomputing backward's dm, and its workspace too
    assert L.fmlp_glu_ckpt_bwd_workspace_size(4096, 4096, 14336) < L.fmlp_glu_bwd_workspace_size(4096, 4096, 14336)


def w4(L, x=X, q=Q, s=S, z=B, b=B, act=4, M=4, K=256, N=72, g=64, y=Y, ws=None, nb=0):
    return L.fmlp_linear_w4(x, q, s, z, b, act, M, K, N, g, y, ws, nb, None)


def glu_w4(L, x=X, q=Q, s=S, zg=B, zu=B, zd=B, act=4, M=4, D=256, H=128, g=64, y=Y, ws=WS, nb=BIG):
    return L.fmlp_glu_w4(x, q, s, zg, q, s, zu, q, s, zd, act, M, D, H, g, y, ws, nb, None)


FOUR = [
    (dict(M=17), E_ARG, "M=17"), (dict(M=-1), E_SHAPE, "M=-1"), (dict(g=16), E_ARG, "group=16"), (dict(g=0), E_ARG, "group=0"),
    (dict(g=-32), E_ARG, "group=-32"), (dict(act=5), E_ARG, "act=5"), (dict(x=None), E_NULL, "x is NULL"),
    (dict(q=None), E_NULL, "q is NULL"), (dict(s=None), E_NULL, " is NULL"), (dict(y=None), E_NULL, "y is NULL"),
    (dict(q=Q + 8), E_ALIGN, "q is not"), (dict(s=S + 2), E_ALIGN, "is not 16-byte"),
]


@pytest.mark.parametrize("kw,status,msg", FOUR + [
    (dict(K=288), E_ALIGN, "K=288"), (dict(K=0), E_SHAPE, "K=0"), (dict(N=20), E_ALIGN, "N=20"), (dict(N=1 << 22), E_SHAPE, "N="),
    (dict(z=B + 8), E_ALIGN, "zeros is not"), (dict(b=B + 8), E_ALIGN, "b is not"),
    (dict(M=16, K=4096), E_WS, "NULL"), (dict(M=16, K=4096, ws=WS, nb=8192), E_WS, "needs"),
    (dict(M=16, K=4096, ws=WS + 8, nb=BIG), E_ALIGN, "workspace")])
def test_linear_w4_validation(L, kw, status, msg):
    assert w4(L, **kw) == status and msg in _err(L)


@pytest.mark.parametrize("kw,status,msg", FOUR + [
    (dict(D=288), E_ALIGN, "D=288"), (dict(H=96), E_ALIGN, "H=96"), (dict(zg=None), E_ARG, "zg and zu"), (dict(zu=None), E_ARG, "zg and zu"),
    (dict(zd=B + 8), E_ALIGN, "zd is not"), (dict(ws=None, nb=0), E_WS, "NULL"), (dict(nb=8192), E_WS, "needs")])
def test_glu_w4_validation(L, kw, status, msg):
    assert glu_w4(L, **kw) == status and msg in _err(L)


def test_w4_sizes_and_no_tokens(L):
    # up to 64 records (tokens x chunks of 128) are made inside the kernel and need no scratch
    assert L.fmlp_linear_w4_workspace_size(1, 8192, 64, 64) == 0 and L.fmlp_linear_w4_workspace_size(4, 2048, 64, 64) == 0
    # records of 16 tokens: 32 slots of 128 bytes, 32 exponents, 16 sums a group; they fit in LDS together
    assert L.fmlp_linear_w4_workspace_size(16, 4096, 64, 64) == 8192 + 32 * (4096 + 32 + 2 * 64)
    assert L.fmlp_linear_w4_workspace_size(16, 4096, 64, 32) == 8192 + (32 * (4096 + 32 + 4 * 64) + 255) // 256 * 256
    # 64 chunks do not fit in LDS: two slices of 32, and the slices' fp32 sums of 16 x 72
    assert L.fmlp_linear_w4_workspace_size(16, 8192, 72, 64) == 8192 + 64 * (4096 + 32 + 2 * 64) + 2 * 16 * 72 * 4
    assert L.fmlp_linear_w4_workspace_size(0, 4096, 64, 64) == 0 and L.fmlp_linear_w4_workspace_size(4, 4096, 64, 48) == 0
    assert L.fmlp_glu_w4_workspace_size(4, 256, 128, 64) == 8192 + 1024
    assert L.fmlp_glu_w4_workspace_size(0, 256, 128, 64) == 0 and L.fmlp_glu_w4_workspace_size(17, 256, 128, 64) == 0
    # the larger of the layers' scratch: the first's 32 chunks in two slices of 16, with two sums each
    assert L.fmlp_glu_w4_workspace_size(16, 4096, 14336, 64) == 8192 + 16 * 14336 * 2 + 32 * (4096 + 32 + 2 * 64) + 2 * 2 * 16 * 14336 * 4
    assert w4(L, M=0, x=None, y=None) == OK
    assert glu_w4(L, M=0, x=None, y=None, ws=None, nb=0) == OK
    assert w4(L, M=0, x=None, y=None, q=None) == E_NULL
