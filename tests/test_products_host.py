"""Refusals and sizes of the 8-bit products, their quantisation and the input
gradients (CPU only: no kernel is launched), and the plain definitions that the
GPU tests use, checked against hand-worked values."""
import ctypes
import os

import pytest
import torch

import bf16_activation_quantized_amd as w4
from products_ref import E4M3, e4m3_of, fp8_values, grouped_ref, int4_values, quantize_ref

OK, ERR_NULL, ERR_SHAPE, ERR_GROUP, ERR_SPLIT, ERR_WS, ERR_ALIGN = 0, 1, 2, 3, 4, 5, 6


def P(v):
    return ctypes.c_void_p(v)


A, MIS, MIS2 = P(0x10000), P(0x10004), P(0x10002)


@pytest.fixture()
def lib():
    # fake device pointers that validation must reject: only where no GPU could run them
    if torch.cuda.is_available():
        pytest.skip("host-only checks: a GPU is visible")
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")
    return w4._lib()


def quantize(lib, x=A, q=A, s=A, M=4, K=256, rows=1):
    return lib.w4a16_fp8_quantize(x, q, s, M, K, rows, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=64), ERR_SHAPE), (dict(K=200), ERR_SHAPE),
    (dict(M=1 << 31), ERR_SHAPE), (dict(K=1 << 31), ERR_SHAPE), (dict(M=1 << 30, K=128), ERR_SHAPE),
    (dict(rows=0), ERR_SHAPE), (dict(rows=2), ERR_SHAPE), (dict(rows=-128), ERR_SHAPE),
    (dict(x=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(s=None), ERR_NULL),
    (dict(x=MIS), ERR_ALIGN), (dict(q=MIS), ERR_ALIGN), (dict(s=MIS2), ERR_ALIGN),
    (dict(M=0, x=None, q=None, s=None), OK),
])
def test_quantize_refusals(lib, kw, want):
    assert quantize(lib, **kw) == want


def gemm(lib, x=A, xs=A, w=A, ws=A, y=A, M=4, N=64, K=256, wk=None, wkb=0):
    return lib.w4a16_fp8_gemm(x, xs, w, ws, y, M, N, K, wk, wkb, None)


def grouped(lib, x=A, xs=A, w=A, ws=A, ms=A, y=A, G=3, M=4, N=64, K=256):
    return lib.w4a16_fp8_gemm_grouped(x, xs, w, ws, ms, y, G, M, N, K, None)


def grad(lib, x=A, xs=A, w=A, ws=A, ms=None, y=A, G=1, M=4, N=128, K=256, wk=None, wkb=0):
    return lib.w4a16_fp8_gemm_grad(x, xs, w, ws, ms, y, G, M, N, K, wk, wkb, None)


COMMON = [
    (dict(M=-1), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=192), ERR_SHAPE),
    (dict(M=1 << 31), ERR_SHAPE), (dict(N=1 << 31), ERR_SHAPE), (dict(K=1 << 31), ERR_SHAPE),
    (dict(N=1 << 20, K=1 << 13), ERR_SHAPE),                 # one W of 4 GiB and more
    (dict(M=(1 << 24) + 1, N=128, K=128), ERR_SHAPE),        # rows
    (dict(M=256, N=128, K=1 << 23), ERR_SHAPE),              # 256 rows of X or dX
    (dict(M=256, N=1 << 23, K=128), ERR_SHAPE),              # of Y or dY
    (dict(G=0), ERR_SHAPE), (dict(G=-1), ERR_SHAPE),
    (dict(x=None), ERR_NULL), (dict(xs=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(y=None), ERR_NULL),
    (dict(x=MIS), ERR_ALIGN), (dict(w=MIS), ERR_ALIGN), (dict(y=MIS), ERR_ALIGN), (dict(xs=MIS2), ERR_ALIGN),
    (dict(ws=MIS2), ERR_ALIGN),
    (dict(M=0, x=None, xs=None, w=None, ws=None, y=None), OK),
]


@pytest.mark.parametrize("kw,want", [c for c in COMMON if "G" not in c[0]])
def test_gemm_refusals(lib, kw, want):
    assert gemm(lib, **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [(dict(ms=None), ERR_NULL), (dict(ms=MIS2), ERR_ALIGN)])
def test_grouped_refusals(lib, kw, want):
    assert grouped(lib, **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [(dict(N=64), ERR_SHAPE), (dict(N=200), ERR_SHAPE), (dict(G=2), ERR_SHAPE),
                                              (dict(G=2, ms=MIS2), ERR_ALIGN)])
def test_grad_refusals(lib, kw, want):
    assert grad(lib, **kw) == want


def w4_grad(lib, dy=A, w=A, s=A, ms=None, dx=A, G=1, M=4, N=64, K=256, g=128, ws=A, wsb=1 << 40):
    return lib.w4a16_gemm_grad(dy, w, s, ms, dx, G, M, N, K, g, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(N=4), ERR_SHAPE),
    (dict(N=63), ERR_SHAPE), (dict(N=100), ERR_SHAPE), (dict(K=192), ERR_GROUP), (dict(g=64), ERR_GROUP),
    (dict(M=1 << 31), ERR_SHAPE), (dict(N=1 << 21, K=1 << 12), ERR_SHAPE), (dict(M=(1 << 24) + 1), ERR_SHAPE),
    (dict(M=256, N=1 << 23, K=128), ERR_SHAPE), (dict(M=256, N=64, K=1 << 23), ERR_SHAPE),
    (dict(G=1 << 30, ms=A, N=1 << 17, K=1 << 16), ERR_SHAPE),   # the weights of all groups
    (dict(G=0), ERR_SHAPE), (dict(G=2), ERR_SHAPE), (dict(G=2, ms=MIS2), ERR_ALIGN),
    (dict(dy=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(dx=None), ERR_NULL),
    (dict(dy=MIS), ERR_ALIGN), (dict(w=MIS), ERR_ALIGN), (dict(s=MIS), ERR_ALIGN), (dict(dx=MIS), ERR_ALIGN),
    (dict(ws=MIS), ERR_ALIGN), (dict(ws=None), ERR_WS), (dict(wsb=0), ERR_WS),
    (dict(M=0, dy=None, w=None, s=None, dx=None, ws=None, wsb=0), OK),
])
def test_w4_grad_refusals(lib, kw, want):
    assert w4_grad(lib, **kw) == want


@pytest.mark.parametrize("G,M,N,K,g", [(1, 1, 8, 128, 128), (1, 300, 1000, 512, 32), (1, 1322, 19456, 2560, 128),
                                       (8, 2048, 2048, 4096, 32)])
def test_w4_grad_workspace_is_required_in_full(lib, G, M, N, K, g):
    need = w4.w4a16_gemm_grad_workspace_bytes(G, M, N, K, g)
    npad = -(-N // 128) * 128
    assert need >= 2 * M * npad + 2 * G * npad * (K // g)
    assert w4_grad(lib, ms=A if G > 1 else None, G=G, M=M, N=N, K=K, g=g, wsb=need - 1) == ERR_WS


@pytest.mark.parametrize("f,call", [(w4.w4a16_fp8_gemm_workspace_bytes, gemm),
                                    (w4.w4a16_fp8_gemm_grad_workspace_bytes, grad)])
def test_partials_are_required_in_full(lib, f, call):
    split = [(M, N, K) for M in (40, 100, 300) for N, K in ((256, 8192), (2560, 9728), (8192, 256)) if f(M, N, K)]
    assert split, "no shape splits its contraction"
    for M, N, K in split:
        need = f(M, N, K)
        out = K if call is grad else N
        assert need % (256) == 0 and need >= 2 * M * out * 4
        assert call(lib, M=M, N=N, K=K) == ERR_WS                       # NULL
        assert call(lib, M=M, N=N, K=K, wk=A, wkb=2 * M * out * 4 - 1) == ERR_WS
        assert call(lib, M=M, N=N, K=K, wk=MIS, wkb=need) == ERR_ALIGN


def test_workspaces_of_invalid_sizes_are_zero():
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")
    for f in (w4.w4a16_fp8_gemm_workspace_bytes, w4.w4a16_fp8_gemm_grad_workspace_bytes):
        assert f(0, 256, 8192) == 0 and f(100, 256, 100) == 0 and f(-1, 256, 256) == 0
    g = w4.w4a16_gemm_grad_workspace_bytes
    assert g(1, 0, 64, 256) == 0 and g(1, 4, 63, 256) == 0 and g(0, 4, 64, 256) == 0 and g(1, 4, 64, 256, 64) == 0


def test_forced_choices_are_checked(lib):
    f = lib.w4a16_fp8_gemm_ex

    def fp8(gr=0, ms=None, G=1, M=300, N=256, K=1024, bm=0, sk=0, wk=None, wkb=0):
        return f(gr, A, A, A, A, ms, A, G, M, N, K, bm, sk, wk, wkb, None)
    assert fp8(bm=48) == ERR_SHAPE and fp8(bm=-1) == ERR_SHAPE and fp8(gr=1, bm=16) == ERR_SHAPE
    assert fp8(bm=64, sk=17) == ERR_SPLIT and fp8(bm=16, sk=2) == ERR_SPLIT and fp8(ms=A, bm=64, sk=2) == ERR_SPLIT
    assert fp8(bm=64, sk=2) == ERR_WS
    g = lib.w4a16_gemm_grad_ex

    def gr4(ms=None, G=1, bm=0, sk=0, wsb=1 << 40):
        return g(A, A, A, ms, A, G, 300, 256, 1024, 128, bm, sk, A, wsb, None)
    assert gr4(bm=48) == ERR_SHAPE and gr4(sk=17) == ERR_SPLIT and gr4(ms=A, sk=2, wsb=2 * 300 * 1024 * 4) == ERR_WS
    assert gr4(bm=64, sk=4, wsb=4 * 300 * 1024 * 4) == ERR_WS


# ------------------------------------------------------------------ the definitions

def test_e4m3_rounding():
    v = torch.tensor([0.0, 448.0, -447.9, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875],
                     dtype=torch.float64)
    want = [0.0, 448.0, -448.0, 16.0, 20.0, 2.0 ** -9, 0.0, 2.0 ** -8, 1.0, 1.25]   # ties to even
    assert e4m3_of(v).tolist() == want
    every = torch.arange(256, dtype=torch.uint8).view(E4M3).float()
    every = every[~every.isnan()].double()
    assert torch.equal(e4m3_of(every), every)


def test_quantize_definition():
    x = torch.zeros(2, 256)
    x[0, 3], x[0, 5], x[1, 200] = 896.0, -2.0, 7.0
    q, s = quantize_ref(x, 1)
    assert s.tolist() == [[2.0, 2.0 ** -100 / 448], [2.0 ** -100 / 448, 7.0 / 448]]
    assert q[0, 3] == 448 and q[0, 5] == -1 and q[1, 200] == 448
    q, s = quantize_ref(x, 128)
    assert s.tolist() == [[2.0, 7.0 / 448]] and q[0, 5] == -1


def test_value_definitions():
    q = torch.ones(3, 256).to(E4M3)
    s = torch.tensor([[2.0, 3.0]])
    v = fp8_values(q, s, 128)
    assert v[2, 127] == 2 and v[0, 128] == 3
    w = torch.tensor([[0x80, 0xF0] + [0x88] * 62], dtype=torch.uint8)
    i = int4_values(w, torch.tensor([[0.5]]), 128)
    assert i[0, :5].tolist() == [-4.0, 0.0, -4.0, 3.5, 0.0]


def test_grouped_definition():
    x = torch.arange(8, dtype=torch.float64).reshape(4, 2)
    ws = [torch.eye(2, dtype=torch.float64), -torch.eye(2, dtype=torch.float64), 2 * torch.eye(2, dtype=torch.float64)]
    y, a = grouped_ref(x, ws, [1, 0, 2], 2)
    assert y[:3].tolist() == [[0, 1], [4, 6], [8, 10]] and y[3].isnan().all() and a[1].tolist() == [4, 6]
