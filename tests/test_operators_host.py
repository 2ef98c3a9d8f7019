"""Refusals and sizes of the adapter projection and of the experts' row
operators (CPU only: no kernel is launched), and the plain definitions that the
GPU tests use, checked against hand-worked values."""
import ctypes
import os

import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
from operators_ref import combine_grad_ref, combine_ref, gather_ref, lora_ref, sort_ref

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


def lora(lib, x=A, w=A, s=A, a=A, b=A, ids=A, sc=A, y=A, M=4, N=64, K=256, g=128, L=3, R=16, sk=0, ws=A, wsb=1 << 30):
    return lib.w4a16_gemm_lora(x, w, s, a, b, ids, sc, y, M, N, K, g, L, R, sk, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE),
    (dict(K=100), ERR_GROUP), (dict(g=64), ERR_GROUP),
    (dict(L=0), ERR_SHAPE), (dict(L=-1), ERR_SHAPE),
    (dict(R=0), ERR_SHAPE), (dict(R=4), ERR_SHAPE), (dict(R=12), ERR_SHAPE), (dict(R=136), ERR_SHAPE),
    (dict(R=-8), ERR_SHAPE),
    (dict(M=1, N=1 << 24, K=128, R=128), ERR_SHAPE),        # one adapter's B of 4 GiB
    (dict(sk=3), ERR_SPLIT), (dict(sk=-1), ERR_SPLIT),
    (dict(x=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(a=None), ERR_NULL),
    (dict(b=None), ERR_NULL), (dict(ids=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(x=MIS), ERR_ALIGN), (dict(w=MIS), ERR_ALIGN), (dict(s=MIS), ERR_ALIGN), (dict(a=MIS), ERR_ALIGN),
    (dict(b=MIS), ERR_ALIGN), (dict(y=MIS), ERR_ALIGN), (dict(ids=MIS2), ERR_ALIGN), (dict(sc=MIS2), ERR_ALIGN),
    (dict(ws=MIS), ERR_ALIGN), (dict(ws=None), ERR_WS), (dict(wsb=0), ERR_WS),
    (dict(M=1 << 16, N=1 << 15, K=128, sk=2), ERR_SHAPE),   # partials of 4 GiB or more
    (dict(M=0), OK), (dict(M=0, x=None, a=None, ids=None, y=None, ws=None, wsb=0), OK),
])
def test_lora_refusals(lib, kw, want):
    assert lora(lib, **kw) == want


@pytest.mark.parametrize("M,N,K,g,L,R,sk", [(1, 64, 256, 128, 3, 16, 0), (16, 512, 1024, 128, 3, 16, 2),
                                            (40, 512, 1024, 128, 3, 8, 0), (100, 8448, 256, 128, 2, 128, 0),
                                            (1322, 19456, 2560, 128, 4, 64, 0), (64, 512, 256, 32, 3, 16, 4)])
def test_lora_workspace_is_required_in_full(lib, M, N, K, g, L, R, sk):
    need = w4.w4a16_gemm_lora_workspace_bytes(M, N, K, L, R, sk, g)
    assert need >= M * R * 4
    assert need >= w4.w4a16_gemm_workspace_bytes(M, N, K, sk, group_size=g) or M <= 48
    assert lora(lib, M=M, N=N, K=K, g=g, L=L, R=R, sk=sk, wsb=need - 1) == ERR_WS


def test_lora_workspace_of_invalid_sizes_is_zero():
    if not os.path.exists(w4.LIB_PATH):
        pytest.skip("libw4a16.so not built")
    f = w4.w4a16_gemm_lora_workspace_bytes
    assert f(0, 64, 256, 3, 16) == 0 and f(4, 64, 100, 3, 16) == 0 and f(4, 64, 256, 3, 12) == 0
    assert f(4, 64, 256, 0, 16) == 0 and f(4, 64, 256, 3, 16, 3) == 0


def sort(lib, ids=A, order=A, pos=A, ms=A, T=8192, k=2, G=8, ws=A, wsb=1 << 30):
    return lib.w4a16_expert_sort(ids, order, pos, ms, T, k, G, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ERR_SHAPE), (dict(k=0), ERR_SHAPE), (dict(k=-1), ERR_SHAPE), (dict(G=0), ERR_SHAPE),
    (dict(G=4097), ERR_SHAPE), (dict(G=-1), ERR_SHAPE), (dict(T=1 << 30, k=2), ERR_SHAPE),
    (dict(ids=None), ERR_NULL), (dict(order=None), ERR_NULL), (dict(pos=None), ERR_NULL), (dict(ms=None), ERR_NULL),
    (dict(T=0, ms=None), ERR_NULL),
    (dict(ids=MIS2), ERR_ALIGN), (dict(order=MIS2), ERR_ALIGN), (dict(pos=MIS2), ERR_ALIGN),
    (dict(ms=MIS2), ERR_ALIGN), (dict(ws=MIS), ERR_ALIGN), (dict(ws=None), ERR_WS), (dict(wsb=0), ERR_WS),
])
def test_sort_refusals(lib, kw, want):
    assert sort(lib, **kw) == want


def test_sort_workspace(lib):
    f = w4.w4a16_expert_sort_workspace_bytes
    assert f(0, 2, 8) == 0 and f(4, 0, 8) == 0 and f(4, 2, 0) == 0 and f(4, 2, 4097) == 0 and f(1 << 30, 2, 8) == 0
    for T, k, G in ((1, 1, 1), (16, 4, 8), (2048, 1, 4096), (256, 8, 128)):   # one kernel
        assert f(T, k, G) == 0
    for T, k, G in ((2049, 1, 1), (8193, 1, 2048), (65536, 8, 128), (1 << 20, 8, 4096), (1 << 28, 7, 300)):
        assert 0 < f(T, k, G) < 1 << 30
        assert sort(lib, T=T, k=k, G=G, wsb=f(T, k, G) - 1) == ERR_WS


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ERR_SHAPE), (dict(k=0), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE), (dict(width=0), ERR_SHAPE),
    (dict(width=1 << 31), ERR_SHAPE), (dict(rows=1 << 31), ERR_SHAPE), (dict(T=1 << 30, k=2), ERR_SHAPE),
    (dict(pos=None), ERR_NULL), (dict(pos=MIS2), ERR_ALIGN),
    (dict(src=None), ERR_NULL), (dict(dst=None), ERR_NULL), (dict(src=MIS), ERR_ALIGN), (dict(dst=MIS), ERR_ALIGN),
    (dict(T=0), OK), (dict(T=0, src=None, dst=None, pos=None), OK),
])
def test_row_call_refusals(lib, kw, want):
    d = dict(src=A, pos=A, dst=A, T=4, k=2, rows=8, width=16)
    d.update(kw)
    tail = (d["T"], d["k"], d["rows"], d["width"], None)
    assert lib.w4a16_expert_gather(d["src"], d["pos"], d["dst"], *tail) == want
    assert lib.w4a16_expert_gather_grad(d["src"], d["pos"], d["dst"], *tail) == want
    assert lib.w4a16_expert_combine(d["src"], d["pos"], A, d["dst"], *tail) == want


@pytest.mark.parametrize("i", range(6))
def test_combine_grad_refusals(lib, i):
    for bad, want in ((None, ERR_NULL), (P(0x10001), ERR_ALIGN)):
        p = [A] * 6
        p[i] = bad
        assert lib.w4a16_expert_combine_grad(*p, 4, 2, 8, 16, None) == want
    assert lib.w4a16_expert_combine(A, A, MIS2, A, 4, 2, 8, 16, None) == ERR_ALIGN   # weights


def test_binding_refusals():
    """Shapes, types and places that the Python calls refuse before the library is reached."""
    t = torch.zeros
    with pytest.raises(TypeError):
        w4.w4a16_expert_sort(t((4, 2), dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        w4.w4a16_expert_sort(t((4, 2), dtype=torch.int32), 8)                 # not on the device
    with pytest.raises(TypeError):
        w4.w4a16_expert_gather(t((4, 8)), t((4, 2), dtype=torch.int32))
    with pytest.raises(TypeError):
        w4.w4a16_expert_combine(t((8, 8)), t((4, 2), dtype=torch.int32))
    with pytest.raises(TypeError):
        w4.w4a16_gemm_lora(t((4, 128)), t((8, 64), dtype=torch.uint8), t((8, 1)), t((1, 8, 128)), t((1, 8, 8)),
                           t((4,), dtype=torch.int32))


# ------------------------------------------------------------------ the definitions themselves

def test_sort_definition():
    ids = np.array([[2, 0], [5, 2], [-1, 0]], dtype=np.int32)                  # 5 and -1: dropped at G = 3
    order, pos, sizes = sort_ref(ids, 3)
    assert sizes.tolist() == [2, 0, 2]
    assert order.tolist() == [1, 5, 0, 3, 2, 4]
    assert pos.tolist() == [[2, 0], [-1, 3], [-1, 1]]


def test_row_definitions():
    pos = np.array([[1, 0], [-1, 2]])
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    assert gather_ref(x, pos, np.full((4, 2), 9.0)).tolist() == [[1, 2], [1, 2], [3, 4], [9, 9]]
    z = np.array([[1.0, -1.0], [2.0, 5.0], [3.0, 0.5], [np.nan, np.nan]])
    w = np.array([[0.5, 2.0], [7.0, 3.0]])
    assert combine_ref(z, pos, w)[0].tolist() == [[3.0, 0.5], [9.0, 1.5]]
    assert combine_ref(z, pos, None)[0].tolist() == [[3.0, 4.0], [3.0, 0.5]]
    dz, _, dw, _ = combine_grad_ref(x, z, pos, w, np.zeros((4, 2)))
    assert dz.tolist() == [[2, 4], [0.5, 1], [9, 12], [0, 0]]
    assert dw.tolist() == [[12.0, -1.0], [0.0, 11.0]]


def test_lora_definition():
    """One row by hand: the projection 1 * 2 (10 - 8) and the adapter 3 * (1 * 4) * 5."""
    x = np.zeros((2, 128))
    x[:, 7] = 1.0
    q = np.full((1, 128), 8.0)
    q[0, 7] = 10.0
    a = np.zeros((1, 8, 128))
    a[0, 2, 7] = 4.0
    b = np.zeros((1, 1, 8))
    b[0, 0, 2] = 5.0
    y, bound = lora_ref(x, q, np.full((1, 1), 2.0), a, b, np.array([0, -1]), np.array([3.0]), 128)
    assert y.tolist() == [[64.0], [4.0]]
    assert np.all(bound > 0)
