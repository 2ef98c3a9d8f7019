"""The 8-bit products and the input gradients at the ends of their ranges, on the
GPU: fewer rows than a tile, so wide that the offsets of a full tile's rows pass
2^32 bytes. Whole numbers, so that every order of summation gives the same bits."""
import pytest
import torch

import bf16_activation_quantized_amd as w4
from products_ref import E4M3

pytestmark = pytest.mark.gpu
DEV = "cuda"


def whole(*shape):
    return torch.randint(-4, 5, shape, device=DEV, dtype=torch.int8)


def whole8(*shape):
    """The same as e4m3, a part at a time."""
    v = whole(*shape)
    table = torch.arange(-4, 5, device=DEV).float().to(E4M3).view(torch.uint8)
    flat = v.view(-1)
    out = torch.empty(flat.shape, dtype=torch.uint8, device=DEV)
    for i in range(0, flat.numel(), 1 << 26):
        out[i:i + (1 << 26)] = table[flat[i:i + (1 << 26)].long() + 4]
    return out.view(E4M3).view(shape)


@pytest.mark.parametrize("M,N", [(65, 33038208), (130, 16500000)])
def test_product_of_wide_rows(M, N):
    """Y against columns of its own."""
    K = 128
    x, xs = whole8(M, K), torch.ones(M, 1, device=DEV)
    w, ws = whole8(N, K), torch.ones(-(-N // 128), 1, device=DEV)
    y = w4.w4a16_fp8_gemm(x, xs, w, ws)
    step = 1 << 20
    for n in range(0, N, step):
        n1 = min(N, n + step)
        assert torch.equal(y[:, n:n1], w4.w4a16_fp8_gemm(x, xs, w[n:n1], ws[n // 128:-(-n1 // 128)])), n


def test_product_of_wide_rows_by_expert():
    M, N, K, G = 70, 30000000, 128, 2
    x, xs = whole8(M, K), torch.ones(M, 1, device=DEV)
    w, ws = whole8(G, N, K), torch.ones(G, -(-N // 128), 1, device=DEV)
    y = w4.w4a16_fp8_gemm_grouped(x, xs, w, ws, torch.tensor([40, 28], dtype=torch.int32, device=DEV),
                                  y=torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV))
    step = 1 << 20
    for e, r in ((0, slice(0, 40)), (1, slice(40, 68))):
        for n in range(0, N, step):
            n1 = min(N, n + step)
            want = w4.w4a16_fp8_gemm(x[r], xs[r], w[e, n:n1], ws[e, n // 128:-(-n1 // 128)])
            assert torch.equal(y[r, n:n1], want), (e, n)
    assert (y[68:] == 7).all()


def columns(full, part, K):
    """dX against the same weights' columns."""
    step = 1 << 19
    for k in range(0, K, step):
        k1 = min(K, k + step)
        assert torch.equal(full[:, k:k1], part(k, k1)), k


def test_8_bit_gradient_of_wide_rows():
    M, N, K = 65, 128, 33030144
    dy, dys = whole8(M, N), torch.ones(M, 1, device=DEV)
    w, ws = whole8(N, K), torch.ones(1, K // 128, device=DEV)
    columns(w4.w4a16_fp8_gemm_grad(dy, dys, w, ws),
            lambda a, b: w4.w4a16_fp8_gemm_grad(dy, dys, w[:, a:b].contiguous(), ws[:, a // 128:b // 128].contiguous()),
            K)


@pytest.mark.parametrize("M,K,gs", [(20, 1 << 26, 128), (65, 33030144, 32)])
def test_4_bit_gradient_of_wide_rows(M, K, gs):
    N = 8
    dy = whole(M, N).bfloat16()
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.ldexp(torch.ones(1, device=DEV), torch.randint(-2, 3, (N, K // gs), device=DEV)).bfloat16()
    columns(w4.w4a16_gemm_grad(dy, w, s, group_size=gs),
            lambda a, b: w4.w4a16_gemm_grad(dy, w[:, a // 2:b // 2].contiguous(), s[:, a // gs:b // gs].contiguous(),
                                            group_size=gs), K)


def test_4_bit_gradient_of_wide_output_gradients():
    """dY's own rows past 2^32 bytes per full tile: the sum of its parts along N (whole numbers below 2^24)."""
    M, N, K = 33, 33030144, 128
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    at = torch.randint(0, N, (M, 200), device=DEV)
    dy.scatter_(1, at, torch.randint(-4, 5, (M, 200), device=DEV).bfloat16())
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.ones(N, K // 128, dtype=torch.bfloat16, device=DEV)
    dx = w4.w4a16_gemm_grad(dy, w, s)
    for m in range(M):
        n = at[m].unique()
        q = torch.stack((w[n] & 15, w[n] >> 4), dim=-1).reshape(len(n), K).double() - 8
        want = (dy[m, n].double()[:, None] * q).sum(0)
        assert torch.equal(dx[m], want.bfloat16()), m


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_past_2_36_values(rows):
    """More blocks than one launch has threads for: rows here and there against calls of their own, zeros elsewhere."""
    M, K = (1 << 23) + 130, 8192
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 3.2 * M * K:
        pytest.skip("210 GB of device memory are needed")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(M, K, dtype=torch.uint8, device=DEV).fill_(0x55).view(E4M3)
    at = [0, 1 << 22, (1 << 22) + 128, (1 << 23) - 128, 1 << 23]      # (multiples of 128)
    for r in at:
        x[r:r + 130] = torch.randn(130, K, device=DEV).bfloat16()
    s = torch.full((-(-M // rows), K // 128), -1.0, device=DEV)
    w4.w4a16_fp8_quantize(x, q=q, scales=s, block_rows=rows)
    for r in at:
        r1 = min(M, r + 256)
        q2, s2 = w4.w4a16_fp8_quantize(x[r:r1].clone(), block_rows=rows)
        assert torch.equal(q[r:r1].view(torch.uint8), q2.view(torch.uint8)), r
        assert torch.equal(s[r // rows:-(-r1 // rows)], s2), r
    step = 1 << 17
    for r in range(512, M, step):
        part = q[r:min(M, r + step)].view(torch.uint8)
        kept = torch.zeros(part.shape[0], dtype=torch.bool, device=DEV)
        for a in at:
            kept[max(0, a - r):max(0, a + 130 - r)] = True
        assert not part.view(torch.int64)[~kept].any(), r
    assert (s > 0).all()
    del x, q, s, part
    torch.cuda.empty_cache()


def test_the_most_threads_of_a_launch():
    """Between 2^31 and 2^32 of them: quantisation of one very long row in blocks of 128 x 128, and 2^24 rows by expert in
    tiles of 16."""
    torch.cuda.empty_cache()
    K = (1 << 31) - 128
    x = torch.zeros(1, K, dtype=torch.bfloat16, device=DEV)
    # (powers of two from the CPU: the device's ldexp is off by 2^-24 at some)
    two = torch.ldexp(torch.ones(50), torch.arange(50)).to(DEV)[torch.arange(K // 128, device=DEV) % 50]
    x[0, 5::128] = (7 * two).bfloat16()
    q, s = w4.w4a16_fp8_quantize(x, block_rows=128)
    assert torch.equal(s[0], two / 64)
    v = q.view(torch.uint8).view(-1, 128)
    assert (v[:, 5] == 0x7E).all() and not v[:, :5].any() and not v[:, 6:].any()      # 448 and zeros
    del x, q, s, v, two
    M, N, K, G = 1 << 24, 448, 128, 74
    x, xs = whole8(M, K), torch.ones(M, 1, device=DEV)
    w, ws = whole8(G, N, K), torch.ones(G, -(-N // 128), 1, device=DEV)
    sizes = torch.full((G,), M // G, dtype=torch.int32, device=DEV)
    sizes[3] += M % G
    y = w4.w4a16_fp8_gemm_grouped(x, xs, w, ws, sizes, tile=(16, 0))      # 16 rows and 64 columns per workgroup
    assert torch.equal(y, w4.w4a16_fp8_gemm_grouped(x, xs, w, ws, sizes, tile=(256, 0)))
    last = M - M // G
    assert torch.equal(y[last:last + 300], w4.w4a16_fp8_gemm(x[last:last + 300], xs[last:last + 300], w[-1], ws[-1]))
    del x, xs, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tile", [None, (16, 1), (128, 1), (256, 1)], ids=str)
@pytest.mark.parametrize("top", [1.0, 2.0 ** 60, 1.9921875, 2.0 ** -90])
def test_least_exact_values_of_the_4_bit_gradient(top, tile):
    """dY down to 2^-31 of its row's largest and scales down to 2^-27 of their column group's are exact; the next
    smaller power with all 8 bits is off by half a step of fp16's subnormals: 2^-39 and 2^-35 of a power of two."""
    N, K, odd = 16, 256, 1 + 2.0 ** -7
    two = 2.0 ** torch.tensor(top).log2().floor().item()
    w = torch.full((N, K // 2), 0x88, dtype=torch.uint8)
    w[5] = 0x99                                                    # q - 8 = 1, all others 0
    dy, s = torch.zeros(2, N), torch.ones(N, K // 128)
    dy[:, 0] = top
    dy[0, 5], dy[1, 5] = odd * two * 2.0 ** -31, odd * two * 2.0 ** -32
    run = lambda dy, s: w4.w4a16_gemm_grad(dy.bfloat16().to(DEV), w.to(DEV), s.bfloat16().to(DEV), tile=tile).double().cpu()  # noqa: E731,E501
    y = run(dy, s)
    assert (y[0] == odd * two * 2.0 ** -31).all()
    assert ((y[1] - odd * two * 2.0 ** -32).abs() == two * 2.0 ** -39).all()
    dy, s = torch.zeros(1, N), torch.full((N, K // 128), top)
    dy[0, 5] = 1
    s[5, 0], s[5, 1] = odd * two * 2.0 ** -27, odd * two * 2.0 ** -28
    y = run(dy, s)
    assert (y[0, :128] == odd * two * 2.0 ** -27).all()
    assert ((y[0, 128:] - odd * two * 2.0 ** -28).abs() == two * 2.0 ** -35).all()
