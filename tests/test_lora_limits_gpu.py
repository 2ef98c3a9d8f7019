"""Elements of x . A^T at the ends of their type: infinite ones, finite ones
past the largest bf16, and small ones, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
from gpu_util import dev
from operators_ref import U32, UB16, f64

pytestmark = pytest.mark.gpu

FMAX = float(np.finfo(np.float32).max)
BF16MAX = 255 * 2.0 ** 120


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4._lib()


# the GEMV; the small-batch kernel at its row counts and past 256 scale groups;
# the LDS-staged kernel; the tile kernel behind either kernel of x . A^T
SHAPES = [
    # M, N, K, group, split_k
    (1, 96, 512, 128, 0), (1, 96, 1024, 128, 2), (1, 96, 1280, 128, 0), (6, 96, 512, 128, 0), (7, 40, 33280, 128, 1),
    (12, 96, 1024, 128, 0), (12, 96, 1024, 128, 2), (20, 96, 512, 128, 0), (45, 96, 512, 128, 0),
    (60, 96, 512, 128, 1), (600, 96, 512, 128, 0), (600, 96, 512, 32, 0),
]


class Case:
    """x of +-1 and nibbles of 8, so that the projection is exactly 0; rows of A
    with `terms` elements of +-1, so that x . A^T holds small whole numbers."""

    def __init__(self, M, N, K, group, R, L, terms, seed):
        rng = np.random.default_rng(seed)
        self.group, self.L = group, L
        self.x = rng.choice([-1.0, 1.0], (M, K))
        self.a = np.zeros((L, R, K))
        for l in range(L):
            for r in range(R):
                self.a[l, r, rng.choice(K, terms, replace=False)] = rng.choice([-1.0, 1.0], terms)
        self.b = rng.choice([-1.0, 1.0], (L, N, R)) * rng.integers(128, 256, (L, N, R)) / 128.0
        self.sc = np.ones(L, dtype=np.float32)
        self.ids = (np.arange(M) + 1) % (L + 1) - 1       # every adapter, and bare rows
        if M == 1:
            self.ids[:] = rng.integers(0, L)
        self.w = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=dev())
        self.s = torch.ones(N, K // group, dtype=torch.bfloat16, device=dev())

    def run(self, sk):
        t = lambda v: torch.from_numpy(v).to(dev()).bfloat16()
        return w4.w4a16_gemm_lora(t(self.x), self.w, self.s, t(self.a), t(self.b),
                                  torch.from_numpy(self.ids.astype(np.int32)).to(dev()),
                                  torch.from_numpy(self.sc).to(dev()), split_k=sk, group_size=self.group)

    def check(self, sk):
        """NaN and infinities where the definition has them; elsewhere within
        one fp32 rounding of h, 2^-16 of each element of h (its two bf16 parts),
        2 R + 4 fp32 additions and half a bf16 step."""
        R = self.a.shape[1]
        ref = np.zeros((len(self.ids), self.b.shape[1]))
        mag = np.zeros_like(ref)
        with np.errstate(all="ignore"):
            for m, l in enumerate(self.ids):
                if l >= 0:
                    h = float(self.sc[l]) * (self.a[l] * self.x[m]).sum(1)
                    ref[m] = (h * self.b[l]).sum(1)
                    mag[m] = np.abs(h * self.b[l]).sum(1)
            acc = (2.0 ** -16 + (2 * R + 5) * U32) * mag
            bound = acc + UB16 * (np.abs(ref) + acc)
        got = f64(self.run(sk))
        assert np.array_equal(np.isnan(got), np.isnan(ref)), \
            f"NaN: {np.count_nonzero(np.isnan(got))} against {np.count_nonzero(np.isnan(ref))}"
        inf = np.isinf(ref)
        assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], ref[inf])
        ok = np.isfinite(ref)
        over = np.abs(got[ok] - ref[ok]) - bound[ok]
        assert over.size == 0 or over.max() <= 0, f"{np.count_nonzero(over > 0)} outside"


@pytest.mark.parametrize("M,N,K,group,sk", SHAPES)
@pytest.mark.parametrize("R", [8, 48, 128])
@pytest.mark.parametrize("place", ["a", "scaling"])
def test_infinite_elements(M, N, K, group, sk, R, place):
    """An infinite element of x . A^T gives +-infinity where B is not zero, and
    NaN where it is."""
    c = Case(M, N, K, group, R, 4, 3, seed=M + K + R)
    if place == "a":
        c.a[:3, R // 2, 17] = np.inf
    else:                             # every rank the same element, of three terms and so not 0, and B positive
        c.a[:3] = c.a[:3, :1]
        c.b[:3] = np.abs(c.b[:3])
        c.sc[:3] = np.float32(np.inf)
    c.b[:3, 5, R // 2] = 0.0
    c.check(sk)


@pytest.mark.parametrize("M,N,K,group,sk", SHAPES)
@pytest.mark.parametrize("R", [8, 48, 128])
def test_elements_past_the_largest_bf16(M, N, K, group, sk, R):
    """+-sc for scales between the largest bf16 and the largest fp32."""
    big = [BF16MAX, np.nextafter(np.float32(BF16MAX), np.float32(np.inf)), BF16MAX + 2.0 ** 119, 3.4e38,
           FMAX, np.nextafter(np.float32(FMAX), np.float32(0))]
    for k in (range(len(big)) if M == 1 else (0,)):
        c = Case(M, N, K, group, R, len(big), 1, seed=M + K + R + k)
        c.sc[:] = np.array(big, dtype=np.float32)
        c.b *= 2.0 ** -120
        if M == 1:
            c.ids[:] = k
        c.check(sk)


@pytest.mark.parametrize("M,N,K,group,sk", SHAPES)
@pytest.mark.parametrize("R", [8, 48, 128])
def test_small_elements(M, N, K, group, sk, R):
    """Elements down to 2^-109: their second part is still a normal bf16."""
    c = Case(M, N, K, group, R, 3, 3, seed=M + K + R)
    c.sc[:] = np.array([1.2345678 * 2.0 ** -100, 1.9999 * 2.0 ** -109, 1.0039 * 2.0 ** -109], dtype=np.float32)
    c.b *= 2.0 ** 100
    c.check(sk)


@pytest.mark.parametrize("M,N,K,group,sk", SHAPES)
@pytest.mark.parametrize("R", [8, 48, 128])
def test_infinite_elements_of_b(M, N, K, group, sk, R):
    """An infinite element of B gives +-infinity in its column, whatever the
    second part of the element of x . A^T that it meets (0, or of either sign)."""
    for seed in range(8 if M == 1 else 2):
        c = Case(M, N, K, group, R, 3, 3, seed=M + K + R + seed)
        c.sc[:] = np.array([1.0, 0.7, 1.3], dtype=np.float32)
        c.b[:, 3, R - 1] = np.inf
        c.b[:, 9, 0] = -np.inf
        c.b[:, 20, :] = np.where(c.b[:, 20, :] > 1.5, np.inf, c.b[:, 20, :])
        c.check(sk)
