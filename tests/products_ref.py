"""Plain 64-bit definitions of the 8-bit products, their quantisation and the
input gradients, for the tests (torch on the CPU; independent of the library)."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn


def e4m3_of(v: torch.Tensor) -> torch.Tensor:
    """The nearest e4m3 value, ties to even, of 64-bit values within +-448."""
    e = torch.frexp(v.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def quantize_ref(x: torch.Tensor, rows: int):
    """(values q before their rounding, scales) of blocks of `rows` x 128, both in 64 bits."""
    x = x.double()
    M, K = x.shape
    q = torch.empty_like(x)
    s = torch.empty(-(-M // rows), K // 128, dtype=torch.float64)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * rows, min(M, (i + 1) * rows)), slice(128 * j, 128 * (j + 1)))
            top = max(x[at].abs().max().item(), 2.0 ** -100)
            s[i, j] = top / 448
            q[at] = x[at] * 448 / top
    return q, s


def fp8_values(q: torch.Tensor, scales: torch.Tensor, rows: int) -> torch.Tensor:
    """64-bit values of e4m3 [M, K] with a scale for each block of rows x 128."""
    each = scales.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)
    return q.float().double() * each


def int4_values(w: torch.Tensor, s: torch.Tensor, gs: int) -> torch.Tensor:
    """64-bit values of packed [N, K / 2] with bf16 scales [N, K / gs]."""
    q = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64)
    q[:, 0::2] = (w & 15).double() - 8
    q[:, 1::2] = (w >> 4).double() - 8
    return q * s.double().repeat_interleave(gs, 1)


def grouped_ref(x: torch.Tensor, ws, sizes, out: int):
    """(sum, sum of magnitudes) of each row with its expert's weights ws[e] [n, p]
    (x [M, n] in 64 bits); rows past the last expert's: NaN."""
    y = torch.full((x.shape[0], out), float("nan"), dtype=torch.float64)
    a = torch.zeros_like(y)
    r = 0
    for w, n in zip(ws, sizes):
        y[r:r + n] = x[r:r + n] @ w
        a[r:r + n] = x[r:r + n].abs() @ w.abs()
        r += n
    return y, a
