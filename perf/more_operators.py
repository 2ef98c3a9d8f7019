"""Measured cases of the 8-bit products with a scale for each block of 128
(w4a16_fp8_quantize, w4a16_fp8_gemm, w4a16_fp8_gemm_grouped and their input
gradient w4a16_fp8_gemm_grad) and of the input gradient of the 4-bit products
(w4a16_gemm_grad), plain and with the ragged rows of a mixture of experts.

A case says what in real use it stands for beside its sizes. run() computes it
in its plain form (elementary torch operations in 32 bits, rounded once), or
with the library's own calls where `own` is true.
"""
import math

import torch

own = False

_OPS = ("quantize", "fp8", "fp8_grouped", "fp8_grad", "w4_grad")
_E4M3 = torch.float8_e4m3fn
_MOST = 2 * 8192 ** 3     # operations of the largest case


def _quantize(M, K, rows, name=None):
    c = {"op": "quantize", "M": M, "K": K, "rows": rows}
    return {"name": name, **c} if name else c


def _product(op, M, N, K, G=0, tail=0.0, group=128, name=None):
    """G = 0: one weight matrix; otherwise G experts, whose rows are M (1 - tail) in all."""
    c = {"op": op, "M": M, "N": N, "K": K, "G": G, "tail": tail, "group": group}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the activations of one decode step of 16 requests
        _quantize(16, 5120, 1, name="quantize decode 16x5120"),
        # the activations of a long prefill batch
        _quantize(16384, 8192, 1, name="quantize long 16384x8192"),
        # one request's decode projection
        _product("fp8", 1, 17408, 5120, name="fp8 decode 1x17408x5120"),
        # the decode step of a small batch
        _product("fp8", 16, 8192, 8192, name="fp8 batch 16x8192x8192"),
        # the fused gate-up projection of a ragged prefill
        _product("fp8", 1322, 19456, 2560, name="fp8 prefill 1322x19456x2560"),
        # a long prefill or training batch
        _product("fp8", 8192, 8192, 8192, name="fp8 long 8192x8192x8192"),
        # one decode step of 16 requests, 6 experts each, of 64
        _product("fp8_grouped", 96, 2048, 4096, 64, name="fp8 experts decode 96x2048x4096 G64"),
        # a long batch's rows in expert order, some slots dropped
        _product("fp8_grouped", 16384, 2048, 4096, 32, 0.02, name="fp8 experts long 16384x2048x4096 G32"),
        # training: the gradient of a tall projection at a ragged length
        _product("fp8_grad", 777, 9728, 2560, name="fp8 grad 777x9728x2560"),
        # training: the experts' gradient, some slots dropped
        _product("fp8_grad", 4096, 2048, 4096, 8, 0.02, name="fp8 experts grad 4096x2048x4096 G8"),
        # training adapters over frozen 4-bit weights: the gate-up projection
        _product("w4_grad", 1322, 19456, 2560, name="grad 1322x19456x2560"),
        # the same through the experts, at group 32
        _product("w4_grad", 2048, 2048, 4096, 8, 0.0, 32, name="experts grad 2048x2048x4096 G8 g32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(_OPS)
    if op == "quantize":
        M, K = _log(rng, 1, 16384), 128 * _log(rng, 1, 128)
        return _quantize(min(M, 16384 * 8192 // K), K, rng.choice((1, 1, 128)))
    G = 0
    if op == "fp8_grouped" or (op != "fp8" and rng.random() < 0.5):
        G = _log(rng, 2, 64)
    M = _log(rng, 1, 16384 if G else 8192)
    K = 128 * _log(rng, 1, 32 if G else 76)
    N = _log(rng, 64, 4096 if G else 19456)
    if op == "fp8_grad":
        N = 128 * max(1, N // 128)
    if op == "w4_grad":
        N = 8 * (N // 8)
    while 2 * M * N * K > _MOST // 2:
        M //= 2
    return _product(op, M, N, K, G, rng.choice((0.0, 0.0, 0.1)) if G else 0.0,
                    rng.choice((128, 128, 32)) if op == "w4_grad" else 128)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _sizes(g, case):
    """Rows per expert: uneven popularity, now and then an expert without rows."""
    rows = case["M"] - int(case["M"] * case["tail"])
    p = torch.softmax(0.7 * _randn(g, case["G"]), 0)
    who = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(who, minlength=case["G"]).int()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    M, K = case["M"], case["K"]
    if op == "quantize":
        x = _randn(g, M, K) * torch.exp(0.5 * _randn(g, 1, K))   # channels of uneven size
        return {"op": op, "x": x.bfloat16(), "rows": case["rows"]}
    N, G = case["N"], case["G"]
    lead = (G,) if G else ()
    s = {"op": op, "sizes": None, "cap": 0, "group": case["group"]}
    if G:
        s["sizes"] = _sizes(g, case)
        s["cap"] = max(1, int(s["sizes"].max()))
    out = K if op.endswith("grad") else N
    s["out"] = torch.zeros(M, out, dtype=torch.bfloat16, device="cuda")   # rows behind the last expert's stay zero
    if op == "w4_grad":
        s["w"] = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["s"] = (0.005 + 0.015 * torch.rand(*lead, N, K // case["group"], generator=g, device="cuda")).bfloat16()
        s["dy"] = (_randn(g, M, N) * torch.exp(_randn(g, M, 1) - 7.0)).bfloat16()   # tokens of uneven loss
        return s
    w = (_randn(g, max(G, 1) * N, K) * K ** -0.5).reshape(max(G, 1), N, K)
    w = torch.nn.functional.pad(w, (0, 0, 0, -N % 128)).reshape(-1, K)
    q, sc = _quantized(w, 128)
    s["w"] = q.reshape(max(G, 1), -1, K)[:, :N].contiguous().reshape(*lead, N, K)
    s["ws"] = sc.reshape(*lead, -1, K // 128)
    if op == "fp8_grad":
        dy = _randn(g, M, N) * torch.exp(_randn(g, M, 1) - 7.0)
        s["x"], s["xs"] = _quantized(dy, 1)
    else:
        x = _randn(g, M, K) * torch.exp(0.5 * _randn(g, 1, K))
        s["x"], s["xs"] = _quantized(x, 1)
    return s


# ------------------------------------------------------------------ plain forms

def _quantized(x, rows):
    """e4m3 values and 32-bit scales of blocks of `rows` x 128: the largest magnitude (at least 2^-100) becomes 448; a
    block with an infinity or a NaN gets the scale NaN and values of zero."""
    M, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, 0, 0, -M % rows)).reshape(-1, rows, K // 128, 128)
    top = b.abs().amax(dim=(1, 3))
    fine = torch.isfinite(top)
    top = torch.where(fine, top.clamp(min=2.0 ** -100), 1.0)
    q = torch.where(fine[:, None, :, None], b * (448.0 / top)[:, None, :, None], 0.0).to(_E4M3)
    return q.reshape(-1, K)[:M], torch.where(fine, top / 448.0, math.nan)


def _values(q, scales, rows):
    """The 32-bit values of e4m3 rows [..., n, K] with a scale for each block of `rows` x 128."""
    s = scales.repeat_interleave(rows, dim=-2)[..., : q.shape[-2], :] if rows > 1 else scales
    return (q.float().reshape(*q.shape[:-1], -1, 128) * s[..., None]).reshape(q.shape)


def _int4_values(w, s, gs):
    q = torch.stack((w & 15, w >> 4), dim=-1).reshape(*w.shape[:-1], -1).float() - 8.0
    return (q.reshape(*q.shape[:-1], -1, gs) * s.float()[..., None]).reshape(q.shape)


def _by_expert(x, w, t):
    """Rows [M, n] times their expert's w [G, n, p]: experts padded to the longest."""
    sizes, cap = t["sizes"].long(), t["cap"]
    G, M = w.shape[0], x.shape[0]
    start = sizes.cumsum(0) - sizes
    at = torch.arange(cap, device=x.device)[None, :]
    row = torch.where(at < sizes[:, None], start[:, None] + at, M)              # [G, cap], M: no row
    wide = torch.cat((x, x.new_zeros(1, x.shape[1])))
    y = torch.bmm(wide[row.reshape(-1)].reshape(G, cap, -1), w)
    out = x.new_zeros(M + 1, w.shape[2])
    out[row.reshape(-1)] = y.reshape(G * cap, -1)
    return out[:M]


def _plain(t):
    if t["op"] == "w4_grad":
        x, w = t["dy"].float(), _int4_values(t["w"], t["s"], t["group"])
    else:
        x, w = _values(t["x"], t["xs"], 1), _values(t["w"], t["ws"], 128)
    if not t["op"].endswith("grad"):
        w = w.transpose(-1, -2).contiguous()
    return (x @ w if t["sizes"] is None else _by_expert(x, w, t)).bfloat16()


def run(state):
    t, op = state, state["op"]
    if own:
        import bf16_activation_quantized_amd as w4
        if op == "quantize":
            return w4.w4a16_fp8_quantize(t["x"], block_rows=t["rows"])
        if op == "fp8":
            return w4.w4a16_fp8_gemm(t["x"], t["xs"], t["w"], t["ws"], y=t["out"])
        if op == "fp8_grouped":
            return w4.w4a16_fp8_gemm_grouped(t["x"], t["xs"], t["w"], t["ws"], t["sizes"], y=t["out"])
        if op == "fp8_grad":
            return w4.w4a16_fp8_gemm_grad(t["x"], t["xs"], t["w"], t["ws"], m_sizes=t["sizes"], dx=t["out"])
        return w4.w4a16_gemm_grad(t["dy"], t["w"], t["s"], m_sizes=t["sizes"], dx=t["out"], group_size=t["group"])
    if op == "quantize":
        return _quantized(t["x"], t["rows"])
    return _plain(t)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantize":
        return {"bytes": 3 * M * K + 4 * (K // 128) * (-(-M // case["rows"])), "flops": 2 * M * K}
    N, G = case["N"], max(1, case["G"])
    rows = M - int(M * case["tail"])
    met = min(G, max(1, rows))       # experts that can have rows
    if case["op"] == "w4_grad":
        byts = met * (N * K // 2 + 2 * N * (K // case["group"])) + 2 * rows * (N + K)
    else:
        inner, outer = (N, K) if case["op"] == "fp8_grad" else (K, N)
        byts = met * (N * K + 4 * (-(-N // 128)) * (K // 128)) + rows * (inner + 4 * (inner // 128) + 2 * outer)
    return {"bytes": byts, "flops": 2 * rows * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3_of(v):
    """The nearest e4m3 value, ties to even, of 64-bit values of magnitude at most 448."""
    e = torch.frexp(v.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    t = prepare(case, seed)
    op, M, K = case["op"], case["M"], case["K"]
    if op == "quantize":
        r = case["rows"]
        scales = torch.empty(-(-M // r), K // 128, dtype=torch.float64, device="cuda")
        q = torch.empty(M, K, dtype=torch.float64, device="cuda")
        for k0 in range(0, K, 1024):
            x = t["x"][:, k0:k0 + 1024].double()
            n = x.shape[1] // 128
            top = x.abs().reshape(M, n, 128).amax(2)
            if r > 1:
                top = torch.stack([top[i:i + r].amax(0) for i in range(0, M, r)])
            scales[:, k0 // 128:k0 // 128 + n] = top / 448
            each = top.repeat_interleave(r, 0)[:M].repeat_interleave(128, 1)
            q[:, k0:k0 + 1024] = _e4m3_of(x * 448 / each)
        return q, scales
    N, G = case["N"], case["G"]
    grad = op.endswith("grad")

    def weights(e, n0, n1):
        """Rows n0 .. n1 of expert e's weights."""
        w = (t["w"][e] if G else t["w"])[n0:n1]
        if op == "w4_grad":
            gs = case["group"]
            w = w.to(torch.int16)
            d = torch.empty(w.shape[0], K, dtype=torch.float64, device="cuda")
            d[:, 0::2] = (w % 16).double() - 8
            d[:, 1::2] = torch.div(w, 16, rounding_mode="floor").double() - 8
            return d * (t["s"][e] if G else t["s"])[n0:n1].double().repeat_interleave(gs, dim=1)
        s = (t["ws"][e] if G else t["ws"]).double()
        block = torch.arange(n0, n1, device="cuda") // 128
        return w.double() * s[block].repeat_interleave(128, dim=1)

    y = torch.zeros(M, K if grad else N, dtype=torch.float64, device="cuda")
    row = 0
    for e, size in enumerate(t["sizes"].tolist() if G else [M]):
        if size == 0:
            continue
        if op == "w4_grad":
            x = t["dy"][row:row + size].double()
        else:
            x = t["x"][row:row + size].double() * t["xs"][row:row + size].double().repeat_interleave(128, dim=1)
        for n0 in range(0, N, 4096):   # the weights in 64 bits are large
            n1 = min(N, n0 + 4096)
            if grad:
                y[row:row + size] += x[:, n0:n1] @ weights(e, n0, n1)
            else:
                y[row:row + size, n0:n1] = x @ weights(e, n0, n1).t()
        row += size
    return y
