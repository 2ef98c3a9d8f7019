"""The experts' row operators on the GPU against their 64-bit definitions:
sort bit-exact, gather bit-exact, combine and the gradients within the bounds
that operators_ref derives; rows that no slot names stay as they were."""
import numpy as np
import pytest
import torch

import bf16_activation_quantized_amd as w4
from gpu_util import dev
from operators_ref import combine_grad_ref, combine_ref, f64, gather_ref, sort_ref, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4._lib()


def _ids(rng, T, k, G, kind):
    if kind == "one":                                   # every slot to one expert
        return np.full((T, k), min(G - 1, 3), dtype=np.int32)
    if kind == "none":                                  # nothing kept
        return np.full((T, k), -1, dtype=np.int32)
    if kind == "skew":                                  # a few popular experts
        return np.minimum(rng.geometric(0.3, (T, k)) - 1, G - 1).astype(np.int32)
    ids = rng.integers(0, G, (T, k)).astype(np.int32)
    if kind == "holes":                                 # padded tokens and ids of other devices
        ids[rng.random((T, k)) < 0.2] = -1
        ids[rng.random((T, k)) < 0.1] = G
        ids[rng.random((T, k)) < 0.05] = np.iinfo(np.int32).max
        ids[rng.random((T, k)) < 0.05] = np.iinfo(np.int32).min
    return ids


SORT_CASES = [
    # T, k, G, kind
    (1, 1, 1, "rand"), (1, 8, 8, "rand"), (3, 1, 4096, "rand"), (16, 4, 8, "holes"), (63, 1, 7, "skew"),
    (64, 1, 64, "rand"), (65, 1, 65, "holes"), (255, 4, 128, "one"), (256, 4, 128, "rand"), (257, 4, 31, "skew"),
    (1000, 6, 160, "holes"), (512, 8, 256, "none"), (4097, 8, 127, "rand"), (2048, 2, 4096, "holes"),
    (40000, 8, 128, "skew"), (33333, 7, 255, "holes"), (300000, 1, 16, "one"), (270001, 2, 1000, "rand"),
    (20000, 8, 4096, "holes"), (8192, 1, 2047, "rand"), (8193, 1, 2048, "holes"), (4096, 2, 4096, "one"),
    (1100000, 2, 60, "skew"), (700001, 3, 4095, "holes"),
    # each shape of the sort, on both sides of its borders, with few and many counts
    (2048, 1, 2048, "rand"), (2049, 1, 2049, "holes"), (683, 3, 5, "skew"), (131072, 1, 190, "holes"),
    (131072, 1, 191, "holes"), (131073, 1, 300, "rand"), (65536, 8, 190, "skew"), (65536, 8, 192, "holes"),
    (174763, 3, 1024, "holes"), (524289, 1, 383, "rand"), (524289, 1, 50, "holes"), (40961, 1, 1025, "holes"),
    (9000, 1, 1200, "rand"), (131072, 1, 255, "rand"), (131072, 1, 256, "skew"), (65536, 8, 255, "holes"),
    (65536, 8, 256, "one"),
]


@pytest.mark.parametrize("T,k,G,kind", SORT_CASES)
def test_sort(T, k, G, kind):
    ids = _ids(np.random.default_rng(T * 31 + k * 7 + G), T, k, G, kind)
    order, pos, sizes = w4.w4a16_expert_sort(torch.from_numpy(ids).to(dev()), G)
    ro, rp, rs = sort_ref(ids, G)
    assert np.array_equal(sizes.cpu().numpy(), rs)
    assert np.array_equal(pos.cpu().numpy(), rp)
    assert np.array_equal(order.cpu().numpy(), ro)


def test_sort_no_tokens():
    for k in (1, 4):
        sizes = torch.full((37,), 5, dtype=torch.int32, device=dev())
        order, pos, sizes = w4.w4a16_expert_sort(torch.empty((0, k), dtype=torch.int32, device=dev()), 37,
                                                 m_sizes=sizes)
        assert order.numel() == 0 and pos.numel() == 0
        assert not sizes.cpu().any()


def _case(T, k, G, width, kind, seed):
    rng = np.random.default_rng(seed)
    ids = _ids(rng, T, k, G, kind)
    pos = sort_ref(ids, G)[1].astype(np.int32)
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, width, generator=gen).bfloat16()
    z = torch.randn(T * k, width, generator=gen).bfloat16()
    w = torch.softmax(torch.randn(T, k, generator=gen), dim=1)
    return x, z, w, pos, torch.from_numpy(pos).to(dev())


ROW_CASES = [
    # T, k, G, width, kind
    (1, 1, 1, 1, "rand"), (1, 4, 8, 128, "rand"), (5, 2, 3, 7, "holes"), (17, 3, 8, 8, "holes"),
    (9, 1, 4, 9, "rand"), (33, 2, 8, 129, "holes"), (13, 8, 16, 512, "rand"), (31, 5, 8, 1001, "holes"),
    (20, 17, 32, 250, "holes"), (7, 3, 4, 2048, "none"), (64, 2, 8, 2056, "rand"), (11, 4, 8, 4100, "skew"),
    (6, 6, 8, 9001, "holes"), (3, 70, 100, 300, "holes"), (300, 8, 64, 1024, "rand"), (5, 2, 4, 20008, "holes"),
]


@pytest.mark.parametrize("T,k,G,width,kind", ROW_CASES)
def test_gather(T, k, G, width, kind):
    x, _, _, pos, dpos = _case(T, k, G, width, kind, T + width)
    xs = torch.full((T * k + 1, width), 7.0, dtype=torch.bfloat16, device=dev())   # a guard row behind
    got = w4.w4a16_expert_gather(x.to(dev()), dpos, xs=xs)
    assert np.array_equal(f64(got), gather_ref(f64(x), pos, np.full((T * k + 1, width), 7.0)))


@pytest.mark.parametrize("T,k,G,width,kind", ROW_CASES)
def test_gather_grad(T, k, G, width, kind):
    _, z, _, pos, dpos = _case(T, k, G, width, kind, T + width)
    got = w4.w4a16_expert_gather_grad(z.to(dev()), dpos)
    ref, bound = combine_ref(f64(z), pos, None)
    within(f64(got), ref, bound, "gather_grad")


@pytest.mark.parametrize("T,k,G,width,kind", ROW_CASES)
def test_combine(T, k, G, width, kind):
    _, z, w, pos, dpos = _case(T, k, G, width, kind, T + width)
    y = torch.full((T, width), float("nan"), dtype=torch.bfloat16, device=dev())
    got = w4.w4a16_expert_combine(z.to(dev()), dpos, w.to(dev()), y=y)
    ref, bound = combine_ref(f64(z), pos, f64(w))
    within(f64(got), ref, bound, "combine")
    first = got.clone()
    again = w4.w4a16_expert_combine(z.to(dev()), dpos, w.to(dev()))
    assert torch.equal(first, again)


@pytest.mark.parametrize("T,k,G,width,kind", ROW_CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_grad(T, k, G, width, kind, in_place):
    x, z, w, pos, dpos = _case(T, k, G, width, kind, T + width)
    zd = z.to(dev())
    dz = zd if in_place else torch.full((T * k, width), 7.0, dtype=torch.bfloat16, device=dev())
    before = f64(z) if in_place else np.full((T * k, width), 7.0)
    got, dw = w4.w4a16_expert_combine_grad(x.to(dev()), zd, dpos, w.to(dev()), dz=dz)
    rz, bz, rw, bw = combine_grad_ref(f64(x), f64(z), pos, f64(w), before)
    within(f64(got), rz, bz, "dz")
    within(f64(dw), rw, bw, "dweights")


def test_fewer_rows_than_slots():
    """Slots whose position is not below `rows` count as dropped, in every call."""
    T, k, G, width, rows = 23, 4, 8, 300, 40
    x, z, w, pos, dpos = _case(T, k, G, width, "rand", 3)
    buf = torch.full((T * k, width), 7.0, dtype=torch.bfloat16, device=dev())
    w4.w4a16_expert_gather(x.to(dev()), dpos, xs=buf[:rows])
    ref = np.full((T * k, width), 7.0)
    ref[:rows] = gather_ref(f64(x), pos, ref[:rows])
    assert np.array_equal(f64(buf), ref)
    ry, by = combine_ref(f64(z)[:rows], pos, f64(w))
    within(f64(w4.w4a16_expert_combine(z[:rows].to(dev()), dpos, w.to(dev()))), ry, by, "combine")
    dz = torch.full((T * k, width), 7.0, dtype=torch.bfloat16, device=dev())
    _, dw = w4.w4a16_expert_combine_grad(x.to(dev()), z[:rows].to(dev()), dpos, w.to(dev()), dz=dz[:rows])
    rz, bz, rw, bw = combine_grad_ref(f64(x), f64(z)[:rows], pos, f64(w), np.full((rows, width), 7.0))
    within(f64(dz[:rows]), rz, bz, "dz")
    assert (dz[rows:] == 7.0).all()
    within(f64(dw), rw, bw, "dweights")
    # no rows at all: zero results
    none = torch.empty((0, width), dtype=torch.bfloat16, device=dev())
    assert not w4.w4a16_expert_combine(none, dpos, w.to(dev())).any()
    w4.w4a16_expert_gather(x.to(dev()), dpos, xs=none)
    _, dw = w4.w4a16_expert_combine_grad(x.to(dev()), none, dpos, w.to(dev()))
    assert not dw.any()


def test_dropped_rows_are_not_read():
    """Infinities and NaN in rows that no slot names reach nothing."""
    T, k, G, width = 40, 3, 8, 136
    x, z, w, pos, dpos = _case(T, k, G, width, "holes", 11)
    kept = int((pos >= 0).sum())
    zb = z.clone()
    zb[kept:] = float("nan")
    zb[kept + 1::2] = float("inf")
    assert torch.equal(w4.w4a16_expert_combine(zb.to(dev()), dpos, w.to(dev())),
                       w4.w4a16_expert_combine(z.to(dev()), dpos, w.to(dev())))
    wb = w.clone()
    wb[torch.from_numpy(pos < 0)] = float("nan")
    dz, dw = w4.w4a16_expert_combine_grad(x.to(dev()), zb.to(dev()), dpos, wb.to(dev()))
    assert torch.isfinite(dz[:kept]).all() and torch.isfinite(dw).all()


def test_infinities_of_named_rows_stay_with_their_token():
    T, k, width = 12, 2, 264
    pos = torch.arange(T * k, dtype=torch.int32, device=dev()).reshape(T, k)
    z = torch.ones(T * k, width, dtype=torch.bfloat16, device=dev())
    z[6] = float("inf")
    z[9, 5] = float("nan")
    y = w4.w4a16_expert_combine(z, pos, torch.full((T, k), 0.5, device=dev()))
    assert torch.isinf(y[3]).all() and torch.isnan(y[4, 5])
    ok = torch.ones(T, width, dtype=torch.bool, device=dev())
    ok[3] = False
    ok[4, 5] = False
    assert (y[ok] == 1.0).all()


@pytest.mark.parametrize("width", [5, 64])
def test_gradients_against_differences(width):
    """combine is linear in z and in the weights: with small integers every
    value is exact in bf16 and fp32, and a step of 1 gives the gradient of
    <y, dy> exactly."""
    T, k, G = 4, 2, 3
    rng = np.random.default_rng(width)
    ids = _ids(rng, T, k, G, "rand")
    ids[1, 1] = -1
    pos = torch.from_numpy(sort_ref(ids, G)[1].astype(np.int32)).to(dev())
    z = torch.from_numpy(rng.integers(-3, 4, (T * k, width))).to(dev()).bfloat16()
    w = torch.from_numpy(rng.integers(-2, 3, (T, k))).to(dev()).float()
    dy = torch.from_numpy(rng.integers(-3, 4, (T, width))).to(dev()).bfloat16()
    x = torch.from_numpy(rng.integers(-3, 4, (T, width))).to(dev()).bfloat16()

    def loss(z, w):
        return (w4.w4a16_expert_combine(z, pos, w).double() * dy.double()).sum().item()

    dz, dw = w4.w4a16_expert_combine_grad(dy, z, pos, w, dz=torch.zeros_like(z))
    base = loss(z, w)
    for t in range(T):
        for j in range(k):
            ws = w.clone()
            ws[t, j] += 1
            assert loss(z, ws) - base == dw[t, j].item()
    for r in range(T * k):
        for c in range(0, width, 3):
            zs = z.clone()
            zs[r, c] += 1
            assert loss(zs, w) - base == dz[r, c].item()

    # gather: dxs stands for dL/dxs
    dxs = z
    def gloss(x):
        xs = torch.zeros(T * k, width, dtype=torch.bfloat16, device=dev())
        return (w4.w4a16_expert_gather(x, pos, xs=xs).double() * dxs.double()).sum().item()
    dx = w4.w4a16_expert_gather_grad(dxs, pos)
    base = gloss(x)
    for t in range(T):
        for c in range(width):
            xst = x.clone()
            xst[t, c] += 1
            assert gloss(xst) - base == dx[t, c].item()


def test_arrays_past_32_bit_offsets():
    """4.8 GB of rows: the last ones are as right as the first."""
    T, width = 580000, 4136
    x = torch.randn(64, width, device=dev()).bfloat16()
    src = x.repeat(T // 64 + 1, 1)[:T]
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev()).reshape(T, 1)
    xs = w4.w4a16_expert_gather(src, pos)
    for r in (0, 1, T // 2, T - 2, T - 1):
        assert torch.equal(xs[r], src[T - 1 - r]), r
    y = w4.w4a16_expert_combine(xs, pos, torch.full((T, 1), 2.0, device=dev()))
    assert torch.equal(y[-1000:], 2 * src[-1000:]) and torch.equal(y[:1000], 2 * src[:1000])
    dz, dw = w4.w4a16_expert_combine_grad(src, xs, pos, torch.full((T, 1), 2.0, device=dev()), dz=y)
    for r in (0, 1, T // 2, T - 2, T - 1):
        assert torch.equal(dz[r], 2 * src[T - 1 - r]), r
    assert torch.allclose(dw[-64:, 0], (src[-64:].float() ** 2).sum(1), rtol=1e-4)


def test_binding_refuses_what_does_not_fit():
    x, z, w, pos, dpos = _case(8, 2, 4, 64, "rand", 1)
    x, z, w = x.to(dev()), z.to(dev()), w.to(dev())
    for f in (lambda: w4.w4a16_expert_sort(dpos[0], 4), lambda: w4.w4a16_expert_sort(dpos.t(), 4),
              lambda: w4.w4a16_expert_sort(dpos, 4, order=torch.empty(3, dtype=torch.int32, device=dev())),
              lambda: w4.w4a16_expert_gather(x[:7], dpos), lambda: w4.w4a16_expert_gather(x, dpos, xs=z[:, :32]),
              lambda: w4.w4a16_expert_combine(z.t(), dpos), lambda: w4.w4a16_expert_combine(z, dpos, w[:, :1]),
              lambda: w4.w4a16_expert_combine(z, dpos.cpu()), lambda: w4.w4a16_expert_gather_grad(z[0], dpos),
              lambda: w4.w4a16_expert_combine_grad(x[:, :32], z, dpos, w)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: w4.w4a16_expert_sort(dpos.long(), 4), lambda: w4.w4a16_expert_gather(x.float(), dpos),
              lambda: w4.w4a16_expert_combine(z, dpos, w.bfloat16()),
              lambda: w4.w4a16_expert_combine_grad(x, z, dpos, None)):
        with pytest.raises(TypeError):
            f()
    for G in (0, 4097):
        with pytest.raises((w4.W4A16Error, RuntimeError)):
            w4.w4a16_expert_sort(dpos, G)


@pytest.mark.parametrize("G,T", [(7, 40000), (2000, 3000), (4096, 9000)])
def test_sort_workspace_is_written_before_it_is_read(G, T):
    ids = _ids(np.random.default_rng(T), T, 3, G, "holes")
    need = w4.w4a16_expert_sort_workspace_bytes(T, 3, G)
    ws = torch.full((need // 4 + 8,), -7, dtype=torch.int32, device=dev())
    order, pos, sizes = w4.w4a16_expert_sort(torch.from_numpy(ids).to(dev()), G, workspace=ws[:need // 4])
    ro, rp, rs = sort_ref(ids, G)
    assert np.array_equal(order.cpu().numpy(), ro) and np.array_equal(pos.cpu().numpy(), rp)
    assert np.array_equal(sizes.cpu().numpy(), rs)
    assert (ws[need // 4:] == -7).all()


def test_side_stream_and_graph_replays():
    """On a stream of the caller's own, and captured: every replay equals the
    eager result, with eager work between."""
    T, k, G, width = 300, 4, 16, 1030
    x, z, w, pos, dpos = _case(T, k, G, width, "holes", 21)
    ids = torch.from_numpy(_ids(np.random.default_rng(21), T, k, G, "holes")).to(dev())
    x, z, w = x.to(dev()), z.to(dev()), w.to(dev())

    def all_calls(stream=None):
        order, p, sizes = w4.w4a16_expert_sort(ids, G, stream=stream)
        xs = torch.zeros(T * k, width, dtype=torch.bfloat16, device=dev()) if stream is None else None
        if stream is not None:
            with torch.cuda.stream(stream):
                xs = torch.zeros(T * k, width, dtype=torch.bfloat16, device=dev())
                dz = torch.zeros_like(xs)
        else:
            dz = torch.zeros_like(xs)
        xs = w4.w4a16_expert_gather(x, p, xs=xs, stream=stream)
        y = w4.w4a16_expert_combine(xs, p, w, stream=stream)
        dz, dw = w4.w4a16_expert_combine_grad(y, xs, p, w, dz=dz, stream=stream)
        dx = w4.w4a16_expert_gather_grad(dz, p, stream=stream)
        return order, p, sizes, xs, y, dz, dw, dx

    want = [t.clone() for t in all_calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = all_calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = all_calls()
    for _ in range(4):
        for t in cap[3:]:
            t.fill_(3)
        cap[3].zero_()
        cap[5].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, cap))
        all_calls()
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,k,width", [(9000, 8, 2056), (45000, 3, 1003), (400000, 2, 176)])
def test_rows_beyond_the_caches(T, k, width):
    """More than 256 MB of expert rows: each call against the same call on a
    few of its tokens, with guard rows behind."""
    G = 16
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, k, G, "holes")
    pos = sort_ref(ids, G)[1].astype(np.int32)
    kept = int((pos >= 0).sum())
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, width, generator=gen, device=dev()).bfloat16()
    z = torch.randn(T * k, width, generator=gen, device=dev()).bfloat16()
    w = torch.rand(T, k, generator=gen, device=dev())
    dpos = torch.from_numpy(pos).to(dev())
    xs = w4.w4a16_expert_gather(x, dpos, xs=torch.full_like(z, 7.0))
    y = w4.w4a16_expert_combine(z, dpos, w)
    dz, dw = w4.w4a16_expert_combine_grad(x, z, dpos, w, dz=torch.full_like(z, 7.0))
    dx = w4.w4a16_expert_gather_grad(z, dpos)
    assert (xs[kept:] == 7.0).all() and (dz[kept:] == 7.0).all()
    tok = np.unique(np.concatenate([[0, 1, T // 2, T - 2, T - 1], rng.integers(0, T, 60)]))
    rows = np.concatenate([pos[t][pos[t] >= 0] for t in tok]).astype(np.int64)
    small = {int(r): i for i, r in enumerate(rows)}     # the named rows of these tokens, renumbered
    sp = np.array([[small[int(p)] if p >= 0 else -1 for p in pos[t]] for t in tok])
    pick = torch.from_numpy(rows).to(dev())
    tt = torch.from_numpy(tok).to(dev())
    xn, zn, wn = f64(x[tt]), f64(z[pick]), f64(w[tt])
    assert np.array_equal(f64(xs[pick]), gather_ref(xn, sp, np.zeros((len(rows), width))))
    within(f64(y[tt]), *combine_ref(zn, sp, wn), "combine")
    within(f64(dx[tt]), *combine_ref(zn, sp, None), "gather_grad")
    rz, bz, rw, bw = combine_grad_ref(xn, zn, sp, wn, np.zeros((len(rows), width)))
    within(f64(dz[pick]), rz, bz, "dz")
    within(f64(dw[tt]), rw, bw, "dweights")
