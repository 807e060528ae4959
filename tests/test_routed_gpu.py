"""Routed tokens against their definitions in 64 bits: qgemm_moe_dispatch, qgemm_moe_combine and
the gradients of both.

Tolerances are counted in roundings.  u = 2^-24 is half a step of fp32, eps / 2 of the output's
type half a step of it.  A sum of n fp32 terms, in any order, is off by at most n u times the sum
of magnitudes (each of its n roundings acts on a partial sum below that); U adds the second-order
terms (n u < 2^-8 here)."""
import numpy as np
import pytest
import torch

from block_quantized_weight_qgemm_b200 import qgemm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24 * 1.01
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_quantized_weight_qgemm_b200 import build
    build.build()
    qgemm.lib()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def routing(T, k, E, seed=0, kind="random"):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)  # repeats within a token too
    if kind == "drop":
        ids[torch.rand(T, k, generator=g) < 0.3] = -1
        ids[torch.rand(T, k, generator=g) < 0.1] = E            # outside on the other side
        ids[torch.rand(T, k, generator=g) < 0.05] = -2 ** 31
    elif kind == "none":
        ids.fill_(-1)
    elif kind == "one":
        ids.fill_(E - 1)
    return ids


def maps(ids, E):
    """(offsets, rows) by Python's stable sort of the slots."""
    flat = ids.reshape(-1).tolist()
    order = sorted((s for s, e in enumerate(flat) if 0 <= e < E), key=lambda s: flat[s])
    rows = np.full(len(flat), -1, dtype=np.int32)
    rows[order] = np.arange(len(order))
    count = np.bincount([flat[s] for s in order], minlength=E)[:E] if order else np.zeros(E, int)
    return np.concatenate([[0], np.cumsum(count)]), rows.reshape(ids.shape)


def randn(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


SORTS = [(1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 10, 512), (37, 3, 7), (255, 1, 256), (410, 10, 512),
         (1025, 4, 4), (2048, 10, 512), (700, 7, 4096), (513, 33, 40), (30011, 6, 257), (4097, 1, 64),
         (2000, 1, 3), (1500, 5, 3500), (8191, 2, 511), (50000, 2, 1), (819, 10, 512)]


@pytest.mark.parametrize("kind", ["random", "drop", "none", "one"])
@pytest.mark.parametrize("T,k,E", SORTS)
def test_dispatch_maps_and_rows(T, k, E, kind):
    ids = routing(T, k, E, seed=T + E, kind=kind)
    H = 24
    x = randn(T, H, dtype=BF16, seed=T)
    xs = torch.full((T * k, H), 7.0, dtype=BF16, device="cuda")
    out, offsets, rows = qgemm.moe_dispatch(x.cuda(), ids.cuda(), E, xs=xs)
    off_ref, rows_ref = maps(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), off_ref)
    assert np.array_equal(rows.cpu().numpy(), rows_ref)
    ref = torch.full((T * k, H), 7.0, dtype=BF16)   # rows behind the last expert stay
    live = rows_ref >= 0
    ref[rows_ref[live]] = x[np.nonzero(live)[0]]
    assert torch.equal(out.cpu().view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 16, 100, 1001, 2048, 5120, 20000])
def test_dispatch_row_widths_bit_for_bit(H, dtype):
    T, k, E = 11, 3, 4
    ids = routing(T, k, E, seed=H, kind="drop")
    esize = dtype.itemsize
    bits = torch.randint(0, 256, (T, H * esize), dtype=torch.uint8, generator=torch.Generator().manual_seed(H))
    x = bits.view(dtype)  # any bits, NaN payloads among them
    out, _, rows = qgemm.moe_dispatch(x.cuda(), ids.cuda(), E)
    out, rows = out.cpu().view(torch.uint8), rows.cpu()
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                assert torch.equal(out[rows[t, j]], bits[t])


def gathered(a, rows):
    """float64 [T, k, H]; zeros where there is no row."""
    r = a.double()[rows.clamp(min=0).long()]
    return torch.where((rows >= 0)[:, :, None], r, torch.zeros_like(r))


CASES = [(1, 1, 8), (1, 8, 2048), (5, 2, 1), (64, 10, 2048), (33, 3, 1001), (19, 9, 6), (130, 17, 264),
         (2, 40, 4100), (301, 2, 16), (7, 8, 9000)]


def inputs_of(T, k, H, dtype, seed, kind="drop"):
    E = 6
    ids = routing(T, k, E, seed=seed, kind=kind)
    rows = torch.from_numpy(maps(ids, E)[1])
    a = randn(T * k, H, dtype=dtype, seed=seed + 1)
    w = randn(T, k, seed=seed + 2)
    n = int((rows >= 0).sum())
    a[n:] = float("nan")              # nothing behind the last expert is read
    w[rows < 0] = float("nan")        # nor the weight of a slot without a row
    return rows, a, w


@pytest.mark.parametrize("din", [F32, BF16])
@pytest.mark.parametrize("dout", [F32, BF16])
@pytest.mark.parametrize("T,k,H", CASES)
def test_combine(T, k, H, din, dout):
    rows, ys, w = inputs_of(T, k, H, din, seed=H + T)
    y = qgemm.moe_combine(ys.cuda(), rows.cuda(), w.cuda(), y_dtype=dout).cpu()
    wd = torch.where(rows >= 0, w, torch.zeros_like(w)).double()[:, :, None]
    terms = gathered(ys, rows) * wd
    ref, mag = terms.sum(1), terms.abs().sum(1)
    # k fused multiply-adds, then the output's rounding
    assert ((y.double() - ref).abs() <= half(dout) * ref.abs() + (1 + half(dout)) * k * U * mag).all()


@pytest.mark.parametrize("din", [F32, BF16])
@pytest.mark.parametrize("dout", [F32, BF16])
@pytest.mark.parametrize("T,k,H", CASES)
def test_gradients(T, k, H, din, dout):
    rows, ys, w = inputs_of(T, k, H, din, seed=H + T + 1)
    dy = randn(T, H, dtype=dout, seed=9)
    dys = torch.full((T * k, H), 7.0, dtype=din, device="cuda")
    dys, dw = qgemm.moe_combine_grad(dy.cuda(), ys.cuda(), rows.cuda(), w.cuda(), dys=dys)
    dys, dw = dys.cpu(), dw.cpu()
    live = rows >= 0
    wd = torch.where(live, w, torch.zeros_like(w)).double()
    want = dy.double()[:, None, :] * wd[:, :, None]
    got = gathered(dys, rows)
    want = torch.where(live[:, :, None], want, torch.zeros_like(want))
    assert ((got - want).abs() <= (half(din) + U) * (1 + U) * want.abs()).all()
    n = int(live.sum())
    assert (dys[n:] == 7.0).all()     # rows no slot names
    terms = dy.double()[:, None, :] * gathered(ys, rows)
    assert ((dw.double() - terms.sum(2)).abs() <= H * U * terms.abs().sum(2)).all()
    assert (dw[~live] == 0).all()
    # the gradient of the tokens: k additions, then the output's rounding
    dx = qgemm.moe_dispatch_grad(ys.cuda(), rows.cuda(), dx_dtype=dout).cpu()
    terms = gathered(ys, rows)
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert ((dx.double() - ref).abs() <= half(dout) * ref.abs() + (1 + half(dout)) * k * U * mag).all()


def test_gradients_against_differences():
    # loss = <combine(ys, w), c> is linear in ys and in w; dispatch is linear in x: central
    # differences with a step of 1 of the fp32 operators themselves give the gradients up to the
    # roundings of two losses of n terms each
    T, k, H, E = 6, 3, 40, 4
    ids = routing(T, k, E, seed=3, kind="drop")
    x, c = randn(T, H, seed=4).cuda(), randn(T, H, seed=5).cuda()
    xs, _, rows = qgemm.moe_dispatch(x, ids.cuda(), E)
    xs[int((rows >= 0).sum()):] = 0
    w = randn(T, k, seed=6).cuda()
    dys, dw = qgemm.moe_combine_grad(c, xs, rows, w)
    dx = qgemm.moe_dispatch_grad(torch.where(torch.arange(T * k, device="cuda")[:, None] < int((rows >= 0).sum()),
                                             dys, torch.zeros_like(dys)), rows, dx_dtype=F32)

    def loss(x_, w_):
        s, _, r = qgemm.moe_dispatch(x_, ids.cuda(), E)
        return float((qgemm.moe_combine(s, r, w_, y_dtype=F32).double() * c.double()).sum())

    mag = float((qgemm.moe_combine(xs.abs() + 1, rows, w.abs() + 1, y_dtype=F32) * c.abs()).double().sum())
    tol = 2 * (k + 1) * U * mag + H * U * mag
    for t, h in ((0, 0), (2, 39), (5, 17)):
        d = torch.zeros_like(x)
        d[t, h] = 1.0
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2 - float(dx[t, h])) <= tol
    for t, j in ((0, 0), (3, 1), (5, 2)):
        d = torch.zeros_like(w)
        d[t, j] = 1.0
        assert abs((loss(x, w + d) - loss(x, w - d)) / 2 - float(dw[t, j])) <= tol


def test_rows_outside_the_buffer_count_as_none():
    T, k, H = 4, 2, 64
    ys, w = randn(T * k, H).cuda(), torch.ones(T, k, device="cuda")
    rows = torch.arange(T * k, dtype=torch.int32).view(T, k)
    rows[1, 0], rows[2, 1], rows[3, 0] = T * k, 2 ** 31 - 1, -7
    ok = (rows >= 0) & (rows < T * k)
    ref = gathered(ys.cpu(), torch.where(ok, rows, torch.full_like(rows, -1))).sum(1)
    assert torch.equal(qgemm.moe_combine(ys, rows.cuda(), w, y_dtype=F32).cpu().double(), ref.float().double())
    assert torch.equal(qgemm.moe_dispatch_grad(ys, rows.cuda(), dx_dtype=F32).cpu().double(), ref.float().double())
    dys = torch.full((T * k, H), 7.0, device="cuda")
    dys, dw = qgemm.moe_combine_grad(torch.ones(T, H, device="cuda"), ys, rows.cuda(), w, dys=dys)
    named = torch.zeros(T * k, dtype=torch.bool)
    named[rows[ok].long()] = True
    assert (dys.cpu()[~named] == 7.0).all() and (dys.cpu()[named] == 1.0).all()
    assert (dw.cpu()[~ok] == 0).all()


def test_special_values_travel():
    T, k, H = 3, 2, 16
    ys = torch.ones(T * k, H)
    ys[0, 0], ys[1, 1], ys[2, 2] = float("inf"), float("nan"), -float("inf")
    rows = torch.arange(T * k, dtype=torch.int32).view(T, k)
    y = qgemm.moe_combine(ys.cuda(), rows.cuda(), torch.ones(T, k, device="cuda"), y_dtype=F32).cpu()
    ref = ys.view(T, k, H).sum(1)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(y.nan_to_num(nan=5.0), ref.nan_to_num(nan=5.0))


def test_captured_replayed_and_on_another_stream():
    # one graph replayed over new inputs, beside eager calls on a second stream
    T, k, E, H = 600, 8, 32, 96
    x, ids = torch.zeros(T, H, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")

    def step(stream=None):
        xs, offsets, rows = qgemm.moe_dispatch(x, ids, E, stream=stream)
        return offsets, rows, qgemm.moe_combine(xs, rows, w, y_dtype=F32, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2, 3):
        ids_h, x_h, w_h = routing(T, k, E, seed=seed), randn(T, H, seed=seed), randn(T, k, seed=seed + 9)
        ids.copy_(ids_h), x.copy_(x_h), w.copy_(w_h)
        torch.cuda.synchronize()
        graph.replay()
        other = step(stream=side)
        torch.cuda.synchronize()
        off_ref, rows_ref = maps(ids_h, E)
        for offsets, rows, y in (got, other):
            assert np.array_equal(offsets.cpu().numpy(), off_ref)
            assert np.array_equal(rows.cpu().numpy(), rows_ref)
        assert torch.equal(got[2], other[2])
        ref = x_h.double() * w_h.double().sum(1, keepdim=True)
        mag = x_h.double().abs() * w_h.double().abs().sum(1, keepdim=True)
        assert ((got[2].cpu().double() - ref).abs() <= (k + 1) * U * mag).all()


def test_rows_past_two_to_the_31_elements():
    # 1.2 million sorted rows of 2048: offsets that pass 32 bits, in elements and in bytes
    T, k, H, E = 150000, 8, 2048, 16
    assert T * k * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    x = torch.randn(T, H, device="cuda", generator=g).to(BF16)
    xs, off, rows = qgemm.moe_dispatch(x, ids, E)
    assert int(off[-1]) == T * k
    t = torch.cat([torch.arange(0, 40), torch.arange(T - 40, T), torch.arange(0, T, 1499)]).cuda()
    at = rows[t].long()
    assert int(at.max()) * H > 2 ** 31
    assert torch.equal(xs[at.reshape(-1)].view(-1, k, H), x[t][:, None, :].expand(-1, k, -1))
    w = torch.rand(T, k, device="cuda", generator=g)
    y = qgemm.moe_combine(xs, rows, w)[t].double()
    ref = x[t].double() * w[t].double().sum(1, keepdim=True)
    mag = x[t].double().abs() * w[t].double().sum(1, keepdim=True)
    assert ((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * k * U * mag).all()
    dys, dw = qgemm.moe_combine_grad(x, xs, rows, w)
    want = x[t].double()[:, None, :] * w[t].double()[:, :, None]
    assert ((dys[at.reshape(-1)].view(-1, k, H).double() - want).abs() <= (2.0 ** -8 + U) * (1 + U) * want.abs()).all()
    sq = (x[t].double() ** 2).sum(1, keepdim=True)
    assert ((dw[t].double() - sq).abs() <= H * U * sq).all()
