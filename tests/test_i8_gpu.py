"""The int8 products against their definition in 64 bits: the row quantisation and the packing code
for code, qgemm_i8_run, the routed forms, and a routed layer run through the whole chain.

Tolerances are counted in roundings: the integer sum is exact; y = fp32(sum) * sw * sx rounds three
times (u = 2^-24 each), then once to the output's type (eps / 2)."""
import numpy as np
import pytest
import torch

from block_quantized_weight_qgemm_b200 import inputs, qgemm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24 * 1.01
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_quantized_weight_qgemm_b200 import build
    build.build()
    qgemm.lib()
    qgemm.device_status(reset=True)
    yield
    assert qgemm.device_status(reset=True) == qgemm.OK


def half(dtype):
    return torch.finfo(dtype).eps / 2


def quantise(a):
    """(codes float64, scales float32) of the rows of a finite array, by the definition."""
    a = a.double()
    s = a.abs().amax(1).float() * (torch.ones(()) / 127)
    q = torch.round(a / torch.where(s > 0, s, torch.ones_like(s)).double()[:, None])
    return q.clamp(-127, 127), s


def check(y, q, sx, p, sw):
    ref = (q @ p.t()) * sw.double()[None, :] * sx.double()[:, None]
    tol = (half(y.dtype) + 3 * U) * (1 + 3 * U) * ref.abs()
    assert torch.isfinite(y).all()
    assert ((y.cpu().double() - ref).abs() <= tol).all()


def tile_major(codes):
    """The packed layout of int8 codes [N, K], from the header's description."""
    N, K = codes.shape
    T, C = -(-N // 128), -(-K // 128)
    full = torch.zeros(T * 128, C * 128, dtype=torch.int8)
    full[:N, :K] = codes
    grp = full.view(T, 128, C, 8, 16).permute(0, 2, 1, 3, 4)
    out = torch.empty_like(grp.contiguous())
    for r in range(128):
        out[:, :, r, [g ^ (r & 7) for g in range(8)], :] = grp[:, :, r]
    return out.reshape(-1).view(torch.uint8)


# ---- quantisation -----------------------------------------------------------------------

def bf16_from_bits(bits):
    return torch.from_numpy(np.asarray(bits, dtype=np.uint16).view(np.int16)).view(BF16)


@pytest.mark.parametrize("top", [127, 254, 1, 60, 40])  # the row maximum's exponent field
def test_every_quotient_rounds_as_the_exact_one(top):
    # row i has maximum 1.i * 2^(top - 127); its other elements are every bf16 value of the ten
    # binades below and the same negated, so that every quotient of that maximum occurs
    rows = []
    for i in range(128):
        mx = (top << 7) | i
        vals = np.arange(max(0, mx - 10 * 128), mx + 1)
        vals = np.concatenate([vals, vals | 0x8000])
        rows.append(np.pad(vals, (0, 2576 - len(vals))))
    x = bf16_from_bits(np.stack(rows))
    codes, scales = qgemm.i8_quant_x(x.cuda())
    q, s = quantise(x)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.cpu().double(), q)


def test_ties_go_to_even():
    # maximum 127 * 2^e: the scale is 2^e and (n + 1/2) 2^e lies halfway between two codes
    n = torch.arange(-127, 127).double()
    x = torch.cat([n + 0.5, torch.tensor([127.0, -127.0])])[None].repeat(3, 1) * torch.tensor([[1.0], [2.0 ** -100], [2.0 ** 90]])
    x = x.to(BF16)
    codes, scales = qgemm.i8_quant_x(x.cuda())
    assert torch.equal(scales.cpu(), torch.tensor([1.0, 2.0 ** -100, 2.0 ** 90]))
    assert torch.equal(codes.cpu()[:, :254].double(), torch.round(n + 0.5)[None].repeat(3, 1))


@pytest.mark.parametrize("M,K", [(1, 16), (3, 32), (401, 16), (777, 256), (300, 272), (1001, 512), (600, 1024), (500, 2048), (401, 2064), (1, 17408), (5, 8208), (2, 131072), (300, 144)])
def test_quant_rows(M, K):
    x = inputs.activations(M, K, seed=M + K)
    codes, scales = qgemm.i8_quant_x(x.cuda())
    q, s = quantise(x)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu().double(), q)


def special_rows(K):
    x = inputs.activations(10, K, seed=5).float()
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, K - 1] = float("nan")
    x[4, 0] = -float("inf")
    x[5] = x[5] * 2.0 ** -133 * 8            # subnormals of bf16
    x[6] = 0
    x[6, 7] = 2.0 ** -133                    # the smallest one
    x[7, 1], x[7, 2] = 3.3e38, 1e-38
    x[8] *= 1e-36
    return x.to(BF16)


@pytest.mark.parametrize("K", [272, 2080])  # quantised in the product's kernel, and in one of its own
def test_special_rows(K):
    x = special_rows(K)
    codes, scales = qgemm.i8_quant_x(x.cuda())
    codes, scales = codes.cpu().double(), scales.cpu()
    bad = torch.tensor([2, 3, 4])
    ok = torch.tensor([0, 1, 5, 6, 7, 8, 9])
    q, s = quantise(x[ok])
    assert torch.equal(scales[ok], s) and torch.equal(codes[ok], q)
    assert torch.isnan(scales[bad]).all() and (codes[bad] == 0).all()
    # in the product: a row with an infinity or NaN is NaN, the others do not see it
    W = inputs.weights(130, K)
    w = qgemm.i8_pack(W.cuda())
    p, sw = quantise(W)
    y = qgemm.i8_run(x.cuda(), w).cpu()
    assert torch.isnan(y[bad]).all() and (y[1] == 0).all()
    # subnormal results: one step of 2^-149 in place of the relative rounding
    ref = (q @ p.t()) * sw.double() * s.double()[:, None]
    assert ((y[ok].double() - ref).abs() <= 4 * U * ref.abs() + 2.0 ** -148).all()
    assert torch.equal(y[0], qgemm.i8_run(x[:1].cuda(), w).cpu()[0])


@pytest.mark.parametrize("N,K", [(1, 16), (127, 128), (128, 144), (300, 1040), (513, 2048)])
def test_pack_and_repack(N, K):
    W = inputs.weights(N, K, seed=N)
    W[N // 2] = 0
    w = qgemm.i8_pack(W.cuda())
    p, s = quantise(W)
    assert torch.equal(w.scales.cpu(), s)
    assert torch.equal(w.codes.cpu(), tile_major(p.to(torch.int8)))
    # a checkpoint's codes, -128 among them, from rows with a stride
    rm = torch.randint(-128, 128, (N, K + 48), dtype=torch.int8, generator=torch.Generator().manual_seed(N))
    r = qgemm.i8_repack_rowmajor(rm.cuda()[:, :K], s.cuda())
    assert torch.equal(r.codes.cpu(), tile_major(rm[:, :K]))


def test_pack_special_channels():
    W = inputs.weights(4, 64)
    W[1, 5], W[2, 0] = float("nan"), float("inf")
    w = qgemm.i8_pack(W.cuda())
    y = qgemm.i8_run(inputs.activations(3, 64).cuda(), w).cpu()
    assert torch.isnan(y[:, 1:3]).all() and torch.isfinite(y[:, [0, 3]]).all()


# ---- the product ------------------------------------------------------------------------

_W = {}


def weight(N, K):
    if (N, K) not in _W:
        W = inputs.weights(N, K, seed=N + K)
        _W[N, K] = (qgemm.i8_pack(W.cuda()),) + quantise(W)
    return _W[N, K]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,K", [(1, 16), (64, 128), (129, 144), (300, 1040), (640, 2048), (128, 17408)])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 100, 128, 129, 255, 256, 257, 300, 384, 385, 513])
def test_run(M, N, K, dtype):
    w, p, sw = weight(N, K)
    x = inputs.activations(M, K, seed=M)
    q, sx = quantise(x)
    check(qgemm.i8_run(x.cuda(), w, y_dtype=dtype), q, sx, p, sw)


def test_largest_sum_is_exact():
    # K = 131072 of codes +-127 against -128: the sums reach +-2130706432, inside int32
    K = 131072
    x = torch.ones(3, K, dtype=BF16)
    x[1] = -1
    x[2, ::2] = -1
    rm = torch.full((130, K), -128, dtype=torch.int8)
    rm[1] = 127
    w = qgemm.i8_repack_rowmajor(rm.cuda(), torch.ones(130, device="cuda"))
    y = qgemm.i8_run(x.cuda(), w).cpu().double()
    sums = torch.tensor([[-128.0] * 130, [128.0] * 130, [0.0] * 130]).double() * 127 * K
    sums[0, 1], sums[1, 1] = 127.0 * 127 * K, -127.0 * 127 * K
    s = float(torch.ones(()) / 127)
    assert ((y - sums * s).abs() <= 3 * U * (sums * s).abs()).all()


def test_rows_do_not_depend_on_the_width():
    # exact sums: one row's result is the same bits at every width and position
    w, _, _ = weight(640, 2048)
    x = inputs.activations(700, 2048, seed=77).cuda()
    full = qgemm.i8_run(x, w).cpu()
    for a, b in ((0, 1), (5, 21), (3, 67), (100, 228), (100, 229), (0, 256), (10, 267), (0, 699)):
        assert torch.equal(qgemm.i8_run(x[a:b].contiguous(), w).cpu(), full[a:b]), (a, b)


@pytest.mark.parametrize("N,K", [(17408, 5120), (5120, 17408)])
@pytest.mark.parametrize("M", [1, 64, 200, 2048])
def test_27b_shapes_on_sampled_channels(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) * 1e-3 + 1e-4
    w = qgemm.i8_repack_rowmajor(rm, sw)
    x = inputs.activations(M, K, seed=M)
    y = qgemm.i8_run(x.cuda(), w)
    rows = torch.from_numpy(inputs.sample_rows(M, 40))
    cols = torch.from_numpy(inputs.sample_rows(N, 200))
    q, sx = quantise(x[rows])
    check(y[rows.cuda()][:, cols.cuda()], q, sx, rm[cols.cuda()].cpu().double(), sw[cols.cuda()].cpu())


# ---- routed -----------------------------------------------------------------------------

N, K = 300, 272
COUNTS = [0, 5, 17, 1, 0, 64, 3, 300, 33, 129, 0]


def offsets_of(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


@pytest.fixture(scope="module")
def experts():
    out = []
    for j in range(2):
        Ws = [inputs.weights(N, K, seed=100 * j + e) for e in range(len(COUNTS))]
        out.append(([qgemm.i8_pack(W.cuda()) for W in Ws], [quantise(W) for W in Ws]))
    return out


def h_check(h, g, u):
    """h = bf16(g / (1 + exp(-g)) * u).  g and u carry 3 roundings each; with sig = 1/(1 + e^-g),
    d ln h / d ln g = 1 + g (1 - sig).  The exponential is off by (2 + 1.173 |g|) steps (its
    documented bound), of which the quotient sees the share 1 - sig; sum, quotient and product round
    once each."""
    sig = 1 / (1 + torch.exp(-g))
    ref = g * sig * u
    rel = 3 * U * (1 + (1 + g * (1 - sig)).abs()) + (1 - sig) * (2 + 1.173 * g.abs()) * 2 * U + 3 * U
    assert ((h.cpu().double() - ref).abs() <= (2.0 ** -8 + rel * 1.01) * ref.abs() + 1e-37).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_moe_run(experts, dtype):
    ws, refs = experts[0]
    M = sum(COUNTS) + 9                       # nine rows that belong to no expert
    x = inputs.activations(M, K, seed=3)
    off = offsets_of(COUNTS)
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    qgemm.i8_moe_run(x.cuda(), off, qgemm.I8ExpertTable(ws), max_rows=max(COUNTS), y=y)
    o = off.tolist()
    for e, (p, sw) in enumerate(refs):
        if o[e] < o[e + 1]:
            check(y[o[e]:o[e + 1]], *quantise(x[o[e]:o[e + 1]]), p, sw)
    assert (y[o[-1]:] == 7.0).all()


def test_moe_gate_up(experts):
    (gw, gr), (uw, ur) = experts
    M = sum(COUNTS)
    x = inputs.activations(M, K, seed=4)
    off = offsets_of(COUNTS)
    h = qgemm.i8_moe_gate_up(x.cuda(), off, qgemm.I8ExpertTable(gw), qgemm.I8ExpertTable(uw), max(COUNTS))
    o = off.tolist()
    for e in range(len(COUNTS)):
        if o[e] < o[e + 1]:
            q, sx = quantise(x[o[e]:o[e + 1]])
            g, u = [(q @ p.t()) * s.double() * sx.double()[:, None] for p, s in (gr[e], ur[e])]
            h_check(h[o[e]:o[e + 1]], g, u)


def test_moe_max_rows_and_bad_offsets(experts):
    # rows past max_rows are not computed; offsets outside [0, M] or falling are clamped
    ws, refs = experts[0]
    tab = qgemm.I8ExpertTable(ws)
    M = sum(COUNTS)
    x = inputs.activations(M, K, seed=6)
    off = offsets_of(COUNTS)
    full = qgemm.i8_moe_run(x.cuda(), off, tab, max_rows=300)
    y = torch.full((M, N), 7.0, device="cuda")
    qgemm.i8_moe_run(x.cuda(), off, tab, max_rows=20, y=y)
    o = off.tolist()
    for e in range(len(COUNTS)):
        n = min(20, o[e + 1] - o[e])
        assert torch.equal(y[o[e]:o[e] + n], full[o[e]:o[e] + n])
        assert (y[o[e] + n:o[e + 1]] == 7.0).all()
    bad = off.clone()
    bad[-1], bad[0], bad[4] = M + 1000, -5, bad[3] - 2    # an expert that ends before it begins
    y2 = torch.full((M, N), 7.0, device="cuda")
    qgemm.i8_moe_run(x.cuda(), bad, tab, max_rows=300, y=y2)
    torch.cuda.synchronize()
    assert torch.equal(y2[o[7]:o[8]], full[o[7]:o[8]])


def test_moe_bad_table_entry_is_refused_on_the_device(experts):
    ws, refs = experts[0]
    tab = qgemm.I8ExpertTable(ws)
    tab.codes[1], tab.codes[2], tab.scales[3], tab.scales[5] = 0, tab.codes[2] + 8, 0, tab.scales[5] + 2
    M = sum(COUNTS)
    x = inputs.activations(M, K, seed=8)
    off = offsets_of(COUNTS)
    y = torch.full((M, N), 7.0, device="cuda")
    qgemm.i8_moe_run(x.cuda(), off, tab, max_rows=300, y=y)
    assert qgemm.device_status(reset=True) == 10  # QGEMM_ERR_DEVICE_ARG
    o = off.tolist()
    for e in range(len(COUNTS)):
        rows = slice(o[e], o[e + 1])
        if e in (1, 2, 3, 5):
            assert (y[rows] == 7.0).all()
        elif COUNTS[e]:
            check(y[rows], *quantise(x[rows]), *refs[e])


def test_moe_one_expert_equals_run(experts):
    ws, _ = experts[0]
    x = inputs.activations(400, K, seed=9).cuda()
    tab = qgemm.I8ExpertTable(ws[:1])
    for M in (1, 20, 130, 400):
        xm = x[:M].contiguous()
        assert torch.equal(qgemm.i8_moe_run(xm, offsets_of([M]), tab, M), qgemm.i8_run(xm, ws[0]))


# ---- a routed layer ---------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["i8", "nvfp4", "mixed"])
def test_routed_layer(fmt):
    """dispatch -> experts' fused gate+up -> down -> combine, and the way back through the two
    gradients, as a layer runs it: padded tokens, an expert without rows, the library's other
    weight formats beside int8.  Each stage is held to the definition applied to that stage's
    own input."""
    T, k, E, H, F = 50, 3, 8, 256, 128
    g = torch.Generator().manual_seed(1)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int()  # expert 7: no rows
    ids[40:43] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    x = inputs.activations(T, H, seed=2)
    Wg, Wu, Wd = [[inputs.weights(n, m, seed=10 * i + e) for e in range(E)]
                  for i, (n, m) in enumerate(((F, H), (F, H), (H, F)))]
    xs, off, rows = qgemm.moe_dispatch(x.cuda(), ids.cuda(), E)
    live = int(off[-1])
    assert live == (T - 3) * k
    mr = int((off[1:] - off[:-1]).max())
    if fmt == "nvfp4":
        tabs = [qgemm.ExpertTable([qgemm.pack("nvfp4", W.cuda()) for W in Ws]) for Ws in (Wg, Wu, Wd)]
        h = qgemm.moe_gate_up(xs, off, tabs[0], tabs[1], mr)
        ys = qgemm.moe_run(h, off, tabs[2], mr)
    else:
        tabs = [qgemm.I8ExpertTable([qgemm.i8_pack(W.cuda()) for W in Ws]) for Ws in (Wg, Wu, Wd)]
        h = qgemm.i8_moe_gate_up(xs, off, tabs[0], tabs[1], mr)
        if fmt == "mixed":
            ys = qgemm.moe_run(h, off, qgemm.ExpertTable([qgemm.pack("q8_0", W.cuda()) for W in Wd]), mr)
        else:
            ys = qgemm.i8_moe_run(h, off, tabs[2], mr)
            o = off.tolist()
            for e in range(E):
                if o[e] < o[e + 1]:
                    q, sx = quantise(xs[o[e]:o[e + 1]].cpu())
                    ge, ue = [(q @ p.t()) * s.double() * sx.double()[:, None]
                              for p, s in (quantise(Wg[e]), quantise(Wu[e]))]
                    h_check(h[o[e]:o[e + 1]], ge, ue)
                    check(ys[o[e]:o[e + 1]], *quantise(h[o[e]:o[e + 1]].cpu()), *quantise(Wd[e]))
    y = qgemm.moe_combine(ys, rows, w.cuda()).cpu().double()
    yd, r = ys[:live].cpu().double(), rows.cpu().long()
    terms = torch.where((r >= 0)[:, :, None], yd[r.clamp(min=0)] * w.double()[:, :, None], torch.zeros(1).double())
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert ((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * k * U * mag).all()
    assert (y[40:43] == 0).all()
    # per token, the whole layer against fp32 weights: quantisation error alone is left (8-bit
    # codes on both sides of each product leave below 2 %, 4-bit codes below 30 %)
    full = torch.zeros(T, H).double()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                gg, uu = Wg[e].double() @ x[t].double(), Wu[e].double() @ x[t].double()
                full[t] += float(w[t, j]) * (Wd[e].double() @ (gg * torch.sigmoid(gg) * uu))
    assert float((y - full).norm() / full.norm()) < (0.3 if fmt == "nvfp4" else 0.05)
    # the way back
    dy = inputs.activations(T, H, seed=12).cuda()
    dys, dw = qgemm.moe_combine_grad(dy, ys, rows, w.cuda())
    want = torch.where((r >= 0)[:, :, None], dy.cpu().double()[:, None, :] * w.double()[:, :, None], torch.zeros(1).double())
    got = dys.cpu().double()[r.clamp(min=0)]
    assert ((got - want).abs() <= 2 * U * want.abs())[r >= 0].all()
    t2 = dy.cpu().double()[:, None, :] * torch.where((r >= 0)[:, :, None], yd[r.clamp(min=0)], torch.zeros(1).double())
    assert ((dw.cpu().double() - t2.sum(2)).abs() <= H * U * t2.abs().sum(2)).all()
    dx = qgemm.moe_dispatch_grad(xs, rows, dx_dtype=F32).cpu().double()
    assert ((dx - x.double() * (r >= 0).sum(1, keepdim=True)).abs() <= k * U * x.double().abs() * k).all()


def test_captured_gemm_shares_no_state_between_graphs():
    # two graphs over one workspace, replayed in turn on one stream with new inputs
    w, p, sw = weight(640, 2048)
    ws = torch.empty(max(qgemm.i8_workspace_size(640, 2048, m) for m in (40, 400)), dtype=torch.uint8, device="cuda")
    xs = [torch.zeros(m, 2048, dtype=BF16, device="cuda") for m in (40, 400)]
    for x in xs:
        qgemm.i8_run(x, w, workspace=ws)
    graphs, outs = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(qgemm.i8_run(x, w, workspace=ws))
    for seed in (1, 2):
        hs = [inputs.activations(x.shape[0], 2048, seed=seed + i) for i, x in enumerate(xs)]
        for x, h in zip(xs, hs):
            x.copy_(h)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for h, y in zip(hs, outs):
            check(y, *quantise(h), p, sw)


@pytest.mark.parametrize("M", [1, 16, 40, 129, 256])
@pytest.mark.parametrize("N,K", [(100, 1280), (640, 1664), (1300, 2048), (2800, 1024), (5000, 1152), (5700, 1792),
                                 (9400, 896), (9500, 1536), (10000, 16400), (6500, 33000 // 16 * 16), (11000, 12288)])
def test_k_split_over_clusters_and_not(M, N, K):
    # from 1 to 75 channel tiles: clusters of eight CTAs down to one share a tile's K, in uneven runs
    g = torch.Generator(device="cuda").manual_seed(N + M)
    rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) + 0.5
    x = inputs.activations(M, K, seed=M)
    q, sx = quantise(x)
    y = qgemm.i8_run(x.cuda(), qgemm.i8_repack_rowmajor(rm, sw))
    check(y, q, sx, rm.cpu().double(), sw.cpu())


@pytest.mark.parametrize("M,N,K", [(1000, 20000, 512), (257, 9600, 2048), (450, 9600, 2048), (600, 1000, 8192),
                                   (64, 19000, 2048)])
def test_last_round_split_over_k(M, N, K):
    # full rounds of tiles, then a last round whose tiles are split over K and summed afterwards
    g = torch.Generator(device="cuda").manual_seed(N + M)
    rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) + 0.5
    x = inputs.activations(M, K, seed=M)
    y = qgemm.i8_run(x.cuda(), qgemm.i8_repack_rowmajor(rm, sw))
    q, sx = quantise(x)
    check(y, q, sx, rm.cpu().double(), sw.cpu())


@pytest.mark.parametrize("T,k,E", [(1, 1, 2), (1, 6, 64), (2, 4, 300), (7, 3, 5)])
def test_few_routed_rows(T, k, E):
    # a unit per expert and tile at most, each shared by a cluster
    g = torch.Generator().manual_seed(T)
    Nf, Kf = 256, 1040
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    x = inputs.activations(T, Kf, seed=k)
    xs, off, _ = qgemm.moe_dispatch(x.cuda(), ids.cuda(), E)
    Ws = [inputs.weights(Nf, Kf, seed=i) for i in range(4)]
    packed, refs = [qgemm.i8_pack(W.cuda()) for W in Ws], [quantise(W) for W in Ws]
    gate = qgemm.I8ExpertTable([packed[e % 4] for e in range(E)])
    up = qgemm.I8ExpertTable([packed[(e + 1) % 4] for e in range(E)])
    o = off.tolist()
    mr = max(b - a for a, b in zip(o, o[1:]))
    y = qgemm.i8_moe_run(xs, off, gate, mr)
    h = qgemm.i8_moe_gate_up(xs, off, gate, up, mr)
    for e in range(E):
        if o[e] < o[e + 1]:
            q, sx = quantise(xs[o[e]:o[e + 1]].cpu())
            check(y[o[e]:o[e + 1]], q, sx, *refs[e % 4])
            gg, uu = [(q @ p.t()) * s.double() * sx.double()[:, None] for p, s in (refs[e % 4], refs[(e + 1) % 4])]
            h_check(h[o[e]:o[e + 1]], gg, uu)


@pytest.mark.parametrize("T", [40, 2100])
def test_routings_one_after_another(T):
    # the products read the offsets early in their launch: with no wait between the steps, every one sees
    # its own routing (one launch dispatches 40 tokens, two 2100)
    k, E, H, F, rounds = 4, 16, 256, 128, 12
    g = torch.Generator().manual_seed(T)
    tab8 = qgemm.I8ExpertTable([qgemm.i8_pack(inputs.weights(F, H, seed=e).cuda()) for e in range(E)])
    tab4 = qgemm.ExpertTable([qgemm.pack("nvfp4", inputs.weights(F, H, seed=e).cuda()) for e in range(E)])
    x = inputs.activations(T, H, seed=1).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    like = [torch.rand(E, generator=g).pow(4) for _ in range(rounds)]     # the first experts of each differ
    ids = [torch.multinomial(p, T * k, replacement=True, generator=g).view(T, k).int().cuda() for p in like]

    def step(i):
        xs, off, rows = qgemm.moe_dispatch(x, ids[i], E)
        return (qgemm.moe_combine(qgemm.i8_moe_run(xs, off, tab8, T * k), rows, w, y_dtype=F32),
                qgemm.moe_combine(qgemm.moe_run(xs, off, tab4, 200), rows, w, y_dtype=F32) if T == 40 else None)

    apart = []
    for i in range(rounds):
        apart.append(step(i))
        torch.cuda.synchronize()
    together = [step(i) for i in range(rounds)]
    torch.cuda.synchronize()
    for a, b in zip(apart, together):
        assert torch.equal(a[0], b[0]) and (a[1] is None or torch.equal(a[1], b[1]))


def test_no_token_has_an_expert():
    ids = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    x = inputs.activations(5, 256).cuda()
    xs, off, rows = qgemm.moe_dispatch(x, ids, 4, xs=torch.zeros(15, 256, dtype=BF16, device="cuda"))
    tab = qgemm.I8ExpertTable([qgemm.i8_pack(inputs.weights(128, 256, seed=e).cuda()) for e in range(4)])
    y = torch.full((15, 128), 7.0, device="cuda")
    qgemm.i8_moe_run(xs, off, tab, 15, y=y)
    h = torch.full((15, 128), 7.0, dtype=BF16, device="cuda")
    qgemm.i8_moe_gate_up(xs, off, tab, tab, 15, h=h)
    assert off.tolist() == [0] * 5 and (y == 7).all() and (h == 7).all() and (xs == 0).all()
    assert (qgemm.moe_combine(y, rows, torch.ones(5, 3, device="cuda")) == 0).all()


def test_on_a_stream_of_its_own():
    # x is made on a side stream and the product runs there; its workspace is the call's own
    w, p, sw = weight(640, 2048)
    side = torch.cuda.Stream()
    xs = [inputs.activations(33, 2048, seed=s) for s in range(6)]
    pinned = [x.pin_memory() for x in xs]
    ys = []
    for h in pinned:
        with torch.cuda.stream(side):
            x = h.cuda(non_blocking=True)
        x.record_stream(side)
        ys.append(qgemm.i8_run(x, w, stream=side))
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # takes freed blocks, on this stream
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        check(y, *quantise(x), p, sw)


def test_outputs_and_codes_past_two_to_the_31():
    # y of 2.3e9 elements, and x of 2.3e9 codes
    g = torch.Generator(device="cuda").manual_seed(0)
    for M, N, K in ((140000, 16400, 64), (140000, 130, 16400)):
        assert M * max(N, K) > 2 ** 31
        rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
        sw = torch.rand(N, device="cuda", generator=g) + 0.5
        x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
        y = qgemm.i8_run(x, qgemm.i8_repack_rowmajor(rm, sw), y_dtype=BF16)
        t = torch.cat([torch.arange(0, 9), torch.arange(M - 9, M), torch.arange(0, M, 9973)]).cuda()
        check(y[t], *quantise(x[t].cpu()), rm.cpu().double(), sw.cpu())
        off = torch.tensor([0, 70001, M], dtype=torch.int32, device="cuda")
        tab = qgemm.I8ExpertTable([qgemm.i8_repack_rowmajor(rm, sw)] * 2)
        assert torch.equal(qgemm.i8_moe_run(x, off, tab, M, y_dtype=BF16)[t], y[t])
        del x, y


def test_two_streams_at_once():
    # products and sorts of two streams overlap on the device; each has its own buffers
    w, p, sw = weight(640, 2048)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [inputs.activations(m, 2048, seed=m) for m in (7, 64, 700, 33, 300, 5)]
    ids = torch.randint(0, 8, (3000, 4), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    dev_x, dev_ids = [x.cuda() for x in xs], ids.cuda()
    one = qgemm.moe_dispatch(torch.zeros(3000, 64, device="cuda"), dev_ids, 8)
    torch.cuda.synchronize()
    got = []
    for r in range(6):
        for i, x in enumerate(dev_x):
            with torch.cuda.stream(streams[(i + r) % 2]):
                got.append((i, qgemm.i8_run(x, w), qgemm.moe_dispatch(torch.zeros(3000, 64, device="cuda"), dev_ids, 8)))
    torch.cuda.synchronize()
    for i, y, (_, off, rows) in got:
        check(y, *quantise(xs[i]), p, sw)
        assert torch.equal(off, one[1]) and torch.equal(rows, one[2])


def test_a_call_on_another_stream_leaves_freed_blocks_alone():
    # z is freed while a kernel of this stream is still to read it: its block is no scratch (nor output) for a
    # call on another stream, which would write it at once
    w, p, sw = weight(640, 2048)
    x_h = inputs.activations(200, 2048, seed=3)
    x = x_h.cuda()
    side = torch.cuda.Stream()
    nbytes = qgemm.i8_workspace_size(640, 2048, 200)
    y_bytes = 200 * 640 * 4
    torch.cuda.synchronize()
    kept = []
    for n in (nbytes, y_bytes):
        kept.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.empty_cache()
    zs = [torch.full((n,), 90 + i, dtype=torch.uint8, device="cuda") for i, n in enumerate((nbytes, y_bytes))]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for z, k in zip(zs, kept):
        k.copy_(z)
    del zs, z
    y = qgemm.i8_run(x, w, stream=side)
    torch.cuda.synchronize()
    for i, k in enumerate(kept):
        assert (k == 90 + i).all()
    check(y, *quantise(x_h), p, sw)
    with pytest.raises(AssertionError):
        qgemm.i8_run(x_h, w, stream=side)


@pytest.mark.parametrize("M,N,K", [(33, 100, 1040), (97, 513, 4096), (150, 64, 64), (200, 2048, 2048), (300, 1024, 5120),
                                   (385, 129, 1040), (513, 640, 16400), (700, 300, 2960), (1000, 4700, 1040),
                                   (1100, 4700, 1040), (2048, 64, 512), (2050, 130, 272), (4096, 1100, 528),
                                   (450, 9600, 2064), (500, 9400, 1040), (1300, 5000, 1040)])
def test_tiles_of_fewer_rows_and_wide_calls(M, N, K):
    # few channels: tiles of 32 rows and more on many SMs, in clusters or not; wide calls on lone CTAs (up to 148
    # tiles), on pairs, and on pairs with a last round of few tiles split over K
    g = torch.Generator(device="cuda").manual_seed(N + M)
    rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) + 0.5
    x = inputs.activations(M, K, seed=M)
    y = qgemm.i8_run(x.cuda(), qgemm.i8_repack_rowmajor(rm, sw))
    q, sx = quantise(x)
    check(y, q, sx, rm.cpu().double(), sw.cpu())


@pytest.mark.parametrize("n,k", [(300, 272), (640, 1040)])
@pytest.mark.parametrize("counts", [[70] * 7 + [0, 97], [256, 300, 211, 257], [20, 0, 45, 3, 17], [640, 12], [150] * 5,
                                    [1, 500, 0, 0, 3, 2, 90]], ids=str)
def test_moe_tiles_and_boxes(counts, n, k):
    # experts of like and unlike size about the means at which tiles and boxes change
    E, M = len(counts), sum(counts)
    Ws = [[inputs.weights(n, k, seed=10 * e + j) for e in range(E)] for j in range(2)]
    tabs = [qgemm.I8ExpertTable([qgemm.i8_pack(W.cuda()) for W in ws]) for ws in Ws]
    refs = [[quantise(W) for W in ws] for ws in Ws]
    x = inputs.activations(M, k, seed=M)
    off = offsets_of(counts)
    y = qgemm.i8_moe_run(x.cuda(), off, tabs[0], max(counts))
    h = qgemm.i8_moe_gate_up(x.cuda(), off, *tabs, max(counts))
    loose = qgemm.i8_moe_run(x.cuda(), off, tabs[0], M)  # an upper bound of the rows is enough
    assert torch.equal(y, loose)
    o = off.tolist()
    for e in range(E):
        a, b = o[e], o[e + 1]
        if a < b:
            q, sx = quantise(x[a:b])
            check(y[a:b], q, sx, *refs[0][e])
            h_check(h[a:b], *[(q @ p.t()) * s.double() * sx.double()[:, None] for p, s in (refs[0][e], refs[1][e])])


@pytest.mark.parametrize("counts,tiles", [([256, 230, 274, 264], 18), ([129] * 9, 16), ([140, 0, 131, 250, 100], 29),
                                          ([129] * 8 + [700], 16)], ids=str)
def test_gate_up_in_one_set_of_accumulators(counts, tiles):
    # tiles of more than 128 rows, where experts and channels fill the SMs once; the expert of 700 rows makes more
    E, M, n, k = len(counts), sum(counts), tiles * 128 - 5, 144
    Ws = [[inputs.weights(n, k, seed=10 * e + j) for e in range(E)] for j in range(2)]
    tabs = [qgemm.I8ExpertTable([qgemm.i8_pack(W.cuda()) for W in ws]) for ws in Ws]
    refs = [[quantise(W) for W in ws] for ws in Ws]
    x = inputs.activations(M, k, seed=M)
    off = offsets_of(counts)
    h = qgemm.i8_moe_gate_up(x.cuda(), off, *tabs, max(counts))
    o = off.tolist()
    for e in range(E):
        if o[e] < o[e + 1]:
            q, sx = quantise(x[o[e]:o[e + 1]])
            h_check(h[o[e]:o[e + 1]],
                    *[(q @ p.t()) * s.double() * sx.double()[:, None] for p, s in (refs[0][e], refs[1][e])])
