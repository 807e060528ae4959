"""int8 weights written again in place: what holds a weight's addresses (expert tables, captured
graphs) sees the new weights, and the checkpoint's tensors stay the caller's.  The first half needs
no GPU: the entry point is replaced, the buffers are host memory."""
import pytest
import torch

from block_quantized_weight_qgemm_b200 import build as qbuild
from block_quantized_weight_qgemm_b200 import inputs, qgemm

BF16 = torch.bfloat16
U = 2.0 ** -24 * 1.01


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qgemm.lib()


# ---- addresses, with no GPU -------------------------------------------------------------

class FakeLib:
    """Takes the place of the library's handle: notes which buffers a call was given."""

    def __init__(self):
        self.codes = []

    def qgemm_i8_repack_rowmajor(self, N, K, codes_rm, pitch, codes, stream):
        self.codes.append(codes)
        return qgemm.OK


@pytest.fixture
def fake(monkeypatch):
    make = qgemm.I8Weight
    ready = make(40, 32, torch.device("cpu"))
    handle = FakeLib()
    monkeypatch.setattr(qgemm, "lib", lambda: handle)
    monkeypatch.setattr(qgemm, "_device", lambda *t: 0)
    monkeypatch.setattr(qgemm, "_current_device", lambda: 0)
    monkeypatch.setattr(qgemm, "_raw_stream", lambda i: 0)
    return handle, ready


def checkpoint(seed, N=40, K=32):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, (N, K), dtype=torch.int8, generator=g), torch.rand(N, generator=g) + 0.5


def test_repack_into_a_weight_keeps_its_buffers(fake):
    handle, w = fake
    tab = qgemm.I8ExpertTable([w, w])
    at = w.codes.data_ptr(), w.scales.data_ptr()
    for seed in (1, 2, 1):
        rm, s = checkpoint(seed)
        kept = s.clone()
        assert qgemm.i8_repack_rowmajor(rm, s, out=w) is w
        assert (w.codes.data_ptr(), w.scales.data_ptr()) == at and handle.codes[-1] == at[0]
        assert tab.scales.tolist() == [at[1]] * 2
        assert torch.equal(w.scales, kept) and torch.equal(s, kept)


def test_a_weight_is_not_tied_to_its_checkpoint(fake):
    # the first checkpoint's scales are not what a reload writes
    _, w = fake
    (rm, s), (rm2, s2) = checkpoint(3), checkpoint(4)
    qgemm.i8_repack_rowmajor(rm, s, out=w)
    kept = s.clone()
    qgemm.i8_repack_rowmajor(rm2, s2, out=w)
    assert torch.equal(s, kept) and torch.equal(w.scales, s2)
    s2.zero_()
    assert (w.scales > 0).all()


def test_repack_takes_parameters_and_works_in_any_mode(fake):
    _, w = fake
    rm, s = checkpoint(5)
    qgemm.i8_repack_rowmajor(rm, torch.nn.Parameter(s), out=w)
    assert not w.scales.requires_grad and torch.equal(w.scales, s)
    with torch.inference_mode():
        w.scales = torch.empty(40)
    qgemm.i8_repack_rowmajor(rm, s, out=w)  # made in inference mode, written outside it
    assert torch.equal(w.scales, s)


def test_table_holds_the_tensors_of_its_addresses(fake):
    _, w = fake
    tab = qgemm.I8ExpertTable([w])
    held = [t.data_ptr() for pair in tab.buffers for t in pair]
    w.codes, w.scales = torch.empty_like(w.codes), torch.empty_like(w.scales)
    assert held == [tab.codes.tolist()[0], tab.scales.tolist()[0]]
    assert held == [t.data_ptr() for pair in tab.buffers for t in pair]


# ---- results, on the GPU ----------------------------------------------------------------

def quantise(a):
    """(codes float64, scales float32) of the rows of a finite array, by the definition."""
    a = a.double()
    s = a.abs().amax(1).float() * (torch.ones(()) / 127)
    return torch.round(a / s.double()[:, None]).clamp(-127, 127), s


def check(y, x, rm, sw):
    # the integer sum is exact; fp32(sum) * sw * sx rounds three times
    q, sx = quantise(x)
    ref = (q @ rm.double().t()) * sw.double()[None, :] * sx.double()[:, None]
    assert ((y.cpu().double() - ref).abs() <= 3 * U * (1 + 3 * U) * ref.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["repack", "pack"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 272), (200, 640, 2048)])
def test_reload_under_a_table_and_a_graph(M, N, K, how):
    x = inputs.activations(M, K, seed=1)
    xd = x.cuda()
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")

    def load(seed, out=None):
        """(weight, codes, scales) of a checkpoint; its own tensors are dropped at once."""
        if how == "pack":
            W = inputs.weights(N, K, seed=seed)
            return (qgemm.i8_pack(W.cuda(), out=out),) + quantise(W)
        rm, s = checkpoint(seed, N, K)
        return qgemm.i8_repack_rowmajor(rm.cuda(), s.cuda(), out=out), rm, s

    w, rm, s = load(1)
    tab = qgemm.I8ExpertTable([w])
    check(qgemm.i8_run(xd, w), x, rm, s)
    check(qgemm.i8_moe_run(xd, off, tab, M), x, rm, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = qgemm.i8_run(xd, w)
    for seed in (2, 3, 1):
        w2, rm, s = load(seed, out=w)
        assert w2 is w
        taken = [torch.full((N,), 7.0, device="cuda") for _ in range(64)]  # takes any block of scales that was freed
        graph.replay()
        moe, run = qgemm.i8_moe_run(xd, off, tab, M), qgemm.i8_run(xd, w)
        for got in (y, moe, run):
            check(got, x, rm, s)
        assert all((t == 7).all() for t in taken)


@pytest.mark.gpu
def test_reload_from_the_same_checkpoint_again():
    # weights of two checkpoints in turn, in one set of buffers: neither checkpoint is written
    N, K, M = 130, 528, 9
    x = inputs.activations(M, K, seed=2)
    sets = [tuple(t.cuda() for t in checkpoint(seed, N, K)) for seed in (1, 2)]
    kept = [(rm.cpu(), s.cpu()) for rm, s in sets]
    w = qgemm.i8_repack_rowmajor(*sets[0])
    for i in (0, 1, 0, 1, 1, 0):
        qgemm.i8_repack_rowmajor(*sets[i], out=w)
        check(qgemm.i8_run(x.cuda(), w), x, *kept[i])
    assert all(torch.equal(a.cpu(), b) for p, q in zip(sets, kept) for a, b in zip(p, q))


@pytest.mark.gpu
def test_reload_on_a_stream_of_its_own():
    N, K, M = 300, 272, 40
    x = inputs.activations(M, K, seed=3)
    side = torch.cuda.Stream()
    xd = x.cuda()
    sets = [tuple(t.cuda() for t in checkpoint(seed, N, K)) for seed in range(4)]
    w = qgemm.i8_repack_rowmajor(*sets[0])
    torch.cuda.synchronize()
    ys = []
    for rm, s in sets:
        qgemm.i8_repack_rowmajor(rm, s, out=w, stream=side)
        ys.append(qgemm.i8_run(xd, w, stream=side))
    torch.cuda.synchronize()
    for y, (rm, s) in zip(ys, sets):
        check(y, x, rm.cpu(), s.cpu())
