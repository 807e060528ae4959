"""One workspace for every width: the size given for M rows is enough for any call of fewer."""
import pytest
import torch

from block_quantized_weight_qgemm_b200 import build as qbuild
from block_quantized_weight_qgemm_b200 import inputs, qgemm

BIG = 1 << 40
ALIGN, WORKSPACE = 5, 6
U = 2.0 ** -24 * 1.01


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qgemm.lib()


def refused(lib, M, N, K, nbytes, routed=False):
    """The status of a call with a workspace of nbytes.  Its address is misaligned, which is looked at after the
    size: no call gets as far as the device."""
    if routed:
        return lib.qgemm_i8_moe_run(16, M, K, 4, 16, M, 16, 16, N, 16, 0, 24, nbytes, None)
    return lib.qgemm_i8_run(16, M, K, 16, 16, N, 16, 0, 24, nbytes, None)


SHAPES = [(10240, 20480), (9600, 8192), (17408, 5120), (5120, 17408), (512, 1024), (512, 2048), (20224, 2048),
          (11000, 12288), (6500, 33008), (300, 1152), (300, 1168), (1, 131072), (130, 16), (40000, 1040)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("routed", [False, True])
def test_a_workspace_serves_every_narrower_call(lib, N, K, routed):
    size = qgemm.i8_moe_workspace_size if routed else qgemm.i8_workspace_size
    widths = sorted(set(range(1, 41)) | set(range(41, 700, 7)) | {255, 256, 257, 384, 385, 1024, 1791, 1792, 1793, 2048, 7235})
    sizes = [size(N, K, M) for M in widths]
    assert sizes == sorted(sizes)
    # (a call's own need is at most the size of its own width, so with sizes in order every pair is covered)
    for M, n in zip(widths, sizes):
        assert refused(lib, M, N, K, n, routed) == ALIGN, M
    assert refused(lib, 1, N, K, sizes[-1], routed) == ALIGN
    assert refused(lib, 2048, N, K, 2048 * K - 1, routed) == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(10240, 20480), (9600, 8192), (300, 2064)])
def test_one_workspace_over_the_widths(lib, N, K):
    # runs, splits of a last round and neither, in one buffer of the widest call's size
    widths = [257, 1, 256, 33, 32, 64, 300, 9]
    ws = torch.empty(qgemm.i8_workspace_size(N, K, max(widths)), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(N)
    rm = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) + 0.5
    w = qgemm.i8_repack_rowmajor(rm, sw)
    cols = torch.from_numpy(inputs.sample_rows(N, 200))
    p, sc = rm[cols.cuda()].cpu().double(), sw[cols.cuda()].cpu().double()
    x = inputs.activations(max(widths), K, seed=K)
    s = x.abs().amax(1).float() * (torch.ones(()) / 127)
    q = torch.round(x.double() / s.double()[:, None])
    xd = x.cuda()
    ys = [qgemm.i8_run(xd[:M], w, workspace=ws) for M in widths]
    torch.cuda.synchronize()
    for M, y in zip(widths, ys):
        # the integer sum is exact; fp32(sum) * sw * sx rounds three times
        ref = (q[:M] @ p.t()) * sc * s[:M].double()[:, None]
        assert ((y[:, cols.cuda()].cpu().double() - ref).abs() <= 3 * U * (1 + 3 * U) * ref.abs()).all()
