"""Routed int8 products under offsets that no routing gives: every access stays inside the buffers and the
rows that are well described are right."""
import pytest
import torch

from block_quantized_weight_qgemm_b200 import build, inputs, qgemm

pytestmark = pytest.mark.gpu

ERR_ARG = 10  # QGEMM_ERR_DEVICE_ARG


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    qgemm.lib()
    qgemm.device_status(reset=True)
    yield
    assert qgemm.device_status(reset=True) == qgemm.OK


def table(E, N, K):
    w = [qgemm.i8_pack(inputs.weights(N, K, seed=i).cuda()) for i in range(2)]
    return qgemm.I8ExpertTable([w[e % 2] for e in range(E)]), w


@pytest.mark.parametrize("E", [2, 7, 600])
def test_falling_offsets(E):
    # 0, M, 0, M, ...: every other expert owns all rows, the last of them writes what is compared
    M, N, K = 300, 140, 272
    tab, w = table(E, N, K)
    x = inputs.activations(M, K, seed=E).cuda()
    off = torch.tensor([0, M] * E, dtype=torch.int32, device="cuda")[:E + 1]
    y = qgemm.i8_moe_run(x, off, tab, M)
    h = qgemm.i8_moe_gate_up(x, off, tab, tab, M)
    assert torch.equal(y, qgemm.i8_run(x, w[0]))   # experts 0, 2, 4, ... hold the same weights
    assert torch.equal(h, qgemm.i8_moe_gate_up(x, torch.tensor([0, M], dtype=torch.int32, device="cuda"),
                                               *[qgemm.I8ExpertTable(w[:1])] * 2, M))


def test_more_units_than_clusters():
    # two rows claimed by four of seven experts, where a cluster would take each unit
    M, N, K, E = 2, 140, 2048, 7
    tab, w = table(E, N, K)
    x = inputs.activations(M, K, seed=5).cuda()
    y = torch.full((M, N), 7.0, device="cuda")
    qgemm.i8_moe_run(x, torch.tensor([0, M] * 4, dtype=torch.int32, device="cuda"), tab, M, y=y)
    assert qgemm.device_status(reset=True) == ERR_ARG
    assert bool((y == 7).all())
    qgemm.i8_moe_run(x, torch.tensor([0, 0, 0, M, 0, M, M, M], dtype=torch.int32, device="cuda"), tab, M, y=y)
    assert qgemm.device_status(reset=True) == qgemm.OK
    assert torch.equal(y, qgemm.i8_run(x, w[0]))  # experts 2 and 4 claim the rows, 3 ends before it begins


def test_more_units_than_an_int_counts():
    # 4096 experts of which every other one claims all of 300 million rows: 2.4e9 units
    M, N, K, E = 300_000_000, 1, 16, 4096
    assert E // 2 * (M // 256) > 2 ** 31
    tab, _ = table(E, N, K)
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    y = torch.full((M, N), 7.0, device="cuda")
    off = torch.tensor([0, M] * E, dtype=torch.int32, device="cuda")[:E + 1]
    qgemm.i8_moe_run(x, off, tab, M, y=y)
    assert qgemm.device_status(reset=True) == ERR_ARG
    assert bool((y == 7).all())
    # the same call with offsets in order is served
    off = torch.full((E + 1,), M, dtype=torch.int32, device="cuda")
    off[0] = 0
    qgemm.i8_moe_run(x, off, tab, M, y=y)
    assert qgemm.device_status(reset=True) == qgemm.OK
    assert bool((y == y[0]).all()) and float(y[0]) != 7.0
