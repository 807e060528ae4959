"""The gathered rows of qgemm_moe_dispatch at slot counts that the one-launch kernel leaves to the sort
and the gather, bit for bit: every vector width of the row mover, rows longer than a block of it."""
import pytest
import torch

from block_quantized_weight_qgemm_b200 import build, qgemm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    qgemm.lib()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 16, 100, 257, 1001, 2048, 2056, 5120, 20000])
@pytest.mark.parametrize("T,k", [(1500, 6), (4500, 2)])  # S = 9000 slots, above the one launch's 8192
def test_rows_bit_for_bit(T, k, H, dtype):
    E, nbytes = 7, H * dtype.itemsize
    g = torch.Generator(device="cuda").manual_seed(H + k)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)  # -1 and E: dropped
    bits = torch.randint(0, 256, (T, nbytes), generator=g, device="cuda", dtype=torch.uint8)  # NaN payloads among them
    fill = 0x5A
    xs = torch.full((T * k, nbytes), fill, dtype=torch.uint8, device="cuda")
    out, off, rows = qgemm.moe_dispatch(bits.view(dtype), ids, E, xs=xs.view(dtype))
    assert out.data_ptr() == xs.data_ptr()
    # the slots by expert, in order within one
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < E)
    order = torch.argsort(torch.where(live, flat, torch.full_like(flat, E)), stable=True)[:int(live.sum())]
    want = torch.full_like(xs, fill)  # rows behind the last expert stay
    want[:order.numel()] = bits[order // k]
    assert torch.equal(xs, want)
    place = torch.full_like(flat, -1)
    place[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(rows.reshape(-1).long(), place)
    assert off.tolist() == [int((flat[live] < e).sum()) for e in range(E + 1)]
