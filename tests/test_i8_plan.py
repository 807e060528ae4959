"""The tiling rule of the int8 products, asked through the library itself: a small host program calls
the planner of libqgemm.so."""
import os
import shutil
import subprocess

import pytest
import torch

from block_quantized_weight_qgemm_b200 import build as qbuild
from block_quantized_weight_qgemm_b200 import inputs, qgemm

PROGRAM = r"""
#include <cstdio>
#include "i8.cuh"
int main() {
  long M, N, K, rows;
  int nmat, E;
  while (scanf("%ld %ld %ld %ld %d %d", &M, &N, &K, &rows, &nmat, &E) == 6) {
    qg::I8Params p{};
    qg::i8_plan(M, N, K, rows, nmat, E, &p);
    printf("%d %d %d %d %d\n", p.NB, p.box, p.cs, p.one_set, p.pair);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = qbuild.build()
    cxx = shutil.which("g++")
    assert cxx, "the tests build a host program with g++"
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(qbuild.NVCC) or qbuild.NVCC)))
    subprocess.run([cxx, "-std=c++17", "-I", qbuild.CSRC, "-I", os.path.join(cuda, "include"), str(d / "plan.cpp"), lib,
                    "-L", os.path.join(cuda, "lib64"), "-lcudart", "-Wl,-rpath,%s:%s" % (os.path.dirname(lib), os.path.join(cuda, "lib64")),
                    "-o", str(d / "plan")], check=True, capture_output=True, text=True)

    def ask(*calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout
        return [dict(zip(("NB", "box", "cs", "one_set", "pair"), map(int, line.split()))) for line in out.splitlines()]

    return ask


@pytest.mark.parametrize("nmat", [1, 2])
@pytest.mark.parametrize("E,N,K", [(512, 2048, 512), (512, 512, 2048), (128, 768, 2048), (300, 300, 1040)])
def test_tiles_do_not_jump_where_rows_reach_the_experts(plan, nmat, E, N, K):
    # hundreds of units on either side of one row per expert, with an upper bound for max_rows
    got = plan(*[(M, N, K, rows, nmat, E) for M in (E - 3, E - 1, E, E + 1) for rows in (E // 2, 3 * E)])
    for rows in (0, 1):
        assert all(p == got[rows] for p in got[rows::2]), got[rows::2]


@pytest.mark.parametrize("nmat", [1, 2])
def test_units_that_run_at_once_are_tiled_for_that(plan, nmat):
    # 4 rows of 512 experts are at most 4 units per channel tile; 130 rows by 16 tiles are not at once on the SMs
    few, many = plan((4, 512, 2048, 4, nmat, 512), (130, 2048, 512, 130, nmat, 512))
    assert few["NB"] == 16 and few["cs"] > 1
    assert many["NB"] == (128 if nmat == 2 else 144) and many["cs"] == 1


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 63, 64, 65, 130])
def test_few_rows_of_many_experts_under_any_bound(M):
    # 64 experts, about M rows: the same bits whatever upper bound of an expert's rows is given, and the definition's
    E, N, K = 64, 300, 400
    g = torch.Generator().manual_seed(M)
    count = torch.bincount(torch.randint(0, E, (M,), generator=g), minlength=E)
    off = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    Ws = [inputs.weights(N, K, seed=i) for i in range(6)]
    packed = [qgemm.i8_pack(W.cuda()) for W in Ws]
    gate, up = (qgemm.I8ExpertTable([packed[(e + j) % 6] for e in range(E)]) for j in (0, 1))
    x = inputs.activations(M, K, seed=M)
    xd, offd, most = x.cuda(), off.cuda(), int(count.max())
    y, h = qgemm.i8_moe_run(xd, offd, gate, most), qgemm.i8_moe_gate_up(xd, offd, gate, up, most)
    for rows in {min(M, most + 1), min(M, 40), M, 1000}:
        if rows >= most:
            assert torch.equal(qgemm.i8_moe_run(xd, offd, gate, rows), y)
            assert torch.equal(qgemm.i8_moe_gate_up(xd, offd, gate, up, rows), h)

    def quantise(a):
        s = a.double().abs().amax(1).float() * (torch.ones(()) / 127)
        return torch.round(a.double() / s.double()[:, None]), s.double()

    (q, sx), refs = quantise(x), [quantise(W) for W in Ws]
    owner = torch.repeat_interleave(torch.arange(E), count)
    ref = torch.stack([(refs[int(e) % 6][0] @ q[m]) * refs[int(e) % 6][1] * sx[m] for m, e in enumerate(owner)])
    # the integer sum is exact; fp32(sum) * sw * sx rounds three times
    assert ((y.cpu().double() - ref).abs() <= 3 * 1.02 * 2.0 ** -24 * ref.abs()).all()
