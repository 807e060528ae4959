"""Refusals and sizes of the routed-token and int8 entry points, with no GPU: every argument
error is found before any device work."""
import ctypes

import pytest

from block_quantized_weight_qgemm_b200 import build as qbuild
from block_quantized_weight_qgemm_b200 import qgemm

FORMAT, SHAPE, K_BLOCK, NULL, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 6
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qgemm.lib()


def _dispatch(lib, x=16, dt=1, T=4, H=64, ids=16, k=2, E=8, off=16, rows=16, xs=16):
    return lib.qgemm_moe_dispatch(x, dt, T, H, ids, k, E, off, rows, xs, None)


def _combine(lib, ys=16, dt=1, T=4, H=64, rows=16, w=16, k=2, y=16, ydt=1):
    return lib.qgemm_moe_combine(ys, dt, T, H, rows, w, k, y, ydt, None)


def _dgrad(lib, dxs=16, dt=1, T=4, H=64, rows=16, k=2, dx=16, xdt=1):
    return lib.qgemm_moe_dispatch_grad(dxs, dt, T, H, rows, k, dx, xdt, None)


def _cgrad(lib, dy=16, ddt=1, ys=16, dt=1, T=4, H=64, rows=16, w=16, k=2, dys=16, dw=16):
    return lib.qgemm_moe_combine_grad(dy, ddt, ys, dt, T, H, rows, w, k, dys, dw, None)


def _run(lib, x=16, M=4, K=64, c=16, s=16, N=8, y=16, ydt=0, ws=16, n=BIG):
    return lib.qgemm_i8_run(x, M, K, c, s, N, y, ydt, ws, n, None)


def _moe(lib, x=16, M=4, K=64, E=2, off=16, mr=4, c=16, s=16, N=8, y=16, ydt=0, ws=16, n=BIG):
    return lib.qgemm_i8_moe_run(x, M, K, E, off, mr, c, s, N, y, ydt, ws, n, None)


def _gate(lib, x=16, M=4, K=64, E=2, off=16, mr=4, gc=16, gs=16, uc=16, us=16, N=8, h=16, ws=16,
          n=BIG):
    return lib.qgemm_i8_moe_gate_up(x, M, K, E, off, mr, gc, gs, uc, us, N, h, ws, n, None)


REFUSED = [
    (_dispatch, dict(dt=2), FORMAT), (_dispatch, dict(T=0), SHAPE), (_dispatch, dict(k=0), SHAPE),
    (_dispatch, dict(H=0), SHAPE), (_dispatch, dict(E=0), SHAPE), (_dispatch, dict(E=4097), SHAPE),
    (_dispatch, dict(T=1 << 30, k=2), SHAPE), (_dispatch, dict(T=-1), SHAPE),
    (_dispatch, dict(x=None), NULL), (_dispatch, dict(ids=None), NULL), (_dispatch, dict(off=None), NULL),
    (_dispatch, dict(rows=None), NULL), (_dispatch, dict(xs=None), NULL),
    (_dispatch, dict(x=8), ALIGN), (_dispatch, dict(xs=24), ALIGN), (_dispatch, dict(ids=18), ALIGN),
    (_dispatch, dict(off=18), ALIGN), (_dispatch, dict(rows=18), ALIGN),
    (_combine, dict(dt=2), FORMAT), (_combine, dict(ydt=-1), FORMAT), (_combine, dict(T=0), SHAPE),
    (_combine, dict(k=0), SHAPE), (_combine, dict(H=0), SHAPE), (_combine, dict(H=1 << 31), SHAPE),
    (_dispatch, dict(H=(1 << 30) + 1), SHAPE), (_combine, dict(H=(1 << 30) + 1), SHAPE),
    (_dgrad, dict(H=(1 << 31) - 1), SHAPE), (_cgrad, dict(H=(1 << 31) - 1), SHAPE),
    (_combine, dict(ys=None), NULL), (_combine, dict(rows=None), NULL), (_combine, dict(w=None), NULL),
    (_combine, dict(y=None), NULL), (_combine, dict(ys=8), ALIGN), (_combine, dict(y=8), ALIGN),
    (_combine, dict(rows=17), ALIGN), (_combine, dict(w=18), ALIGN),
    (_dgrad, dict(dt=2), FORMAT), (_dgrad, dict(xdt=2), FORMAT), (_dgrad, dict(T=0), SHAPE),
    (_dgrad, dict(dxs=None), NULL), (_dgrad, dict(rows=None), NULL), (_dgrad, dict(dx=None), NULL),
    (_dgrad, dict(dxs=8), ALIGN), (_dgrad, dict(dx=8), ALIGN), (_dgrad, dict(rows=18), ALIGN),
    (_cgrad, dict(ddt=2), FORMAT), (_cgrad, dict(dt=2), FORMAT), (_cgrad, dict(k=-1), SHAPE),
    (_cgrad, dict(dy=None), NULL), (_cgrad, dict(ys=None), NULL), (_cgrad, dict(rows=None), NULL),
    (_cgrad, dict(w=None), NULL), (_cgrad, dict(dys=None), NULL), (_cgrad, dict(dw=None), NULL),
    (_cgrad, dict(dy=8), ALIGN), (_cgrad, dict(ys=8), ALIGN), (_cgrad, dict(dys=8), ALIGN),
    (_cgrad, dict(dw=18), ALIGN), (_cgrad, dict(rows=18), ALIGN), (_cgrad, dict(w=18), ALIGN),
    (_run, dict(M=0), SHAPE), (_run, dict(N=0), SHAPE), (_run, dict(K=0), SHAPE),
    (_run, dict(K=131088), SHAPE), (_run, dict(K=24), K_BLOCK), (_run, dict(ydt=2), FORMAT),
    (_run, dict(x=None), NULL), (_run, dict(c=None), NULL), (_run, dict(s=None), NULL),
    (_run, dict(y=None), NULL), (_run, dict(x=8), ALIGN), (_run, dict(c=8), ALIGN),
    (_run, dict(y=8), ALIGN), (_run, dict(s=18), ALIGN), (_run, dict(K=4096, ws=None), WORKSPACE),
    (_run, dict(K=4096, n=255), WORKSPACE), (_run, dict(ws=24), ALIGN),
    (_moe, dict(M=0), SHAPE), (_moe, dict(E=0), SHAPE), (_moe, dict(E=4097), SHAPE), (_moe, dict(mr=0), SHAPE),
    (_moe, dict(K=131088), SHAPE), (_moe, dict(K=24), K_BLOCK), (_moe, dict(ydt=2), FORMAT),
    (_moe, dict(x=None), NULL), (_moe, dict(off=None), NULL), (_moe, dict(c=None), NULL),
    (_moe, dict(s=None), NULL), (_moe, dict(y=None), NULL), (_moe, dict(off=18), ALIGN),
    (_moe, dict(c=20), ALIGN), (_moe, dict(s=20), ALIGN), (_moe, dict(y=8), ALIGN),
    (_moe, dict(ws=None), WORKSPACE), (_moe, dict(n=255), WORKSPACE),
    (_gate, dict(h=None), NULL), (_gate, dict(uc=None), NULL), (_gate, dict(us=None), NULL),
    (_gate, dict(gs=20), ALIGN), (_gate, dict(uc=20), ALIGN), (_gate, dict(h=8), ALIGN),
    (_gate, dict(K=24), K_BLOCK), (_gate, dict(ws=None), WORKSPACE),
]


@pytest.mark.parametrize("call,args,status", REFUSED,
                         ids=["%s-%s" % (c.__name__[1:], "-".join("%s=%s" % a for a in d.items()))
                              for c, d, _ in REFUSED])
def test_refused_before_any_device_work(lib, call, args, status):
    assert call(lib, **args) == status


def test_sizes(lib):
    sz, s2 = ctypes.c_size_t(), ctypes.c_size_t()
    assert qgemm.i8_packed_size(300, 144) == (3 * 2 * 16384, 1200)
    assert lib.qgemm_i8_packed_size(300, 24, ctypes.byref(sz), ctypes.byref(s2)) == K_BLOCK
    assert lib.qgemm_i8_packed_size(300, 144, None, None) == NULL
    # codes and scales of x at least, at every width, growing with it
    at = [qgemm.i8_workspace_size(17408, 5120, M) for M in (1, 64, 65, 257, 8192)]
    assert at == sorted(at) and all(b >= M * 5124 for b, M in zip(at, (1, 64, 65, 257, 8192)))
    assert qgemm.i8_moe_workspace_size(512, 2048, 640) >= 640 * 2052
    assert qgemm.i8_workspace_size(512, 1024, 16) == 0     # a small call's product quantises x itself
    assert lib.qgemm_i8_workspace_size(8, 64, 0, ctypes.byref(sz)) == SHAPE
    assert lib.qgemm_i8_moe_workspace_size(8, 64, 4, None) == NULL
    assert lib.qgemm_i8_quant_x(16, 4, 24, 16, 16, None) == K_BLOCK
    assert lib.qgemm_i8_quant_x(16, 0, 32, 16, 16, None) == SHAPE
    assert lib.qgemm_i8_quant_x(16, 4, 32, 16, None, None) == NULL
    assert lib.qgemm_i8_quant_x(16, 4, 32, 20, 16, None) == ALIGN
    assert lib.qgemm_i8_pack(None, 4, 32, 16, 16, None) == NULL
    assert lib.qgemm_i8_pack(16, 4, 32, 16, 18, None) == ALIGN
    assert lib.qgemm_i8_repack_rowmajor(4, 32, 16, 31, 16, None) == SHAPE   # pitch below a row
    assert lib.qgemm_i8_repack_rowmajor(4, 32, None, 32, 16, None) == NULL
    assert lib.qgemm_i8_repack_rowmajor(4, 32, 16, 32, 24, None) == ALIGN
