"""Host-side checks of the gate and the adapters that need no GPU: every documented error
code comes before any device state is touched, in the documented order."""
import os

import pytest

A16, A4, A2 = 0x10000, 0x20004, 0x30002      # fake addresses: validation never dereferences


@pytest.fixture(scope="module")
def lib():
    from moe_grouped_gemm_lhs_amd import build, binding
    if not os.path.exists(binding.LIB_PATH):
        if not os.path.exists(build.HIPCC):
            pytest.skip("libdg.so not built and hipcc unavailable")
        build.build()
    return binding.load_library()


def route(lib, z=A16, dtype=0, ld=64, bias=None, valid=None, T=8, E=64, k=4, score=0, ids=A4, w=A4,
          counts=None, loss=None, coef=None, ws=None, wsb=0):
    return lib.dg_moe_route(z, dtype, ld, bias, valid, T, E, k, score, 0, 1.0, 0.0, ids, w, counts, loss,
                            coef, ws, wsb, None)


def test_route_codes(lib):
    for bad in (dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=17), dict(E=4, k=5), dict(T=-1),
                dict(ld=63), dict(T=1 << 31), dict(T=1 << 29, k=8)):
        assert route(lib, **bad) == 2, bad
    assert route(lib, dtype=2) == 7
    assert route(lib, score=2) == 7
    assert route(lib, score=2, k=0) == 2                  # shapes first
    assert route(lib, T=0, z=None, ids=None, w=None) == 0
    assert route(lib, z=None) == 1
    assert route(lib, ids=None) == 1
    assert route(lib, w=None) == 1
    need = lib.dg_moe_route_workspace_bytes(5000, 64)
    assert need > 64 * 8
    assert route(lib, counts=A4, loss=A4, ws=A16, wsb=need) == 1          # loss without coef
    assert route(lib, loss=A4, coef=A4, ws=A16, wsb=need) == 1            # loss without counts
    assert route(lib, z=A16 + 2) == 3
    assert route(lib, z=A16 + 1, dtype=1) == 3
    assert route(lib, ids=A4 + 1) == 3
    assert route(lib, bias=A4 + 2) == 3
    assert route(lib, T=5000, counts=A4) == 4
    assert route(lib, T=5000, counts=A4, ws=A16, wsb=need - 1) == 4
    assert route(lib, T=5000, counts=A4, ws=A16 + 8, wsb=need) == 4
    assert lib.dg_moe_route_workspace_bytes(1, 64) == 0        # a row alone needs none
    assert lib.dg_moe_route_workspace_bytes(8, 0) == 0


def backward(lib, z=A16, dtype=0, ld=64, T=8, E=64, k=4, score=0, ids=A4, gw=A4, coef=A4, gl=A4, out=A16,
             ldo=64):
    return lib.dg_moe_route_backward(z, dtype, ld, None, T, E, k, score, 0, 1.0, ids, gw, coef, gl, out,
                                     ldo, None)


def test_backward_codes(lib):
    assert backward(lib, k=0) == 2
    assert backward(lib, ldo=60) == 2
    assert backward(lib, dtype=3) == 7
    assert backward(lib, T=0, z=None, out=None) == 0
    assert backward(lib, z=None) == 1
    assert backward(lib, out=None) == 1
    assert backward(lib, ids=None) == 1
    assert backward(lib, coef=None) == 1                  # grad_loss without coef
    assert backward(lib, out=A16 + 2) == 3
    assert backward(lib, gw=A4 + 1) == 3


def lora(lib, X=A16, ldx=512, A=A16, B=A16, ids=A4, scales=None, ranks=None, base=None, ldb=0, out=A16,
         ldo=256, T=200, N=256, K=512, R=16, L=4, ws=A16, wsb=1 << 30):
    return lib.dg_lora_bf16(X, ldx, A, B, ids, scales, ranks, base, ldb, out, ldo, T, N, K, R, L, ws, wsb,
                            None)


def test_lora_codes(lib):
    for bad in (dict(K=500, ldx=504), dict(K=0), dict(R=4), dict(R=12), dict(R=136), dict(L=0), dict(T=-1),
                dict(N=-1), dict(N=(1 << 22) + 1, ldo=1 << 23), dict(ldx=508), dict(ldx=504), dict(ldo=255), dict(base=A16, ldb=255),
                dict(base=A16, ldb=264, out=A16), dict(T=1 << 31), dict(K=1 << 23, ldx=1 << 23)):
        assert lora(lib, **bad) == 2, bad
    assert lora(lib, T=0, X=None, ws=None) == 0
    assert lora(lib, N=0, ldo=0, X=None, ws=None) == 0
    for name in ("X", "A", "B", "ids", "out"):
        assert lora(lib, **{name: None}) == 1, name
    for name in ("X", "A", "B"):
        assert lora(lib, **{name: A16 + 8}) == 3, name
    assert lora(lib, ids=A4 + 2) == 3
    assert lora(lib, out=A16 + 1) == 3
    need = lib.dg_lora_workspace_bytes(200, 256, 512, 16, 4)
    assert need >= 200 * 16 * 4
    assert lora(lib, wsb=need - 1) == 4
    assert lora(lib, ws=None) == 4
    assert lora(lib, ws=A16 + 8) == 4
    assert lib.dg_lora_workspace_bytes(0, 256, 512, 16, 4) == 0
    assert lib.dg_lora_workspace_bytes(8, 256, 500, 16, 4) == 0


def test_device_check_without_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid-looking fake pointers would be launched")
    assert route(lib) == 5
    assert backward(lib) == 5
    assert lora(lib, out=A2, scales=A4, ranks=A4) == 5
