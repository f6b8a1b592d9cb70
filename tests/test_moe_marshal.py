"""The marshalling module of the gate and the adapters, on CPU tensors: pointers and strides of
what the calls take, the errors of what they do not, and argument conversion."""
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def native():
    from moe_grouped_gemm_lhs_amd import binding, build, moe_ops
    if not (os.path.exists(binding.LIB_PATH) and os.path.exists(build.MARSHAL)):
        if not os.path.exists(build.HIPCC):
            pytest.skip("not built and hipcc unavailable")
        build.build()
    return moe_ops._load_native()


CPU = torch.device("cpu")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int32, torch.uint8])
def test_vector(native, dtype):
    for shape in ((), (0,), (1,), (5,), (3, 4), (2, 3, 8)):
        t = torch.zeros(shape, dtype=dtype)
        assert native.vector(t, "t", dtype, shape, CPU) == t.data_ptr()
    t = torch.zeros(10, dtype=dtype)[3:]
    assert native.vector(t, "t", dtype, (7,), CPU) == t.data_ptr()
    assert native.vector(None, "t", dtype, (7,), CPU) is None
    leaf = torch.nn.Parameter(torch.zeros(4))
    assert native.vector(leaf, "t", torch.float32, (4,), CPU) == leaf.data_ptr()


def test_vector_refusals(native):
    t = torch.zeros(4, 6)
    with pytest.raises(TypeError, match="w must be torch.int32"):
        native.vector(t, "w", torch.int32, (4, 6), CPU)
    for shape in ((4, 5), (4,), (4, 6, 1), (), (4, 6.5), (4, 1 << 70)):
        with pytest.raises(ValueError, match="w must have shape"):
            native.vector(t, "w", torch.float32, shape, CPU)
    with pytest.raises(ValueError, match="contiguous"):
        native.vector(t.t(), "w", torch.float32, (6, 4), CPU)
    with pytest.raises(ValueError, match="must be on cuda:0"):
        native.vector(t, "w", torch.float32, (4, 6), torch.device("cuda:0"))
    with pytest.raises(AttributeError):
        native.vector([1.0], "w", torch.float32, (1,), CPU)
    with pytest.raises(TypeError):
        native.vector(t, "w")


def test_rows(native):
    f = torch.float32
    t = torch.zeros(6, 10)
    assert native.rows(t, "t", f, (6, 10), CPU) == (t.data_ptr(), 10)
    v = t[1:5, 2:7]
    assert native.rows(v, "t", f, (4, 5), CPU) == (v.data_ptr(), 10)
    assert native.rows(t[:, :1], "t", f, (6, 1), CPU) == (t.data_ptr(), 10)
    # of one row or none the stride says nothing
    assert native.rows(t[:1, :4], "t", f, (1, 4), CPU) == (t.data_ptr(), 4)
    e = torch.zeros(0, 7)
    assert native.rows(e, "t", f, (0, 7), CPU)[1] == 7
    one = torch.zeros(1, 5).expand(3, 5)
    assert native.rows(one, "t", f, (3, 5), CPU) == (one.data_ptr(), 0)     # the call refuses 0


def test_rows_refusals(native):
    t = torch.zeros(6, 10)
    with pytest.raises(ValueError, match="dense rows"):
        native.rows(t.t(), "t", torch.float32, (10, 6), CPU)
    with pytest.raises(ValueError, match="dense rows"):
        native.rows(t[:, ::2], "t", torch.float32, (6, 5), CPU)
    with pytest.raises(TypeError):
        native.rows(t, "t", torch.bfloat16, (6, 10), CPU)
    with pytest.raises(ValueError):
        native.rows(t, "t", torch.float32, (6, 9), CPU)
    with pytest.raises(AttributeError):
        native.rows(None, "t", torch.float32, (6, 9), CPU)


@pytest.mark.parametrize("row", [lambda: torch.zeros(6, 10)[:1, ::2], lambda: torch.zeros(6, 10)[:, :1].t(),
                                 lambda: torch.zeros(1, 1).expand(1, 5)],
                         ids=["every other column", "a column as a row", "one number repeated"])
def test_a_row_alone_must_be_dense(native, row):
    """Of one row only the row stride says nothing; its elements must follow each other."""
    from moe_grouped_gemm_lhs_amd import moe_ops
    t = row()
    assert t.shape[0] == 1 and t.stride(1) != 1
    for rows in (native.rows, moe_ops._rows):
        with pytest.raises(ValueError, match="dense rows"):
            rows(t, "t", torch.float32, tuple(t.shape), CPU)


def test_rows_that_hold_nothing_may_have_any_strides(native):
    from moe_grouped_gemm_lhs_amd import moe_ops
    t = torch.zeros(6, 10)
    for rows in (native.rows, moe_ops._rows):
        assert rows(t[:0, ::2], "t", torch.float32, (0, 5), CPU)[1] == 5
        assert rows(t.t()[:1, :1], "t", torch.float32, (1, 1), CPU) == (t.data_ptr(), 1)
        assert rows(t[:1, :0], "t", torch.float32, (1, 0), CPU)[1] == 0


def test_calls_convert_their_arguments(native):
    from moe_grouped_gemm_lhs_amd.binding import load_library
    lib = load_library()
    for sizes in ((1, 2112, 7168, 16, 8), (5000, 64, 256, 64, 3), (-1, 8, 128, 8, 1)):
        assert native.dg_lora_workspace_bytes(*sizes) == lib.dg_lora_workspace_bytes(*sizes)
    assert native.dg_moe_route_workspace_bytes(5000, 64) == lib.dg_moe_route_workspace_bytes(5000, 64)
    with pytest.raises(TypeError):
        native.dg_moe_route_workspace_bytes(5000)
    with pytest.raises(TypeError):
        native.dg_moe_route_workspace_bytes(5000, "64")
    with pytest.raises(OverflowError):
        native.dg_moe_route_workspace_bytes(5000, 1 << 64)
    # status codes come through: a shape, then a null pointer
    args = [0x10000, 0, 64, None, None, 8, 64, 4, 0, False, 1.0, 0, 0x10000, 0x10000, None, None, None,
            None, 0, None]
    assert native.dg_moe_route(*args[:2], 63, *args[3:]) == 2
    assert native.dg_moe_route(None, *args[1:]) == 1
    with pytest.raises(OverflowError):
        native.dg_moe_route(args[0], 1 << 40, *args[2:])


def test_one_compiler_builds_everything(monkeypatch):
    """hipcc, or what HIPCC names, is all that a build calls."""
    from moe_grouped_gemm_lhs_amd import build
    commands = []
    monkeypatch.setattr(build, "HIPCC", "/where/hipcc")
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd, **kw: commands.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda *a: None)
    monkeypatch.setattr(build.os, "remove", lambda *a: None)
    build.build()
    assert len(commands) == len(build.SOURCES) + 2
    assert all(c[0] == "/where/hipcc" for c in commands), [c[0] for c in commands]
