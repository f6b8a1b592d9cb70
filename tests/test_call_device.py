"""Where the calls of the binding run: on their tensors' device, also when another is the current
one.  Looked at on the CPU, with arguments that only say where they are."""
import pytest

torch = pytest.importorskip("torch")

from moe_grouped_gemm_lhs_amd import binding, moe_ops  # noqa: E402


class Entered(Exception):
    pass


class On:
    """What a call looks at first of a tensor on cuda:1."""
    is_cuda = True
    device = torch.device("cuda:1")

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


CODES = (On((128, 256), torch.uint8), On((128, 2), torch.float32), On((128, 256), torch.uint8),
         On((1, 2), torch.float32))
GROUPED = (On((4, 128, 256), torch.uint8), On((4, 1, 2), torch.float32))
BF = torch.bfloat16
CALLS = {
    "dg_gemm_fp8_nt": CODES,
    "dg_gemm_fp8_nt_noalloc": CODES,
    "dg_grouped_gemm_fp8_contiguous": CODES[:2] + GROUPED + (On((128,), torch.int32),),
    "dg_grouped_gemm_fp8_masked": (On((4, 32, 256), torch.uint8), On((4, 32, 2), torch.float32)) + GROUPED +
                                  (On((4,), torch.int32),),
    "dg_quantize_fp8_1x128": (On((4, 256), BF),),
    "dg_quantize_fp8_128x128": (On((4, 256), BF),),
    "dg_transpose_fp8": (On((16, 256), torch.uint8),),
    "dg_moe_route": (On((4, 8), torch.float32), 2),
    "dg_moe_route_backward": (On((4, 8), torch.float32), On((4, 2), torch.int32)),
    "dg_lora_bf16": (On((4, 256), BF), On((2, 8, 256), BF), On((2, 64, 8), BF), On((4,), torch.int32)),
}


@pytest.fixture
def current(monkeypatch):
    """cuda:0 is current; entering a device's context raises Entered with that device."""
    def enter(self):
        raise Entered(self.idx)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda.device, "__enter__", enter)


@pytest.mark.parametrize("call", list(CALLS))
def test_the_tensors_device_is_entered(call, current):
    with pytest.raises(Entered) as e:
        getattr(binding if hasattr(binding, call) else moe_ops, call)(*CALLS[call])
    assert e.value.args == (1,)


class Allocated(Exception):
    pass


@pytest.mark.parametrize("call", list(CALLS))
def test_outputs_belong_to_the_stream_that_is_given(call, monkeypatch):
    """Outputs, and the zeros that the grouped calls' unwritten rows keep, are allocated with that
    stream as the current one: nothing else orders them before the launch."""
    entered = []

    class Stream:
        device, cuda_stream = On.device, 0x1000

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *exc):
            return False

    def allocate(*args, **kwargs):
        raise Allocated(tuple(entered))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, allocate)
    # the arguments' pointers are not looked at before the outputs are allocated
    native = type("Native", (), {"rows": staticmethod(lambda *a: (0, 8)), "vector": staticmethod(lambda *a: 0)})
    monkeypatch.setattr(moe_ops, "_native", native)
    stream = Stream()
    with pytest.raises(Allocated) as e:
        getattr(binding if hasattr(binding, call) else moe_ops, call)(*CALLS[call], stream=stream)
    assert e.value.args == ((stream,),)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_device_is_refused(call, monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda:0"), 0x1000

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(moe_ops, "_native", object())
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        getattr(binding if hasattr(binding, call) else moe_ops, call)(*CALLS[call], stream=Stream())
