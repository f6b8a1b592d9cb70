"""Where the feed-forward operators run: on their tensors' device, also when another is the current
one, and on the stream that is given.  Looked at on the CPU, with arguments that only say where
they are."""
import pytest

torch = pytest.importorskip("torch")

from moe_grouped_gemm_lhs_amd import ffn_ops, moe_ops  # noqa: E402

BF, U8, F, I = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class Reached(Exception):
    pass


class On:
    """What a call looks at of a tensor on cuda:1."""
    is_cuda = True
    device = torch.device("cuda:1")

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)


ROWS = On((130, 256), U8), On((130, 2), F)
CALLS = {
    "dg_rms_norm_fp8": (On((4, 256), BF),),
    "dg_rms_norm_backward": (On((4, 256), BF), On((4, 256), BF), On((4,), F)),
    "dg_gated_fp8_nt": (*ROWS, On((512, 256), U8), On((4, 2), F)),
    "dg_grouped_gated_fp8_contiguous": (*ROWS, On((3, 512, 256), U8), On((3, 4, 2), F), On((130,), I)),
    "dg_grouped_gated_fp8_masked": (On((3, 9, 256), U8), On((3, 9, 2), F), On((3, 512, 256), U8),
                                    On((3, 4, 2), F), On((3,), I)),
    "dg_gated_backward": (On((130, 128), BF), *ROWS),
    "dg_wgrad_fp8": (*ROWS, *ROWS),
    "dg_grouped_wgrad_fp8_contiguous": (*ROWS, *ROWS, On((130,), I), 3),
}


@pytest.fixture
def native(monkeypatch):
    """The marshalling module's checks of pointers, which these arguments have none of."""
    class Native:
        rows = staticmethod(lambda *a: (0, 8))
        vector = staticmethod(lambda *a: 0)

    monkeypatch.setattr(moe_ops, "_native", Native)


@pytest.mark.parametrize("call", list(CALLS))
def test_the_tensors_device_is_entered(call, native, monkeypatch):
    def enter(self):
        raise Reached(self.idx)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda.device, "__enter__", enter)
    with pytest.raises(Reached) as e:
        getattr(ffn_ops, call)(*CALLS[call])
    assert e.value.args == (1,)


@pytest.mark.parametrize("call", list(CALLS))
def test_outputs_belong_to_the_stream_that_is_given(call, native, monkeypatch):
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
        raise Reached(tuple(entered))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, allocate)
    stream = Stream()
    with pytest.raises(Reached) as e:
        getattr(ffn_ops, call)(*CALLS[call], stream=stream)
    assert e.value.args == ((stream,),)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_device_is_refused(call, native, monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda:0"), 0x1000

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        getattr(ffn_ops, call)(*CALLS[call], stream=Stream())


def test_every_call_is_here():
    calls = {n for n in dir(ffn_ops) if n.startswith("dg_") and "workspace" not in n}
    assert calls == set(CALLS)
