"""What rms_norm and packed_linear refuse and accept, without a device: calls
either fail validation, or get as far as a workspace that is not there, or reach
a library that only records them."""
import pytest
import torch

import post_weight_quantization_19_amd as P
from post_weight_quantization_19_amd import _lib as B

FAKE = 0x100000          # never dereferenced
INVALID, WS = B.PWQ_ERR_INVALID_ARG, B.PWQ_ERR_WORKSPACE
WIDTH = {B.PWQ_I8: 1, B.PWQ_BF16: 2, B.PWQ_F32: 4}


def linear(x, y, ntok=200, m=250, n=250, ldx=None, ldy=None, xdt=B.PWQ_F32, ydt=B.PWQ_F32):
    """packed_linear of rows that need a workspace (250 columns: a copy of x)."""
    xs = FAKE if xdt == B.PWQ_I8 else None
    return B.lib().pwq_packed_linear(x, xdt, ntok, ldx or n, xs, FAKE << 8, m, n, FAKE << 8, None,
                                     0, None, None, 0, y, ydt, ldy or m, None, 0, None)


@pytest.mark.parametrize("xdt,ydt", [(B.PWQ_F32, B.PWQ_F32), (B.PWQ_BF16, B.PWQ_BF16),
                                     (B.PWQ_I8, B.PWQ_BF16), (B.PWQ_BF16, B.PWQ_F32)])
def test_packed_linear_output_over_its_input(xdt, ydt):
    a, b = WIDTH[xdt], WIDTH[ydt]
    size, far = 200 * 250 * a, FAKE << 4
    assert linear(far, far, xdt=xdt, ydt=ydt) == INVALID
    assert b"overlap" in B.lib().pwq_last_error()
    assert linear(far, far + 16, xdt=xdt, ydt=ydt) == INVALID
    assert linear(far, far + size - b, xdt=xdt, ydt=ydt) == INVALID
    assert linear(far + 200 * 250 * b - a, far, xdt=xdt, ydt=ydt) == INVALID
    # next to each other, in memory and in a row
    assert linear(far, far + size, xdt=xdt, ydt=ydt) == WS
    assert linear(far + 200 * 250 * b, far, xdt=xdt, ydt=ydt) == WS
    ld = 250 * (a + b)
    assert linear(far, far + 250 * a, ldx=ld // a, ldy=ld // b, xdt=xdt, ydt=ydt) == WS
    assert linear(far + 250 * b, far, ldx=ld // a, ldy=ld // b, xdt=xdt, ydt=ydt) == WS
    assert linear(far, far + 250 * a - b, ldx=ld // a, ldy=ld // b, xdt=xdt, ydt=ydt) == INVALID
    assert linear(far, far + 250 * a + b, ldx=ld // a, ldy=ld // b, xdt=xdt, ydt=ydt) == INVALID


def test_rms_norm_outputs_over_each_other():
    def norm(x=FAKE, res=FAKE << 4, total=FAKE << 5, y=FAKE << 6, ntok=3, n=64, ldx=64, ldr=64,
             lds=64, ldy=64):
        return B.lib().pwq_rms_norm(x, B.PWQ_BF16, ntok, n, ldx, res, ldr, FAKE << 8, 0, 1e-6,
                                    total, lds, y, B.PWQ_BF16, ldy, None, None)

    size = 3 * 64 * 2
    for other in (FAKE, FAKE << 4, FAKE << 5):
        for shift in (0, 2, size - 2, 2 - size):
            assert norm(y=other + shift) == INVALID, (hex(other), shift)
            assert b"overlap" in B.lib().pwq_last_error()
    for other in (FAKE, FAKE << 4):
        for shift in (2, size - 2, 2 - size):
            assert norm(total=other + shift) == INVALID, (hex(other), shift)
    assert norm(total=FAKE, lds=128) == INVALID
    assert norm(y=FAKE + 100, ldx=128, ldy=128) == INVALID


# ------------------------------------------------------------------ several GPUs

class OnGpu0(torch.Tensor):
    """A tensor that says it is on a GPU (its memory is the host's: the library
    is replaced)."""
    index = 0

    def get_device(self):
        return self.index

    is_cuda = property(lambda self: True)


class OnGpu1(OnGpu0):
    index = 1


@pytest.fixture
def gpus(monkeypatch):
    """Calls of the library as (name, current GPU, stream); GPU 0 is current."""
    state = {"current": 0, "calls": []}

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *error):
            state["current"] = self.before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                state["calls"].append((name, state["current"], args[-1]))
                return 0
            return call

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + (index or 0),
                        raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(P, "lib", Library)
    return state


def of(gpu, *shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(gpu)


def layer_on(gpu, m=32, n=64):
    return {"qweight": of(gpu, m, n // 2, dtype=torch.uint8), "scales": of(gpu, m, 2),
            "zeros": of(gpu, m, 2, dtype=torch.uint8), "n": n, "group": 32,
            "outlier_off": of(gpu, 3, dtype=torch.int32),
            "outliers": of(gpu, 5, dtype=torch.int32)}


@pytest.mark.parametrize("gpu", [OnGpu0, OnGpu1])
def test_calls_run_on_the_gpu_of_their_input(gpus, gpu):
    P.rms_norm(of(gpu, 3, 64), of(gpu, 64), of(gpu, 3, 64), out_dtype=torch.int8)
    P.packed_linear(of(gpu, 3, 64), layer_on(gpu))
    assert gpus["calls"] == [("pwq_rms_norm", gpu.index, 1000 + gpu.index),
                             ("pwq_packed_linear", gpu.index, 1000 + gpu.index)]
    assert gpus["current"] == 0


def test_tensors_of_another_gpu_are_refused(gpus):
    a, b = OnGpu0, OnGpu1
    x = of(a, 3, 64)
    for args in ((of(b, 64),), (of(a, 64), of(b, 3, 64)),
                 (of(a, 64), x, 1e-6, None, of(b, 3, 64))):
        with pytest.raises(ValueError, match="GPU"):
            P.rms_norm(x, *args)
    packed = layer_on(a)
    for name in ("qweight", "scales", "zeros", "outlier_off", "outliers"):
        with pytest.raises(ValueError, match="GPU"):
            P.packed_linear(x, dict(packed, **{name: layer_on(b)[name]}))
    with pytest.raises(ValueError, match="GPU"):
        P.packed_linear(x, packed, out=of(b, 3, 32))
    with pytest.raises(ValueError, match="GPU"):
        P.packed_linear(x.to(torch.int8).as_subclass(a), packed, x_scales=of(b, 3))
    codes = of(a, 32, 64, dtype=torch.int32)
    for scales, zeros in ((of(b, 32, 2), of(a, 32, 2, dtype=torch.int32)),
                          (of(a, 32, 2), of(b, 32, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            P.pack_weights(codes, scales, P.Grid("asym", 4, 32), zeros)
    assert gpus["calls"] == []


def test_host_tensors_are_refused(gpus):
    x = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="GPU"):
        P.rms_norm(x, torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        P.rms_norm(of(OnGpu0, 3, 64), torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        P.packed_linear(x, layer_on(OnGpu0))


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("which", range(4))
def test_tensors_that_require_a_gradient(gpus, which):
    """Refused while gradients are recorded: they would be lost in silence."""
    def tensors(*shapes):
        ts = [of(OnGpu0, *s) for s in shapes]
        ts[which].requires_grad_()
        return ts

    def norm():
        x, weight, residual, total = tensors((3, 64), (64,), (3, 64), (3, 64))
        P.rms_norm(x, weight, residual, sum_out=total)

    def linear():
        x, out, scales, steps = tensors((3, 64), (3, 32), (32, 2), (3,))
        if which == 3:
            x = x.to(torch.int8).as_subclass(OnGpu0)
        P.packed_linear(x, dict(layer_on(OnGpu0), scales=scales), out=out,
                        x_scales=steps if which == 3 else None)

    for call in (norm, linear):
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert gpus["calls"] == []
    with torch.no_grad():
        norm()
        linear()
    assert len(gpus["calls"]) == 2
