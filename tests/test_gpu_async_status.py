"""What the calls that only enqueue report afterwards: failures and traced times."""

import pytest
import torch

pytestmark = pytest.mark.gpu

QUANTIZE, MATMUL, DISTILL = 24, 25, 27        # gptq_kernel_kind values


def setup(lib, dev):
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(200, 1024, generator=g, device=dev)
    codes, scales = lib.gptq_fp8_quantize(torch.randn(512, 1024, generator=g, device=dev))
    logits = torch.randn(4, 900, generator=g, device=dev)
    tv = torch.zeros(4, 8, device=dev)
    ti = torch.arange(32, dtype=torch.int32, device=dev).reshape(4, 8)
    bad = ti.clone()
    bad[1, 4] = 900
    linear = lambda **kw: lib.gptq_fp8_linear(x, codes, scales, **kw)
    return linear, lambda i=ti: lib.gptq_distill_loss(logits, tv, i), bad


def report(lib):
    with pytest.raises(lib.GptqError) as e:
        lib.gptq_async_status()
    return e.value.status


@pytest.mark.parametrize("index_first", [True, False])
def test_a_timeout_is_always_reported(lib, cuda_device, index_first):
    """Outputs are unset after a wait that ran out, but right after a bad index: the index must not
    hide the wait."""
    linear, distill, bad = setup(lib, cuda_device)
    linear(), distill()
    lib.gptq_async_status()
    try:
        if index_first:
            distill(bad)
            torch.cuda.synchronize()
        lib.gptq_set_wait_limit(1)
        linear()
        lib.gptq_set_wait_limit(0)
        if not index_first:
            torch.cuda.synchronize()
            distill(bad)
        assert report(lib) == lib.GPTQ_ERR_TIMEOUT
    finally:
        lib.gptq_set_wait_limit(0)
    lib.gptq_async_status()                         # once
    distill(bad)
    assert report(lib) == lib.GPTQ_ERR_INVALID_ARG
    lib.gptq_async_status()
    ref = linear()
    assert torch.equal(linear(), ref)
    lib.gptq_async_status()


@pytest.fixture
def tracing(lib):
    lib.gptq_profile_enable(True)
    lib.gptq_profile_reset()
    yield
    lib.gptq_profile_enable(False)
    lib.gptq_profile_reset()


def test_trace_of_another_stream(lib, cuda_device, tracing):
    """Waiting for one stream collects the times of launches that have ended; those of another
    stream that have not are collected when they have, and disturb no call between."""
    linear, distill, _ = setup(lib, cuda_device)
    linear(), distill()
    lib.gptq_async_status()
    lib.gptq_profile_reset()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)              # about a tenth of a second
    linear(stream=side)
    distill()
    lib.gptq_async_status()                         # the current stream's alone
    assert not side.query()
    assert lib.gptq_profile_read(DISTILL)[1] == 1 and lib.gptq_profile_read(MATMUL)[1] == 0
    distill()
    lib.gptq_async_status()
    lib.gptq_async_status(stream=side)
    assert lib.gptq_profile_read(DISTILL)[1] == 2
    ms, n = lib.gptq_profile_read(MATMUL)
    assert n == 1 and 0 < ms < 50
    assert lib.gptq_profile_read(QUANTIZE)[1] == 1


def test_trace_survives_a_refused_call(lib, cuda_device, tracing):
    _, distill, _ = setup(lib, cuda_device)
    distill()
    lib.gptq_async_status()
    lib.gptq_profile_reset()
    distill()
    with pytest.raises(lib.GptqError):
        lib.gptq_top_logits(torch.zeros(2, 300, device=cuda_device), 257)
    lib.gptq_async_status()
    assert lib.gptq_profile_read(DISTILL)[1] == 1
