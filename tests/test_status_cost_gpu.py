"""What conv2d_device_status and conv2d_set_wait_limit cost: a few transfers of a
word, whatever number of kernels report to them."""
import time

import pytest

pytestmark = pytest.mark.gpu


def _median_us(call, n=100):
    import torch
    for _ in range(20):
        call()
    took = []
    for _ in range(9):
        torch.cuda.synchronize()
        began = time.perf_counter()
        for _ in range(n):
            call()
        took.append((time.perf_counter() - began) / n * 1e6)
    return sorted(took)[4]


def test_status_and_limit_are_a_few_transfers():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build, capi
    build.build()
    stream = torch.cuda.current_stream().cuda_stream
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = _median_us(word.item)                            # a word to the host, waited for
    assert _median_us(lambda: capi.conv2d_device_status(stream)) < 3 * one
    assert _median_us(lambda: capi.conv2d_set_wait_limit(0, stream)) < 3 * one
    assert capi.conv2d_device_status(stream) == 0


def test_status_is_reported_once_to_one_of_many_threads():
    """A wait that ran out is reported by one call, and nothing is left for the next."""
    import threading

    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build, capi, head
    build.build()
    h = torch.randn(600, 1024, device="cuda").bfloat16()
    w = torch.randn(2000, 1024, device="cuda").bfloat16()
    target = torch.zeros(600, dtype=torch.int64, device="cuda")
    op = head.LinearCrossEntropy(600, 1024, 2000, "bf16")
    op(h, w, target)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    capi.conv2d_device_status(stream)
    try:
        capi.conv2d_set_wait_limit(1, stream)
        op(h, w, target)
        torch.cuda.synchronize()
    finally:
        capi.conv2d_set_wait_limit(0, stream)
    seen = []
    threads = [threading.Thread(target=lambda: seen.extend(capi.conv2d_device_status(stream) for _ in range(50)))
               for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 200 and sum(v != 0 for v in seen) == 1
