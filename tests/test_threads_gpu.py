"""Calls of one kernel from several threads, with small and large shapes: what one
thread's shape needs of a kernel (its shared memory) takes nothing from another's."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_convolution_gb300 import build
    build.build()


def _run(makers, calls=2000):
    """Each maker's call, `calls` times in a thread and a stream of its own."""
    import torch
    errors, start = [], threading.Barrier(len(makers))

    def loop(make):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                call, check = make()
                stream.synchronize()
                start.wait()
                for _ in range(calls):
                    out = call()
                stream.synchronize()
                check(out)
        except Exception as e:
            errors.append(repr(e))
            start.abort()

    threads = [threading.Thread(target=loop, args=(m,)) for m in makers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def _loss(hidden, tokens, dtype="bf16"):
    def make():
        import torch
        from dense_convolution_gb300 import head
        op = head.LinearCrossEntropy(tokens, hidden, 64, dtype, reduction="none")
        t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        h, w = torch.ones(tokens, hidden, device="cuda", dtype=t), torch.ones(64, hidden, device="cuda", dtype=t)
        target = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")

        def check(out):                                    # 64 equal logits
            assert torch.allclose(out[0], torch.full((tokens,), 64.0, device="cuda").log(), atol=1e-3)
        return (lambda: op(h, w, target, workspace=ws)), check
    return make


def _norm(rows, cols, pixels=None, backward=False):
    def make():
        import torch
        from dense_convolution_gb300 import head
        op = head.LayerNorm(rows, cols, "bf16", "f32", pixels=pixels)
        x = torch.randn((rows // pixels, cols, pixels) if pixels else (rows, cols), device="cuda").bfloat16()
        y, mean, rstd = op(x, stats=True)
        ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")
        if not backward:
            out = torch.empty_like(y)
            return (lambda: op(x, y=out)), lambda got: None if got.equal(y) else pytest.fail("another result")
        want = op.backward(y, x, None, mean, rstd)[0]
        return ((lambda: op.backward(y, x, None, mean, rstd, workspace=ws)),
                lambda got: None if got[0].equal(want) else pytest.fail("another result"))
    return make


@pytest.mark.parametrize("small,large", [
    (_loss(128, 1), _loss(8192, 1)), (_loss(64, 4), _loss(3000, 4)), (_loss(64, 7, "f32"), _loss(2500, 7, "f32")),
    (_norm(200, 256, 25), _norm(200, 1024, 25)), (_norm(128, 264, 64), _norm(128, 512, 64)),
    (_norm(200, 256, 25, True), _norm(200, 1024, 25, True)), (_norm(128, 264, 64, True), _norm(128, 512, 64, True)),
    (_norm(8000, 1088), _norm(8000, 1536)), (_norm(8000, 1088, None, True), _norm(8000, 1536, None, True))],
    ids=["one_token", "four_tokens", "fp32_tokens", "planes", "fast_planes", "planes_backward", "fast_planes_backward",
         "rows", "rows_backward"])
def test_head_shapes_side_by_side(small, large):
    _run([small, large, small, large])


def _conv(shape, dtype, algo, tuning=None):
    def make():
        import torch
        from dense_convolution_gb300.conv import Conv2d
        N, Ci, H, W, Co, K = shape
        op = Conv2d(N, Ci, H, W, Co, K, K, 1, 0, dtype, algo, tuning=tuning)
        t = {"f32": torch.float32, "f16": torch.float16}[dtype]
        x = torch.randn(N, Ci, H, W, device="cuda").to(t)
        w = torch.randn(Co, Ci, K, K, device="cuda").to(t)
        ws, y = op.alloc_workspace(), op.alloc_output()
        want = op(x, w)
        return (lambda: op(x, w, y=y, workspace=ws)), lambda got: None if got.equal(want) else pytest.fail("another result")
    return make


@pytest.mark.parametrize("small,large", [
    (_conv((1, 64, 12, 12, 64, 3), "f16", "implicit_tc", {"stages": 2}), _conv((1, 64, 12, 12, 64, 3), "f16", "implicit_tc")),
    (_conv((1, 4, 12, 12, 16, 3), "f32", "implicit_fp32_cc"), _conv((1, 16, 12, 100, 64, 3), "f32", "implicit_fp32_cc")),
    (_conv((1, 4, 12, 12, 16, 3), "f32", "im2win_fp32_cc"), _conv((1, 4, 12, 900, 16, 3), "f32", "im2win_fp32_cc")),
    (_conv((1, 3, 12, 40, 64, 3), "f16", "im2win_tc"), _conv((1, 16, 12, 40, 64, 7), "f16", "im2win_tc")),
    (_conv((1, 24, 12, 12, 64, 3), "f16", "im2win_tc"), _conv((1, 256, 12, 40, 64, 3), "f16", "im2win_tc"))],
    ids=["tensor_core", "fp32", "strips", "window_rows", "window_tiles"])
def test_convolutions_side_by_side(small, large):
    _run([small, large, small, large])
