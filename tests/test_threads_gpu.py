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
