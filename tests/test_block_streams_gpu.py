"""The microscaled 4-bit operators and layer norm on a stream that is not the current
one, while the current one still has work pending on memory that was just freed."""
import pytest

from tests.test_fp4_gpu import qg, torch, _no_device_timeouts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def test_calls_on_another_stream_leave_pending_memory_alone(torch, qg):
    """Blocks of the sizes that the calls allocate are freed while the current stream has yet
    to write to them: what a call on `side` allocates must not be among them."""
    M, N, K = 640, 512, 384
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.Generator("cuda").manual_seed(3)
        X, dY, W = (torch.randn(s, device="cuda", generator=g).to(torch.bfloat16) for s in ((M, K), (M, N), (N, K)))
        gamma = torch.rand(K, device="cuda", generator=g)
        wq, ws, wtq, wts = qg.fp4_quantize_both(W)
        _, mean, rstd = qg.layer_norm(X, gamma, None)

    def everything(**kw):
        q, s = qg.fp4_quantize(X, **kw)
        return [t for out in ((q, s), qg.fp4_quantize_both(X, **kw), (qg.fp4_tensor_scale(X, **kw),),
                              (qg.fp4_dequantize(q, s, K, **kw),), (qg.fp4_gemm(q, s, wq, ws, K, **kw),),
                              (qg.fp4_linear(X, wq, ws, **kw),), qg.fp4_linear_backward(dY, X, wtq, wts, **kw),
                              qg.layer_norm(X, gamma, None, **kw), qg.layer_norm_fp4(X, gamma, None, stats=True, **kw),
                              qg.layer_norm_backward(dY[:, :K], X, gamma, mean, rstd, **kw)) for t in out]

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = everything()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [qg.workspace_size(op, M, N, K) for op in (qg.QG_OP_FP4_LINEAR, qg.QG_OP_FP4_LINEAR_BACKWARD)]
    sizes += [qg.workspace_size(qg.QG_OP_LAYER_NORM_BACKWARD, 1, 1, K), qg.workspace_size(qg.QG_OP_FP4_TENSOR_SCALE, 1, 1, 1)]
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for b in blocks:
        b.fill_(77)
    del blocks, b
    got = everything(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
