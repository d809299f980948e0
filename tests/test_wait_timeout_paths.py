"""The bounded waits of every matmul path, run out for real.

In the build whose waits give up at once (see test_wait_timeout), each tile path, with and
without an epilogue, and the scale search must end, record AWQ_ERR_DEVICE_TIMEOUT when
a wait ran out, and leave nothing in flight: the copies and tensor-core products issued
land before a CTA exits, whichever of its warps gave up.  The regular library then
computes the same bits as before on the same context.
"""
import ctypes

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq
from test_epilogue_gpu import _layer
from test_wait_timeout import waitlib  # noqa: F401  (the module's fixture: the test build)

pytestmark = pytest.mark.gpu
P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


def _p(t):
    return None if t is None else t.data_ptr()


# decode, register-fed, tcgen05 small batch, stream-K and one tile per CTA
@pytest.mark.parametrize("M,K,N", [(1, 8192, 1024), (2, 4096, 2048), (5, 4096, 1024), (20, 10240, 4096), (30, 4096, 1024),
                                   (60, 8192, 2048), (100, 2048, 512), (256, 4096, 1024), (1100, 1024, 9472)])
@pytest.mark.parametrize("epilogue", [False, True])
def test_matmul_waits_run_out_and_the_context_survives(waitlib, M, K, N, epilogue):  # noqa: F811
    f = waitlib.awq_w4a16_gemm_epilogue
    f.argtypes = [P, P, P, P, P, I64, I64, I64, P, I32, I32, P, P, P, SZ, P, P]
    f.restype = ctypes.c_int
    X, s, Q, sc, z = _layer(M, K, N, M, scaled=True)
    b = r = None
    act = 0
    if epilogue:
        b, r, act = torch.randn(N, device="cuda").half(), torch.randn(M, N, device="cuda").half(), awq.ACTIVATIONS["silu"]
    name = "silu" if epilogue else None
    before = awq.w4a16_gemm_epilogue(X, s, Q, sc, z, bias=b, act=name, residual=r)
    for _ in range(3):
        ws = torch.zeros(awq.gemm_workspace_size(M, K, N), dtype=torch.uint8, device="cuda")
        Y, st = torch.zeros(M, N, dtype=torch.float16, device="cuda"), awq.new_status("cuda")
        torch.cuda.synchronize()
        rc = f(_p(X), _p(s), _p(Q), _p(sc), _p(z), M, K, N, _p(b), act, 0, _p(r), _p(Y), _p(ws), ws.numel(), _p(st),
               torch.cuda.current_stream().cuda_stream)
        assert rc == awq.OK
        torch.cuda.synchronize()              # the kernels finished: no hang, no fault
        # a short call's waits may all find their data landed at the first poll: then nothing ran out and Y is right
        code = int(st)
        assert code == awq.ERR_TIMEOUT or (code == awq.OK and torch.equal(Y, before))
        st = awq.new_status("cuda")
        assert torch.equal(awq.w4a16_gemm_epilogue(X, s, Q, sc, z, bias=b, act=name, residual=r, status=st), before)
        awq.raise_on_status(st)


def test_scale_search_waits_run_out_and_the_context_survives(waitlib):  # noqa: F811
    f = waitlib.awq_scale_search
    f.argtypes = [P, I64, I64, P, I64, P, P, P, P, SZ, P, P]
    f.restype = ctypes.c_int
    R, K, N = 200, 2048, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(R, K, generator=g, device="cuda").half()
    W = (torch.randn(K, N, generator=g, device="cuda") * 0.02).half()
    before = awq.scale_search(x, W)
    ws = torch.zeros(awq.scale_search_workspace_size(R, K, N), dtype=torch.uint8, device="cuda")
    losses, best = torch.zeros(9, dtype=torch.float64, device="cuda"), torch.zeros(K, dtype=torch.float16, device="cuda")
    j, st = torch.zeros(1, dtype=torch.int32, device="cuda"), awq.new_status("cuda")
    torch.cuda.synchronize()
    rc = f(_p(x), R, K, _p(W), N, _p(losses), _p(best), _p(j), _p(ws), ws.numel(), _p(st),
           torch.cuda.current_stream().cuda_stream)
    assert rc == awq.OK
    torch.cuda.synchronize()
    assert int(st) == awq.ERR_TIMEOUT
    for a, b in zip(awq.scale_search(x, W), before):
        assert torch.equal(a, b)


def test_quantizer_waits_run_out_and_the_context_survives(waitlib):  # noqa: F811
    f = waitlib.awq_quantize_pack
    f.argtypes = [P, P, I64, I64, P, P, P, P, P]
    f.restype = ctypes.c_int
    K, N = 4096, 6144
    g = torch.Generator(device="cuda").manual_seed(2)
    W, s = torch.randn(K, N, generator=g, device="cuda").half(), torch.ones(K, dtype=torch.float16, device="cuda")
    before = awq.quantize_pack(W, s)
    for _ in range(3):
        Q, sc, z = (torch.zeros_like(t) for t in before)
        st = awq.new_status("cuda")
        torch.cuda.synchronize()
        assert f(_p(W), _p(s), K, N, _p(Q), _p(sc), _p(z), _p(st), torch.cuda.current_stream().cuda_stream) == awq.OK
        torch.cuda.synchronize()
        code = int(st)      # garbage read too early may also look like a value that is not finite
        assert code in (awq.ERR_TIMEOUT, awq.ERR_NONFINITE) or (code == awq.OK and torch.equal(Q, before[0]))
        assert all(torch.equal(a, b) for a, b in zip(awq.quantize_pack(W, s), before))
