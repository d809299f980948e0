"""A host thread whose first CUDA call is one of the library's."""
import threading

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq
from test_epilogue_gpu import _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 2, 8, 40, 100, 300])
def test_first_call_of_a_thread(M):
    K, N = 1024, 512
    X, s, Q, sc, z = _layer(M, K, N, M, scaled=True)
    want = awq.w4a16_gemm(X, s, Q, sc, z)
    Y, st = torch.zeros_like(want), awq.new_status("cuda")
    ws = torch.zeros(awq.gemm_workspace_size(M, K, N), dtype=torch.uint8, device="cuda")
    args = (X.data_ptr(), s.data_ptr(), Q.data_ptr(), sc.data_ptr(), z.data_ptr(), M, K, N, Y.data_ptr(), ws.data_ptr(),
            ws.numel(), st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    code = []
    t = threading.Thread(target=lambda: code.append(awq.lib().awq_w4a16_gemm(*args)))
    t.start()
    t.join(30)
    torch.cuda.synchronize()
    assert code == [awq.OK]
    awq.raise_on_status(st)
    assert torch.equal(Y, want)
