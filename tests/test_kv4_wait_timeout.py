"""The bounded waits of the cache's prompt attention kernel, run out for real.

As for the matmul kernels: a test build whose waits give up at once (limit zero, the
timer read on every poll).  The calls must end, record AWQ_ERR_DEVICE_TIMEOUT, and leave a
context on which the regular library computes the same bits as before.  (The split
kernel's only waits are for copies asked for two tiles earlier: they find them landed, so its
time-out cannot be reached this way.)
"""
import ctypes

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq
from test_kv4_gpu import _rows
from test_wait_timeout import waitlib  # noqa: F401  (the module's fixture: the test build)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [60, 300])
def test_attention_waits_run_out_and_the_context_survives(waitlib, new):  # noqa: F811
    P, I64, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    f = waitlib.awq_kv4_attention
    f.argtypes = [P, I64, I64, I64, P, I64, I64, I64, I64, P, I64, P, P, I64, I64, F, I64, P, P, SZ, P, P]
    f.restype = ctypes.c_int
    lens, Hk, D, page = [40000, 30000], 8, 128, 256
    held = [-(-n // page) for n in lens]
    table = torch.full((2, held[0]), -1, dtype=torch.int32)
    table[0, : held[0]], table[1, : held[1]] = torch.arange(held[0]), torch.arange(held[0], sum(held))
    p = awq.KV4Pages(sum(held), page, 2, held[0], block_table=table.cuda(),
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    c = awq.KV4Cache(p, Hk, D)
    c.data.random_(0, 256)                                       # any codes
    words = c.data.view(torch.int32).view(-1, (16 * D + 128) // 4)
    words[:, 4 * D:] = 0x00082E66                                # zero point 8, step 0.1
    q = _rows(2 * new, 8, D, 2).cuda()
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    before = c.attention(q, cu=cu, max_new=new)
    ws = torch.empty(awq.kv4_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros_like(q), awq.new_status("cuda")
    torch.cuda.synchronize()
    rc = f(q.data_ptr(), 8 * D, 2 * new, 8, c.data.data_ptr(), p.num_pages, page, Hk, D, p.block_table.data_ptr(),
           p.max_pages, p.lens.data_ptr(), cu.data_ptr(), 2, new, D ** -0.5, 0, out.data_ptr(), ws.data_ptr(), ws.numel(),
           st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == awq.OK
    torch.cuda.synchronize()              # the kernels finished: no hang, no fault
    assert int(st) == awq.ERR_TIMEOUT
    st = awq.new_status("cuda")
    assert torch.equal(c.attention(q, cu=cu, max_new=new, status=st), before)
    awq.raise_on_status(st)


@pytest.mark.parametrize("lens,new,window", [([700, 300], [300, 300], 0), ([200, 130], [150, 100], 0), ([4000, 900], [300, 90], 60)])
def test_masked_tiles_run_out_and_the_context_survives(waitlib, lens, new, window):  # noqa: F811
    # prompts whose last tiles are masked: the softmax warps' wait for half a tile's product runs out while the
    # issuer's own waits may not; nothing may be in flight when the CTA gives its tensor memory back
    P, I64, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    f = waitlib.awq_kv4_attention
    f.argtypes = [P, I64, I64, I64, P, I64, I64, I64, I64, P, I64, P, P, I64, I64, F, I64, P, P, SZ, P, P]
    f.restype = ctypes.c_int
    Hk, D, page = 4, 128, 64
    held = [-(-n // page) for n in lens]
    table = torch.full((2, held[0]), -1, dtype=torch.int32)
    table[0, : held[0]], table[1, : held[1]] = torch.arange(held[0]), torch.arange(held[0], sum(held))
    p = awq.KV4Pages(sum(held), page, 2, held[0], block_table=table.cuda(),
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    c = awq.KV4Cache(p, Hk, D)
    c.data.random_(0, 256)
    words = c.data.view(torch.int32).view(-1, (16 * D + 128) // 4)
    words[:, 4 * D:] = 0x00083666                                # zero point 8, step 0.4: the reference moves often
    q = _rows(sum(new), 8, D, 3).cuda()
    cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
    before = c.attention(q, cu=cu, max_new=max(new), window=window)
    ws = torch.empty(awq.kv4_attention_workspace_size(D), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        out, st = torch.zeros_like(q), awq.new_status("cuda")
        torch.cuda.synchronize()
        rc = f(q.data_ptr(), 8 * D, sum(new), 8, c.data.data_ptr(), p.num_pages, page, Hk, D, p.block_table.data_ptr(),
               p.max_pages, p.lens.data_ptr(), cu.data_ptr(), 2, max(new), D ** -0.5, window, out.data_ptr(), ws.data_ptr(),
               ws.numel(), st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == awq.OK
        torch.cuda.synchronize()              # the kernels finished: no hang, no fault
        assert int(st) == awq.ERR_TIMEOUT
        st = awq.new_status("cuda")
        assert torch.equal(c.attention(q, cu=cu, max_new=max(new), window=window, status=st), before)
        awq.raise_on_status(st)
