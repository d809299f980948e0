"""Host threads that share a stream, with the library's own kernels: results are those of one thread."""
import threading

import numpy as np
import pytest
import torch

import weight_only_quantization_quantize_b200 as awq
from test_epilogue_gpu import _layer
from test_kv4_gpu import _filled, _rows

pytestmark = pytest.mark.gpu


def _attention(lens, new, seed, max_pages=None):
    p, c, _ = _filled(lens, 2, 128, 32, seed=seed, max_pages=max_pages)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, cud = _rows(cu[-1], 8, 128, seed).cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    return lambda: c.attention(q, cu=cud, max_new=max(new))


def _linear(M, seed):
    X, s, Q, sc, z = _layer(M, 2048, 1024, seed, scaled=True)
    lin = awq.QuantLinear(Q, sc, z, s, act="silu")
    return lambda: lin(X)


def _noalloc(M, seed):
    X, s, Q, sc, z = _layer(M, 2048, 1024, seed, scaled=True)

    def call():
        Y = torch.empty(M, 1024, dtype=torch.float16, device="cuda")
        code = awq.lib().awq_w4a16_gemm_noalloc(X.data_ptr(), s.data_ptr(), Q.data_ptr(), sc.data_ptr(), z.data_ptr(), M, 2048,
                                                1024, Y.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
        assert code == awq.OK
        return Y
    return call


@pytest.mark.parametrize("own_stream", [False, True])
def test_threads_get_what_one_thread_gets(own_stream):
    # split decode and prompt attention, mixed batches, products with a pre-pass and with partial tiles
    jobs = [_attention([4000, 900], [1, 1], 1), _attention([3000, 2000], [1, 1], 2), _attention([1500, 700], [60, 33], 3, 256),
            _attention([900, 333], [200, 1], 4, 256), _linear(8, 5), _linear(40, 6), _linear(100, 7), _linear(16, 8)]
    if not own_stream:      # its scratch array is one for the device: calls on one stream only
        jobs += [_noalloc(16, 9), _noalloc(20, 10)]
    wants = [j() for j in jobs]
    torch.cuda.synchronize()
    outs, errors, go = [[] for _ in jobs], [], threading.Barrier(len(jobs))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own_stream else torch.cuda.default_stream()):
                go.wait(30)
                for _ in range(40):
                    outs[i].append(jobs[i]())
                torch.cuda.current_stream().synchronize()
        except BaseException as e:
            errors.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join(120)
    torch.cuda.synchronize()
    assert not errors, errors
    for i, (got, want) in enumerate(zip(outs, wants)):
        assert len(got) == 40 and all(torch.equal(g, want) for g in got), i
