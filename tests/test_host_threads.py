"""Host threads that share a stream: a call's kernels, which pass data through the stream's workspace, are
enqueued together.  No GPU: the C entry points are replaced by ones that watch who is inside."""
import threading
import time
import types

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq

CPU = torch.device("cpu")


class Watch:
    """Stands for a C call: the most calls that were inside at once, by stream (the last argument)."""

    def __init__(self):
        self.inside, self.most, self.meet = {}, {}, None

    def __call__(self, *args):
        s = args[-1]
        n = self.inside[s] = self.inside.get(s, 0) + 1
        self.most[s] = max(self.most.get(s, 0), n)
        if self.meet:
            self.meet.wait(10)
        time.sleep(0.02)          # as a C call does, this lets other threads run
        self.inside[s] -= 1
        return awq.OK


@pytest.fixture
def calls(monkeypatch):
    """The binding's entry points on host tensors, every C call a Watch; `stream` gives each thread's stream."""
    w, stream = Watch(), {}
    mine = lambda *a: stream.get(threading.get_ident(), 7)
    fake = types.SimpleNamespace(
        awq_w4a16_gemm=w, awq_w4a16_gemm_epilogue=w, awq_w4a16_gemv=w, awq_kv4_attention=w,
        awq_w4a16_gemm_workspace_size=lambda *a: 64, awq_w4a16_gemv_workspace_size=lambda *a: 64)
    monkeypatch.setattr(awq, "lib", lambda: fake)
    monkeypatch.setattr(awq, "_raw_stream", mine)
    monkeypatch.setattr(awq, "_stream", mine)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", mine)
    monkeypatch.setattr(awq, "_current_device", lambda: None)
    monkeypatch.setattr(awq, "_capturing", lambda: False)
    monkeypatch.setattr(awq, "_need", lambda *a: None)
    for cache in ("_workspaces", "_kv4_workspaces", "_stream_locks"):
        if hasattr(awq, cache):
            monkeypatch.setattr(awq, cache, {})
    X, Q = torch.zeros(3, 128, dtype=torch.float16), torch.zeros(16, 16, dtype=torch.int32)
    sc, z = torch.zeros(1, 16, dtype=torch.float16), torch.zeros(1, 2, dtype=torch.int32)
    layers = []
    for act in (None, "silu"):
        l = object.__new__(awq.QuantLinear)
        l.K, l.N, l.device, l.out_features, l._dev_index, l._lib = 128, 16, CPU, 16, None, fake
        l._plain, l._wptrs, l._bptr, l._act, l._gate = act is None, (None, 1, 1, 1), None, awq.ACTIVATIONS[act], 0
        layers.append(l)
    cache = object.__new__(awq.KV4Cache)
    cache.pages = types.SimpleNamespace(device=CPU, max_requests=1)
    cache.head_dim, cache.kv_heads, cache._lib, cache._workspace_size, cache._read = 64, 1, fake, 64, ()
    q = torch.zeros(1, 1, 64, dtype=torch.float16)
    return types.SimpleNamespace(watch=w, stream=stream, all={
        "gemm": lambda **k: awq.w4a16_gemm(X, None, Q, sc, z, **k), "gemv": lambda **k: awq.w4a16_gemv(X[:1], None, Q, sc, z, **k),
        "epilogue": lambda **k: awq.w4a16_gemm_epilogue(X, None, Q, sc, z, act="silu", **k),
        "layer": lambda **k: layers[0](X, **k), "fused layer": lambda **k: layers[1](X, **k),
        "attention": lambda **k: cache.attention(q, **k)})


def _together(jobs, stream=None, streams=None):
    errors, go = [], threading.Barrier(len(jobs))

    def work(i, job):
        try:
            if streams:
                stream[threading.get_ident()] = streams[i]
            go.wait(10)
            for _ in range(4):
                job()
        except BaseException as e:
            errors.append(e)
    ts = [threading.Thread(target=work, args=(i, j)) for i, j in enumerate(jobs)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(60)
    assert not errors, errors


@pytest.mark.parametrize("name", ["gemm", "gemv", "epilogue", "layer", "fused layer", "attention"])
def test_calls_of_threads_on_one_stream_stay_together(calls, name):
    _together([calls.all[name]] * 3)
    assert calls.watch.most == {7: 1}


def test_different_calls_on_one_stream_stay_together(calls):
    _together(list(calls.all.values()))
    assert calls.watch.most == {7: 1}


@pytest.mark.parametrize("name", ["fused layer", "attention"])
def test_streams_do_not_wait_for_each_other(calls, name):
    calls.watch.meet = threading.Barrier(2)     # both calls have to be inside at once
    _together([calls.all[name]] * 2, calls.stream, [8, 9])
    assert calls.watch.most == {8: 1, 9: 1}


def test_own_workspaces_take_no_lock(calls):
    calls.watch.meet = threading.Barrier(2)
    ws = [torch.zeros(64, dtype=torch.uint8) for _ in range(2)]
    _together([lambda w=w: calls.all["fused layer"](workspace=w) for w in ws])
    assert calls.watch.most == {7: 2}


def test_a_failed_call_frees_its_stream(calls, monkeypatch):
    bad = lambda *a: awq.ERR_CUDA
    for owner in (awq.lib(),):
        monkeypatch.setattr(owner, "awq_kv4_attention", bad)
    with pytest.raises(awq.AwqError):
        calls.all["attention"]()
    done = []
    t = threading.Thread(target=lambda: done.append(calls.all["gemm"]()))
    t.start()
    t.join(10)
    assert done
