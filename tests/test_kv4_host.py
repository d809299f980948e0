"""Host-side refusals of the cache's and the epilogue's entry points: no launch, no GPU."""
import ctypes

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq

A = 0x7F0000000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from weight_only_quantization_quantize_b200 import _build
    _build.build()
    return awq.lib()


def test_page_bytes(L):
    for page in (16, 32, 64, 128, 256):
        for d in (64, 128):
            assert L.awq_kv4_page_bytes(page, d) == page * (d + 8)   # half a byte per code, 4 bytes per row and tensor
    for page, d in ((8, 64), (24, 64), (512, 128), (0, 64), (-16, 64), (16, 96), (16, 0)):
        assert L.awq_kv4_page_bytes(page, d) == 0
    with pytest.raises(ValueError):
        awq.kv4_page_bytes(48, 64)
    assert L.awq_kv4_attention_workspace_size(128) > L.awq_kv4_attention_workspace_size(64) > 0
    assert L.awq_kv4_attention_workspace_size(80) == 0


def test_reserve_refusals(L):
    def call(new=A, lens=A, B=4, page=16, table=A, mp=8, free=A, count=A, num=32, T=4, slots=A, pos=A, cu=A, lo=A, co=A, st=None):
        return L.awq_kv4_reserve(P(new), P(lens), B, page, P(table), mp, P(free), P(count), num, T, P(slots), P(pos),
                                 P(cu), P(lo), P(co), P(st), None)
    for name in ("new", "lens", "table", "free", "count", "slots", "cu", "lo", "co"):
        assert call(**{name: 0}) == awq.ERR_NULL, name
        assert call(**{name: A + 2}) == awq.ERR_ALIGN, name
    assert call(slots=A + 4) == awq.ERR_ALIGN
    assert call(st=A + 1) == awq.ERR_ALIGN
    for bad in (dict(B=0), dict(B=4097), dict(page=17), dict(page=512), dict(mp=0), dict(mp=1 << 28), dict(num=0),
                dict(num=1 << 31), dict(T=0), dict(T=1 << 31)):
        assert call(**bad) == awq.ERR_SHAPE, bad


def test_release_refusals(L):
    def call(done=A, lens=A, B=4, page=16, table=A, mp=8, free=A, count=A, num=32, st=None):
        return L.awq_kv4_release(P(done), P(lens), B, page, P(table), mp, P(free), P(count), num, P(st), None)
    for name in ("done", "lens", "table", "free", "count"):
        assert call(**{name: 0}) == awq.ERR_NULL
        assert call(**{name: A + 1}) == awq.ERR_ALIGN
    assert call(page=20) == awq.ERR_SHAPE and call(B=-1) == awq.ERR_SHAPE


def test_append_and_load_refusals(L):
    def app(k=A, ks=256, v=A, vs=256, slots=A, T=3, H=2, D=128, cache=A, num=8, page=16, st=None):
        return L.awq_kv4_append(P(k), ks, P(v), vs, P(slots), T, H, D, P(cache), num, page, P(st), None)

    def load(slots=A, T=3, H=2, D=128, cache=A, num=8, page=16, k=A, v=A, st=None):
        return L.awq_kv4_load(P(slots), T, H, D, P(cache), num, page, P(k), P(v), P(st), None)
    for f, names in ((app, ("k", "v", "slots", "cache")), (load, ("k", "v", "slots", "cache"))):
        for name in names:
            assert f(**{name: 0}) == awq.ERR_NULL
            assert f(**{name: A + 4}) == awq.ERR_ALIGN
        for bad in (dict(T=0), dict(T=1 << 31), dict(H=0), dict(H=1025), dict(D=96), dict(num=0), dict(page=8)):
            assert f(**bad) == awq.ERR_SHAPE
    assert app(ks=248) == awq.ERR_SHAPE and app(vs=0) == awq.ERR_SHAPE
    assert app(ks=260) == awq.ERR_ALIGN


def test_attention_refusals(L):
    def call(q=A, qs=1024, T=4, H=8, cache=A, num=32, page=16, Hk=2, D=128, table=A, mp=8, lens=A, cu=A, B=4, mn=1,
             scale=0.1, window=0, out=A, ws=A, wsb=1 << 40, st=None):
        return L.awq_kv4_attention(P(q), qs, T, H, P(cache), num, page, Hk, D, P(table), mp, P(lens), P(cu), B, mn, scale,
                                   window, P(out), P(ws), wsb, P(st), None)
    for name in ("q", "cache", "table", "lens", "out"):
        assert call(**{name: 0}) == awq.ERR_NULL
        assert call(**{name: A + 2}) == awq.ERR_ALIGN
    for bad in (dict(T=0), dict(H=9), dict(H=0), dict(H=2048, Hk=1), dict(Hk=0), dict(D=32), dict(page=48), dict(mp=0),
                dict(B=0), dict(B=4097), dict(mn=0), dict(mn=1 << 31), dict(window=-1), dict(window=1 << 31),
                dict(qs=1016), dict(num=0), dict(cu=0, T=3), dict(mn=1 << 24, mp=1 << 26)):
        assert call(**bad) == awq.ERR_SHAPE, bad
    assert call(qs=1028) == awq.ERR_ALIGN
    assert call(ws=0) == awq.ERR_WORKSPACE and call(wsb=100) == awq.ERR_WORKSPACE


def test_epilogue_refusals(L):
    def call(X=A, Q=A, sc=A, z=A, M=4, K=256, N=32, b=A, act=0, gated=0, r=A, Y=A, ws=A, wsb=1 << 40, st=None):
        return L.awq_w4a16_gemm_epilogue(P(X), None, P(Q), P(sc), P(z), M, K, N, P(b), act, gated, P(r), P(Y), P(ws), wsb,
                                         P(st), None)
    for name in ("X", "Q", "sc", "Y"):
        assert call(**{name: 0}) == awq.ERR_NULL
    for name in ("X", "Q", "sc", "z", "Y", "b", "r"):
        assert call(**{name: A + 2}) == awq.ERR_ALIGN, name
    for bad in (dict(act=-1), dict(act=5), dict(N=24, gated=1), dict(K=100), dict(M=0)):
        assert call(**bad) == awq.ERR_SHAPE, bad
    assert call(ws=0) == awq.ERR_WORKSPACE and call(wsb=16) == awq.ERR_WORKSPACE


def test_interleaved_weights():
    g, u = torch.arange(6.0).reshape(2, 3), -torch.arange(6.0).reshape(2, 3)
    w = awq.interleave_gate_up(g, u)
    assert w.shape == (2, 6) and torch.equal(w[:, 0::2], g) and torch.equal(w[:, 1::2], u)
    b = awq.interleave_gate_up(g[0], u[0])
    assert torch.equal(b[0::2], g[0]) and torch.equal(b[1::2], u[0])
    with pytest.raises(ValueError):
        awq.interleave_gate_up(g, u[:1])


def test_host_tensors_are_refused():
    with pytest.raises(TypeError):
        awq.KV4Pages(4, 16, 1, 4, device="cpu")
    with pytest.raises(TypeError):
        awq.KV4Pages(4, 16, 1, 4, block_table=torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        awq.w4a16_gemm_epilogue(torch.zeros(1, 128, dtype=torch.float16), None, None, None, None)


def test_attention_takes_serving_bounds(L):
    # shapes are judged before the workspace: a missing one shows that the bounds were taken
    def call(B, H, Hk, tokens, mn, page=16, D=128):
        return L.awq_kv4_attention(P(A), H * D, 1 << 20, H, P(A), 1 << 20, page, Hk, D, P(A), tokens // page, P(A), P(A), B, mn,
                                   0.1, 0, P(A), None, 0, None, None)
    for B, H, Hk, tokens, mn in ((256, 32, 8, 65536, 2048), (64, 32, 8, 131072, 4096), (8, 64, 64, 131072, 32768),
                                 (8, 64, 8, 131072, 32768), (4096, 64, 8, 131072, 131072), (1, 64, 1, 1 << 24, 1 << 20),
                                 (4096, 8, 8, 1 << 20, 1)):
        assert call(B, H, Hk, tokens, mn) == awq.ERR_WORKSPACE, (B, H, Hk, tokens, mn)
    # one item of a one-page table is 9 units (a tile, and what an item costs besides): 4096 * 1024 * 9 stays below
    # 2^32, 4096 * 1024 * (2^16 / 64 + 8) does not
    assert call(4096, 1024, 1024, 16, 1) == awq.ERR_WORKSPACE
    assert call(4096, 1024, 1024, 1 << 16, 1) == awq.ERR_SHAPE
    # the limit itself: 4096 * 64 * (tokens / 64 + 8) against 2^32, items of 8 rows, then three of 16
    assert call(4096, 64, 64, 64 * (16384 - 9), 8) == awq.ERR_WORKSPACE
    assert call(4096, 64, 64, 64 * (16384 - 8), 8) == awq.ERR_SHAPE
    assert call(4096, 64, 64, 64 * 5453, 33) == awq.ERR_WORKSPACE
    assert call(4096, 64, 64, 64 * 5454, 33) == awq.ERR_SHAPE
    # more than 2^52 query rows times positions
    assert call(1, 8, 2, 1 << 30, 1 << 20) == awq.ERR_WORKSPACE
    assert call(1, 8, 2, 1 << 30, (1 << 20) + 1) == awq.ERR_SHAPE
