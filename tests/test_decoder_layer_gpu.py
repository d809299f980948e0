"""A decoder layer with 4-bit weights and a 4-bit cache, operator after operator as it would be served.

Fused QKV with bias -> pages, store, attention -> O with residual -> gated MLP -> down with residual, for a
ragged batch of prompts and then single tokens.  Every operator's result is held to its own bound, with the
inputs that it really had (the previous operators' outputs), so no tolerance is passed on.
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantization_quantize_b200 as awq
from test_epilogue_gpu import _finish, _product

pytestmark = pytest.mark.gpu


def _linear(K, N, seed, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(K, N, generator=g, device="cuda") * 0.03).half()
    s = awq.compute_scales(awq.act_stats(torch.randn(64, K, generator=g, device="cuda").half()))
    Q, sc, z = awq.quantize_pack(W, s)
    return awq.QuantLinear(Q, sc, z, s, **kw)


def _check(lin, X, Y, residual=None):
    want, bound = _finish(*_product(X, lin.s, lin.Q, lin.scales, lin.zeros), lin.bias, lin.act, lin.gated, residual)
    assert bool(((Y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("D,Hq,Hk,page", [(64, 8, 2, 16), (128, 4, 4, 32)])
def test_prompts_then_tokens(D, Hq, Hk, page):
    hidden, inner = Hq * D, 1024
    g = torch.Generator(device="cuda").manual_seed(9)
    qkv = _linear(hidden, (Hq + 2 * Hk) * D, 1, bias=torch.randn((Hq + 2 * Hk) * D, generator=g, device="cuda").half())
    o, up = _linear(hidden, hidden, 2), _linear(hidden, 2 * inner, 3, act="silu", gated=True)
    down = _linear(inner, hidden, 4)
    B = 3
    pages = awq.KV4Pages(64, page, B, 16)
    cache = awq.KV4Cache(pages, Hk, D)
    host = np.zeros(tuple(cache.data.shape), np.uint8)
    lens = np.zeros(B, np.int64)
    st = awq.new_status("cuda")
    for new in ([90, 1, 33], [1, 1, 1], [1, 0, 1], [3, 2, 0]):
        total = sum(new)
        h = torch.randn(total, hidden, generator=g, device="cuda").half()
        slots, positions, cu = pages.reserve(torch.tensor(new, dtype=torch.int32, device="cuda"), total, status=st)
        lens = lens + new
        assert pages.lens.tolist() == lens.tolist()
        assert positions.tolist() == [int(n) - m + i for n, m in zip(lens, new) for i in range(m)]
        x = qkv(h, status=st)
        _check(qkv, h, x)
        q, k, v = x[:, : hidden].unflatten(1, (Hq, D)), x[:, hidden: hidden + Hk * D], x[:, hidden + Hk * D:]
        cache.append(k, v, slots, status=st)
        ref.store(host, k.reshape(total, Hk, D).cpu().numpy(), v.reshape(total, Hk, D).cpu().numpy(), slots.tolist(), page)
        assert np.array_equal(cache.data.cpu().numpy(), host)
        a = cache.attention(q, cu=cu, max_new=max(new), status=st)
        want, bound = ref.attention(q, host, pages.block_table.cpu().numpy(), lens, cu.tolist(), page, D ** -0.5)
        assert bool(((a.cpu().double() - want).abs() <= bound).all())
        a = a.flatten(1)
        y = o(a, residual=h, status=st)
        _check(o, a, y, h)
        m = up(y, status=st)
        _check(up, y, m)
        z = down(m, residual=y, status=st)
        _check(down, m, z, y)
        awq.raise_on_status(st)
    pages.release(torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda"), status=st)
    awq.raise_on_status(st)
    assert pages.lens.tolist() == [0, int(lens[1]), 0]
    assert int(pages.free_count) == 64 - -(-int(lens[1]) // page)
