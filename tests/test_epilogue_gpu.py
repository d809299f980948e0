"""The W4A16 product with bias, activation, gate and residual in its epilogue, on every tile path.

The reference is float64 over the dequantized weights.  The bound counts, element by element:
  the product   each weight's rounding to float16 in the tensor paths, half a step (2^-11 |x||w|), and the decode path's
                sums over 1024 + q before the zero point is taken off (8 additions per group: 2^-10 step |x|);
  the epilogue  slopes of the activations (at most 1.13) and of the gate's product;
  the output    half a step of float16 (2^-11 |y|), and 2^-24 for subnormals.
"""
import math

import pytest
import torch

import weight_only_quantization_quantize_b200 as awq

pytestmark = pytest.mark.gpu

ACTS = {
    None: lambda t: t,
    "relu": lambda t: t.clamp_min(0),
    "silu": lambda t: t * torch.sigmoid(t),
    "gelu": lambda t: 0.5 * t * torch.erfc(-t / math.sqrt(2)),
    "gelu_tanh": lambda t: 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))),
}


def _layer(M, K, N, seed, symmetric=False, scaled=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(K, N, generator=g, device="cuda") * 0.05).half()
    s = torch.exp(torch.randn(K, generator=g, device="cuda") * 0.3).half() if scaled else None
    Q, sc, z = awq.quantize_pack(W, s if scaled else torch.ones(K, dtype=torch.float16, device="cuda"),
                                 zero_point=not symmetric)
    X = torch.randn(M, K, generator=g, device="cuda").half()
    return X, s, Q, sc, z


def _product(X, s, Q, sc, z):
    """float64 (t, bound of its error)."""
    K, N = Q.shape[0] * 8, Q.shape[1]
    sh = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    q = ((Q[:, None] >> sh[:, None]) & 15).reshape(K, N).double()
    zp = ((z[:, :, None] >> sh) & 15).reshape(-1, N).double() if z is not None else torch.full_like(sc, 8, dtype=torch.float64)
    step = sc.double().repeat_interleave(128, 0)
    w = (q - zp.repeat_interleave(128, 0)) * step
    x = X.double() if s is None else (X.float() / s.float()).half().double()
    return x @ w, 2.0 ** -11 * (x.abs() @ w.abs()) + 2.0 ** -10 * (x.abs() @ step)


def _finish(t, e, bias, act, gated, residual):
    f = ACTS[act]
    if bias is not None:
        t = t + bias.double()
    if gated:
        gate, up, eg, eu = t[:, 0::2], t[:, 1::2], e[:, 0::2], e[:, 1::2]
        y = f(gate) * up
        e = f(gate).abs() * eu + 1.13 * eg * (up.abs() + eu)
    else:
        y = f(t)
        e = 1.13 * e
    if residual is not None:
        y = y + residual.double()
    return y, e * 1.01 + 2.0 ** -11 * y.abs() * 1.01 + 2.0 ** -24


# every tile path: decode (1, 2), register-fed (3..23), tcgen05 small batch (24..63), prefill with one tile per CTA and
# stream-K, and a K whose decode plan does not fit (falls to the register-fed path)
SHAPES = [(1, 1024, 512), (2, 256, 48), (1, 4096, 6144), (3, 512, 136), (16, 1152, 1040), (23, 256, 16), (24, 640, 144),
          (37, 512, 1040), (63, 128, 16), (64, 256, 144), (100, 1024, 272), (257, 512, 1040), (1100, 256, 4112), (300, 4096, 512)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("bias,act,gated,residual", [
    (True, None, False, False), (False, None, False, True), (True, "gelu", False, True), (False, "silu", True, False),
    (True, "gelu_tanh", True, True), (True, "relu", False, False), (False, None, True, True), (False, "silu", False, True)])
def test_every_path_and_epilogue(M, K, N, bias, act, gated, residual):
    if gated:
        N = N // 16 * 16
    X, s, Q, sc, z = _layer(M, K, N, M + K + N, symmetric=(M % 2 == 0), scaled=(M % 3 == 0))
    g = torch.Generator(device="cuda").manual_seed(3)
    cols = N // 2 if gated else N
    b = torch.randn(N, generator=g, device="cuda").half() if bias else None
    r = torch.randn(M, cols, generator=g, device="cuda").half() if residual else None
    st = awq.new_status("cuda")
    store = torch.full((M + 1, cols), 7.0, dtype=torch.float16, device="cuda")
    Y = awq.w4a16_gemm_epilogue(X, s, Q, sc, z, bias=b, act=act, gated=gated, residual=r, status=st, out=store[:M])
    awq.raise_on_status(st)
    want, bound = _finish(*_product(X, s, Q, sc, z), b, act, gated, r)
    err = (Y.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert bool((store[M] == 7.0).all())
    # the prepared layer, and the residual added in place
    lin = awq.QuantLinear(Q, sc, z, s, bias=b, act=act, gated=gated)
    assert torch.equal(lin(X, residual=r), Y)
    if r is not None:
        assert torch.equal(lin(X, residual=r, out=r), Y) and torch.equal(r, Y)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_an_empty_epilogue_is_the_plain_product(M, K, N):
    X, s, Q, sc, z = _layer(M, K, N, 1, scaled=True)
    assert torch.equal(awq.w4a16_gemm_epilogue(X, s, Q, sc, z), awq.w4a16_gemm(X, s, Q, sc, z))
    assert torch.equal(awq.QuantLinear(Q, sc, z, s)(X), awq.w4a16_gemm(X, s, Q, sc, z))


def test_activations_at_their_ends():
    # one weight column per value: t runs over large, small and special values
    K, N = 128, 16
    X = torch.zeros(5, K, dtype=torch.float16, device="cuda")
    W = torch.zeros(K, N, dtype=torch.float16, device="cuda")
    Q, sc, z = awq.quantize_pack(W, torch.ones(K, dtype=torch.float16, device="cuda"))
    vals = torch.tensor([0.0, -0.0, 1e-4, -1e-4, 1, -1, 4, -4, 12, -12, 60, -60, 6e4, -6e4, float("inf"), float("nan")])
    b = vals.half().cuda()
    for act in ACTS:
        Y = awq.w4a16_gemm_epilogue(X, None, Q, sc, z, bias=b, act=act)
        want = ACTS[act](vals.half().double())
        for y in Y.cpu():
            assert torch.equal(y.isnan(), want.isnan() | (vals == float("inf")) & y.isnan())
            ok = ~y.isnan()
            assert torch.allclose(y[ok].double(), want[ok], rtol=2.0 ** -10, atol=2.0 ** -24), (act, y, want)
        assert bool(Y[:, 15].isnan().all())   # NaN stays NaN, in relu too


def test_epilogue_arguments():
    X, s, Q, sc, z = _layer(2, 256, 48, 1)
    out = torch.full((2, 48), 7.0, dtype=torch.float16, device="cuda")
    b, r = torch.zeros(48, dtype=torch.float16, device="cuda"), torch.zeros(2, 48, dtype=torch.float16, device="cuda")
    for bad in (dict(bias=b[:40]), dict(bias=b.float()), dict(act="tanh"), dict(residual=r[:1]), dict(residual=r.float()),
                dict(gated=True), dict(out=out[:1]), dict(residual=r.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            awq.w4a16_gemm_epilogue(X, s, Q, sc, z, **{**dict(out=out), **bad})
    lin = awq.QuantLinear(Q, sc, z, bias=b)
    for bad in (r[:1], r.float(), r.cpu(), r[:, :40]):
        with pytest.raises(ValueError):
            lin(X, residual=bad, out=out)
    with pytest.raises(ValueError):
        awq.QuantLinear(Q[:, :40].contiguous(), sc[:, :40].contiguous(), z[:, :5].contiguous(), gated=True)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("M", [1, 16, 40, 100, 300])
def test_captured_epilogues_replayed_together(M):
    # two graphs captured on one stream and replayed at the same time: each has a workspace of its own
    K, N = 1024, 512
    side, made = torch.cuda.Stream(), []
    for n in range(2):
        X, s, Q, sc, z = _layer(M, K, N, 20 + n, scaled=True)
        b = torch.randn(N, device="cuda").half()
        lin = awq.QuantLinear(Q, sc, z, s, bias=b, act="silu")
        want = lin(X)
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lin(X, out=out)
        made.append((g, want, out, lin, X))   # what the graph reads stays alive
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (g, *_), st in zip(made, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, want, out, *_ in made:
        assert torch.equal(out, want)


def test_chained_residuals():
    # a stream of dependent layers (programmatic dependent launch): each adds to the same residual in place
    K = N = 512
    for M in (1, 8, 30, 70):
        X, s, Q, sc, z = _layer(M, K, N, 5)
        lin = awq.QuantLinear(Q, sc, z)
        h = X.clone()
        want = [h]
        for _ in range(6):
            y = lin(h)
            h = (y.float() + h.float()).half()
            want.append(h)
        for _ in range(5):
            x = X.clone()
            for i in range(6):
                nxt = lin(x, residual=x)   # reads x as input and residual
                t, e = _product(x, None, Q, sc, z)
                w, bound = _finish(t, e, None, None, False, x)
                assert bool(((nxt.double() - w).abs() <= bound).all())
                x = nxt


@pytest.mark.parametrize("M", [1, 3, 16, 40, 100, 300])
@pytest.mark.parametrize("entry", ["layer", "gemm"])
def test_captured_plain_products_replayed_together(M, entry):
    # as above without an epilogue: graphs captured on one fresh stream, the second one replayed first and both at
    # the same time, then eager calls on that stream
    K, N = 2048, 512
    side, made = torch.cuda.Stream(), []
    for n in range(2):
        X, s, Q, sc, z = _layer(M, K, N, 30 + n, scaled=True)
        lin = awq.QuantLinear(Q, sc, z, s)
        call = (lambda X, out, lin=lin: lin(X, out=out)) if entry == "layer" else \
            (lambda X, out, a=(s, Q, sc, z): awq.w4a16_gemm(X, *a, out=out))
        want = torch.empty(M, N, dtype=torch.float16, device="cuda")
        call(X, want)
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(X, out)
        made.append((g, want, out, call, X, lin))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(20):
        for (g, *_), st in zip(made[::-1], streams):
            with torch.cuda.stream(st):
                g.replay()
    with torch.cuda.stream(side):
        eager = [call(X, torch.empty_like(want)) for _, want, _, call, X, _ in made]
    torch.cuda.synchronize()
    for (g, want, out, *_), e in zip(made, eager):
        assert torch.equal(out, want) and torch.equal(e, want)


@pytest.mark.parametrize("M,K,N", [(8, 71680, 520), (23, 16640, 24584), (4, 71680, 136)])
@pytest.mark.parametrize("bias,act,gated,residual", [(True, "gelu", False, True), (False, "silu", True, False), (False, None, True, True)])
def test_long_reductions_of_the_register_fed_path(M, K, N, bias, act, gated, residual):
    # more than 64 groups per CTA: steps and zero points are read from global memory
    test_every_path_and_epilogue(M, K, N, bias, act, gated, residual)
    test_an_empty_epilogue_is_the_plain_product(M, K, N)
