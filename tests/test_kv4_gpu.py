"""The paged 4-bit key/value cache on the GPU, against plain 64-bit statements.

Page tables and stored bytes are exact; the attention is held to a bound that
counts the kernel's roundings element by element (kv4_reference.attention).
"""
import random

import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantization_quantize_b200 as awq

pytestmark = pytest.mark.gpu


def _rows(T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g)
    x[..., ::29] *= 5
    return x.half()


def _bytes(t):
    return t.cpu().numpy().copy()


# ------------------------------------------------------------------ page tables
@pytest.mark.parametrize("B,page,total_extra,cached,new", [
    (1, 16, 0, 0, 1), (1, 64, 3, 0, 300), (3, 16, 5, 40, 9), (37, 32, 1, 500, 33), (513, 16, 7, 70, 1),
    (4096, 16, 0, 33, 2), (100, 256, 11, 1000, 700), (9, 128, 0, 128, 128), (5, 16, 9000, 10, 4000)])
def test_reserve_matches_a_plain_restatement(B, page, total_extra, cached, new):
    r = random.Random(B * page + new)
    lens = [r.randint(0, cached) for _ in range(B)]
    add = [r.choice([0, new, r.randint(0, new)]) for _ in range(B)]
    add[0] = new
    held = [-(-n // page) for n in lens]
    max_pages = -(-(cached + new) // page) + 1
    num = sum(-(-(a + b) // page) for a, b in zip(lens, add)) + 3
    order = list(range(num))
    r.shuffle(order)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at: at + h]
        at += h
    free = np.array(order[at:] + [-1] * at, np.int32)
    total = sum(add) + total_extra
    want = ref.reserve(add, lens, table, free, num - at, page, total)

    def state():
        return awq.KV4Pages(num, page, B, max_pages, block_table=torch.from_numpy(table).cuda(),
                            lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            free_pages=torch.from_numpy(free).cuda(),
                            free_count=torch.tensor([num - at], dtype=torch.int32, device="cuda"))
    nl = torch.tensor(add, dtype=torch.int32, device="cuda")
    for in_place in (True, False):
        p, st = state(), awq.new_status("cuda")
        nxt = None if in_place else torch.full((B,), -5, dtype=torch.int32, device="cuda")
        nf = None if in_place else torch.full((1,), -5, dtype=torch.int32, device="cuda")
        slots, pos, cu = p.reserve(nl, total, next_lens=nxt, next_free=nf, status=st)
        awq.raise_on_status(st)
        got = (slots, pos, cu, p.lens if in_place else nxt, (p.free_count if in_place else nf), p.block_table)
        for g, w, name in zip(got, want, ("slots", "positions", "cu", "lens", "free_count", "table")):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
        if not in_place:
            assert p.lens.tolist() == lens and int(p.free_count) == num - at
            p.reserve(nl, total)   # the same step again, now in place
            assert p.lens.tolist() == want[3].tolist()
    # release some requests: pages go back in order
    done = [int(r.random() < 0.5) for _ in range(B)]
    st = awq.new_status("cuda")
    p.release(torch.tensor(done, dtype=torch.int32, device="cuda"), status=st)
    awq.raise_on_status(st)
    back = [int(x) for b in range(B) if done[b] for x in want[5][b, : -(-int(want[3][b]) // page)]]
    count = want[4] + len(back)
    assert int(p.free_count) == count
    assert p.free_pages.cpu().numpy()[:count].tolist() == free[: want[4]].tolist() + back
    assert p.lens.tolist() == [0 if d else int(n) for d, n in zip(done, want[3])]
    for b in range(B):
        n = -(-int(want[3][b]) // page)
        row = p.block_table[b].tolist()
        assert row[:n] == ([-1] * n if done[b] else want[5][b, :n].tolist())


def test_refused_steps_change_nothing():
    def fresh():
        return awq.KV4Pages(6, 16, 3, 4, lens=torch.tensor([17, 0, 5], dtype=torch.int32, device="cuda"),
                            block_table=torch.tensor([[4, 1, -1, -1], [-1] * 4, [3, -1, -1, -1]], dtype=torch.int32, device="cuda"),
                            free_pages=torch.tensor([0, 2, 5, -1, -1, -1], dtype=torch.int32, device="cuda"),
                            free_count=torch.tensor([3], dtype=torch.int32, device="cuda"))
    for add, total, code in [([16, 48, 0], 64, awq.ERR_CAPACITY), ([1, -1, 0], 10, awq.ERR_RANGE),
                             ([48, 0, 0], 60, awq.ERR_RANGE), ([3, 3, 3], 8, awq.ERR_RANGE),
                             ([2**31 - 1, 2**31 - 1, 2**31 - 1], 8, awq.ERR_RANGE)]:
        p, st = fresh(), awq.new_status("cuda")
        before = [t.clone() for t in (p.block_table, p.lens, p.free_pages, p.free_count)]
        slots, pos, cu = p.reserve(torch.tensor(add, dtype=torch.int32, device="cuda"), total, status=st)
        assert int(st) == code
        assert bool((slots == -1).all()) and bool((pos == -1).all()) and bool((cu == 0).all())
        for a, b in zip(before, (p.block_table, p.lens, p.free_pages, p.free_count)):
            assert torch.equal(a, b)
    p, st = fresh(), awq.new_status("cuda")
    p.block_table[0, 1] = 99   # a page that the cache does not have
    before = [t.clone() for t in (p.block_table, p.lens, p.free_pages, p.free_count)]
    p.release(torch.ones(3, dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE
    for a, b in zip(before, (p.block_table, p.lens, p.free_pages, p.free_count)):
        assert torch.equal(a, b)
    p, st = fresh(), awq.new_status("cuda")
    p.free_count.fill_(5)      # more pages than the cache has would be free
    p.release(torch.ones(3, dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE and int(p.free_count) == 5


# ------------------------------------------------------------------ store and load
def _edge_rows(x):
    """Rows at the ends of the range: zeros, one sign, the largest, subnormals, one value."""
    D = x.shape[-1]
    edges = torch.stack([torch.zeros(D), torch.full((D,), 65504.0), torch.full((D,), -65504.0),
                         torch.linspace(-65504, 65504, D), torch.linspace(5, 6, D), torch.linspace(-6, -5, D),
                         torch.full((D,), 2.0**-24), torch.linspace(-2.0**-20, 2.0**-20, D), torch.full((D,), -0.0),
                         torch.arange(D) % 16 / 4.0]).half()
    n = min(len(edges), x.shape[0])
    x[:n, 0] = edges[:n]
    return x


@pytest.mark.parametrize("T,H,D,page,fused", [(1, 1, 64, 16, False), (1, 8, 128, 16, True), (37, 3, 128, 32, True),
                                              (130, 2, 64, 64, True), (515, 8, 128, 256, False), (64, 5, 64, 128, True)])
def test_stored_bytes_and_values(T, H, D, page, fused):
    k, v = _edge_rows(_rows(T, H, D, T)), _edge_rows(_rows(T, H, D, T + 1)).flip(0).contiguous()
    pages = -(-T // page) + 2
    p = awq.KV4Pages(pages, page, 1, pages)
    c = awq.KV4Cache(p, H, D)
    c.data.random_(0, 256)
    want = _bytes(c.data)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T]
    if T > 2:
        slots[1] = -1
        slots[T - 1] = -(1 << 40)
    ref.store(want, k.numpy(), v.numpy(), slots.tolist(), page)
    if fused:
        row = torch.randn(T, 3 * H * D + 8).half().cuda()
        row[:, H * D: 2 * H * D], row[:, 2 * H * D: 3 * H * D] = k.cuda().flatten(1), v.cuda().flatten(1)
        kd, vd = row[:, H * D: 2 * H * D].unflatten(1, (H, D)), row[:, 2 * H * D: 3 * H * D]
    else:
        kd, vd = k.cuda(), v.cuda()
    st = awq.new_status("cuda")
    c.append(kd, vd, slots.cuda(), status=st)
    awq.raise_on_status(st)
    assert np.array_equal(_bytes(c.data), want)
    # read back, a slot twice and one that holds nothing
    ask = torch.cat([slots, slots[:1], torch.tensor([-3])])
    gk, gv = c.load(ask.cuda(), status=st)
    awq.raise_on_status(st)
    real = (ask >= 0).numpy()
    wk, wv, _, _ = ref.values(want, ask.clamp_min(0).numpy(), page, D)
    for g, w in ((gk, wk), (gv, wv)):
        w = torch.from_numpy(np.where(real[:, None, None], w, 0.0)).half()   # one rounding
        assert torch.equal(g.cpu(), w)


def test_bad_slots_and_values_are_reported():
    H, D, page = 2, 64, 16
    p = awq.KV4Pages(3, page, 1, 3)
    c = awq.KV4Cache(p, H, D)
    k, v = _rows(3, H, D, 1), _rows(3, H, D, 2)
    want = _bytes(c.data)
    slots = [5, 3 * page, 47]
    ref.store(want, k.numpy()[[0, 2]], v.numpy()[[0, 2]], [5, 47], page)
    st = awq.new_status("cuda")
    c.append(k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE
    assert np.array_equal(_bytes(c.data), want)
    st = awq.new_status("cuda")
    gk, gv = c.load(torch.tensor([3 * page, 1 << 50], device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE and not gk.any() and not gv.any()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for which in (0, 1):
            x = [k.clone(), v.clone()]
            x[which][1, 1, 7] = bad
            st = awq.new_status("cuda")
            c.append(x[0].cuda(), x[1].cuda(), torch.tensor([0, 1, 2], device="cuda"), status=st)
            assert int(st) == awq.ERR_NONFINITE
            # the other tokens are stored as ever
            wk, wv, _, _ = ref.values(_bytes(c.data), [0, 2], page, D)
            one = np.zeros_like(want)
            ref.store(one, k.numpy(), v.numpy(), [0, 1, 2], page)
            rk, rv, _, _ = ref.values(one, [0, 2], page, D)
            assert np.array_equal(wk, rk) and np.array_equal(wv, rv)


# ------------------------------------------------------------------ attention
def _filled(lens, H, D, page, seed, spare=3, poison=True, max_pages=None):
    """Pages and a cache with lens[b] tokens each; every unused byte poisoned (steps NaN, zero points 65535)."""
    B = len(lens)
    held = [-(-n // page) for n in lens]
    num = sum(held) + spare
    mp = max_pages or max(max(held), 1)
    order = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at: at + h]
        at += h
    p = awq.KV4Pages(num, page, B, mp, block_table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    data = torch.full((num, H, awq.kv4_page_bytes(page, D)), 0xFF if poison else 0, dtype=torch.uint8, device="cuda")
    c = awq.KV4Cache(p, H, D, data=data)
    slots = torch.cat([table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
                       for b, n in enumerate(lens)] or [torch.zeros(0, dtype=torch.long)])
    if len(slots):
        c.append(_rows(len(slots), H, D, seed + 1).cuda(), _rows(len(slots), H, D, seed + 2).cuda(), slots.cuda())
    return p, c, table


def _check_attention(c, table, q, cu, lens, max_new, window=0, scale=None, use_cu=True, extra_rows=0):
    D = c.head_dim
    T = q.shape[0]
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, q.shape[1], D), 7.0, dtype=torch.float16, device="cuda")
    st = awq.new_status("cuda")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda") if use_cu else None
    got = c.attention(q.cuda(), cu=cud, max_new=max_new, scale=scale, window=window, out=out, status=st)
    awq.raise_on_status(st)
    assert got is out
    want, bound = ref.attention(q, _bytes(c.data), table.numpy(), lens, cu, c.pages.page_size, scale, window)
    g = out.cpu().double()
    n = cu[-1]
    err = (g[:n] - want[:n]).abs()
    assert bool((err <= bound[:n]).all()), float((err / bound[:n].clamp_min(1e-300)).max())
    assert bool((g[n:] == 7.0).all()), "rows behind the last request"
    return out


@pytest.mark.parametrize("D,Hk,group,page", [(128, 2, 4, 16), (128, 1, 8, 64), (64, 3, 1, 32), (64, 2, 5, 16),
                                             (128, 2, 7, 256), (128, 1, 16, 128), (64, 1, 40, 16), (128, 8, 1, 16)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 15, 16, 17, 31, 32, 33], [1000, 3, 0, 257], [4099]])
def test_single_tokens(D, Hk, group, page, lens):
    p, c, table = _filled(lens, Hk, D, page, seed=len(lens) + D + page)
    q = _rows(len(lens) + 2, Hk * group, D, 9)
    cu = list(range(len(lens) + 1))
    a = _check_attention(c, table, q, cu, lens, 1)
    b = _check_attention(c, table, q, cu, lens, 1, use_cu=False)
    assert torch.equal(a, b)
    _check_attention(c, table, q, cu, lens, 1, window=1)
    _check_attention(c, table, q, cu, lens, 1, window=20, scale=0.3)


@pytest.mark.parametrize("D,Hk,group,page", [(128, 2, 4, 16), (64, 2, 1, 32), (128, 1, 8, 64), (64, 1, 6, 16)])
@pytest.mark.parametrize("lens,new", [([40, 5, 33], [3, 5, 1]), ([300, 64, 0, 17], [7, 0, 0, 17]), ([700], [90]),
                                      ([130, 129, 1], [130, 65, 1]), ([515, 40], [33, 40])])
def test_runs_of_tokens(D, Hk, group, page, lens, new):
    p, c, table = _filled(lens, Hk, D, page, seed=sum(lens) + D)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = _rows(cu[-1] + 3, Hk * group, D, 11)
    _check_attention(c, table, q, cu, lens, max(new))
    _check_attention(c, table, q, cu, lens, max(new) + 500)
    _check_attention(c, table, q, cu, lens, max(new), window=19)


def test_more_queries_than_cached_tokens_and_empty_requests():
    # queries before the first token see nothing and give zeros
    p, c, table = _filled([3, 0], 2, 128, 16, seed=5)
    q = _rows(9, 8, 128, 1)
    out = _check_attention(c, table, q, [0, 5, 9], [3, 0], 5)
    assert not out[:2].any() and not out[5:9].any()


@pytest.mark.parametrize("new", [3, 5, 90])
def test_windows_over_every_position_are_none(new):
    # the longest window, and queries that stand before the first token
    p, c, table = _filled([3], 2, 128, 16, seed=6)
    q = _rows(new, 8, 128, 1)
    whole = _check_attention(c, table, q, [0, new], [3], new)
    for window in (16, 2**31 - 1):
        assert torch.equal(_check_attention(c, table, q, [0, new], [3], new, window=window), whole)


def test_large_and_small_magnitudes():
    # keys and values at both ends of the format: no overflow of weights times steps, no loss to subnormals
    H, D, page = 1, 128, 16
    for kmag, vmag in [(1.0, 60000.0), (1.0, 2e-4), (1000.0, 1.0), (1e-3, 1e-3)]:
        p, c, table = _filled([200], H, D, page, seed=3)
        k, v = _rows(200, H, D, 1).float() / 25 * kmag, _rows(200, H, D, 2).float() / 25 * vmag
        pos = torch.arange(200)
        c.append(k.half().cuda(), v.half().cuda(), (table[0].long()[pos // page] * page + pos % page).cuda())
        _check_attention(c, table, _rows(1, 8, D, 4), [0, 1], [200], 1)


def test_strided_queries_and_out_of_order_streams():
    lens, Hk, D = [77, 300], 2, 128
    p, c, table = _filled(lens, Hk, D, 32, seed=8)
    fused = _rows(2, 8 + 4, D, 3).cuda()
    q = fused[:, :8]
    want, bound = ref.attention(q, _bytes(c.data), table.numpy(), lens, [0, 1, 2], 32, D ** -0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = c.attention(q)
    torch.cuda.current_stream().wait_stream(side)
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    assert torch.equal(out, c.attention(q))


def test_bad_pages_and_lengths_are_reported_and_not_followed():
    lens, Hk, D, page = [64, 40], 2, 64, 16
    p, c, table = _filled(lens, Hk, D, page, seed=4)
    q = _rows(2, 4, D, 2)
    for bad in (-1, p.num_pages, 2**31 - 1):
        p.block_table.copy_(table.cuda())
        p.block_table[0, 3] = bad   # its tokens 48..63 are not seen
        st = awq.new_status("cuda")
        out = c.attention(q.cuda(), status=st)
        assert int(st) == awq.ERR_RANGE
        want, bound = ref.attention(q, _bytes(c.data), table.numpy(), [48, 40], [0, 1, 2], page, D ** -0.5)
        assert bool(((out.cpu().double() - want).abs() <= bound).all())
    p.block_table.copy_(table.cuda())
    p.lens[1] = 1000   # longer than its row of the table: clamped, and the missing pages skipped
    st = awq.new_status("cuda")
    out = c.attention(q.cuda(), status=st)
    assert int(st) == awq.ERR_RANGE
    want, bound = ref.attention(q, _bytes(c.data), table.numpy(), [64, 40], [0, 1, 2], page, D ** -0.5)
    assert bool(((out.cpu().double() - want)[0].abs() <= bound[0]).all())
    p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    for cu in ([0, 3, 2], [0, 1, 9], [-1, 1, 2]):
        st = awq.new_status("cuda")
        c.attention(q.cuda(), cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_new=2, status=st)
        assert int(st) == awq.ERR_RANGE


def test_offsets_beyond_32_bits():
    # a cache of over 4 GB whose last pages are used, for store, load and attention
    H, D, page = 8, 128, 16
    num = (5 << 30) // (H * awq.kv4_page_bytes(page, D))
    data = torch.empty(num, H, awq.kv4_page_bytes(page, D), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[num - 1, 2, num - 3, num // 2]], dtype=torch.int32)
    p = awq.KV4Pages(num, page, 1, 4, block_table=table.cuda(), lens=torch.tensor([59], dtype=torch.int32, device="cuda"))
    c = awq.KV4Cache(p, H, D, data=data)
    pos = torch.arange(59)
    slots = (table[0].long()[pos // page] * page + pos % page).cuda()
    k, v = _rows(59, H, D, 1), _rows(59, H, D, 2)
    c.append(k.cuda(), v.cuda(), slots)
    gk, gv = c.load(slots)
    small = np.zeros((4, H, awq.kv4_page_bytes(page, D)), np.uint8)
    ref.store(small, k.numpy(), v.numpy(), pos.tolist(), page)
    wk, wv, _, _ = ref.values(small, pos.numpy(), page, D)
    assert torch.equal(gk.cpu(), torch.from_numpy(wk).half()) and torch.equal(gv.cpu(), torch.from_numpy(wv).half())
    q = _rows(1, 16, D, 3)
    want, bound = ref.attention(q, small, np.arange(4)[None], [59], [0, 1], page, D ** -0.5)
    assert bool(((c.attention(q.cuda()).cpu().double() - want).abs() <= bound).all())


def test_captured_graphs_follow_lengths_and_do_not_share_workspaces():
    # two graphs captured on one stream, replayed at the same time on two others, with lengths changed in between
    Hk, D, page = 4, 128, 16
    made = []
    side = torch.cuda.Stream()
    for n in range(2):
        p, c, table = _filled([900, 2000], Hk, D, page, seed=n)
        q = _rows(2, 16, D, 5 + n).cuda()
        out = torch.zeros(2, 16, D, dtype=torch.float16, device="cuda")
        c.attention(q, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.attention(q, out=out)
        made.append((g, p, c, table, q, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([900, 2000], [513, 64], [1, 1999]):
        for g, p, c, table, q, out in made:
            p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for (g, *_), s in zip(made, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, p, c, table, q, out in made:
            want, bound = ref.attention(q.cpu(), _bytes(c.data), table.numpy(), lens, [0, 1, 2], page, D ** -0.5)
            assert bool(((out.cpu().double() - want).abs() <= bound).all())
            assert torch.equal(out, c.attention(q))   # the same bits as an eager call


def test_arguments_are_checked_before_any_launch():
    p, c, table = _filled([20], 2, 64, 16, seed=1)
    q = _rows(1, 4, 64, 1).cuda()
    out = torch.full((1, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    for bad in (dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(max_new=0), dict(window=-1),
                dict(out=out[:, :2]), dict(out=out.float()), dict(cu=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(cu=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(q=q[:0])):
        args = dict(q=q, out=out)
        args.update(bad)
        with pytest.raises((TypeError, ValueError, awq.AwqError)):
            c.attention(args.pop("q"), **args)
    s = torch.zeros(1, dtype=torch.int64, device="cuda")
    k = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=k.cpu()), dict(slots=s.int()), dict(slots=s.new_zeros(2))):
        args = dict(k=k, v=k, slots=s)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            c.append(**args)
    with pytest.raises(TypeError):
        c.load(s.int())
    with pytest.raises(ValueError):
        c.load(s.view(1, 1))
    nl = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (dict(total=0), dict(new_lens=nl.long()), dict(new_lens=nl.new_zeros(2)), dict(next_free=nl.new_zeros(2))):
        args = dict(new_lens=nl, total=4)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            p.reserve(**args)
    with pytest.raises(ValueError):
        awq.KV4Pages(4, 24, 1, 4)
    with pytest.raises(ValueError):
        awq.KV4Pages(4, 16, 4097, 4)
    with pytest.raises(ValueError):
        awq.KV4Pages(4, 16, 1, 2**27)
    with pytest.raises(ValueError):
        awq.KV4Cache(p, 2, 96)
    with pytest.raises(ValueError):
        awq.KV4Cache(p, 2, 64, data=torch.zeros(2, 2, 8, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("D,Hk,group,page", [(128, 1, 4, 16), (64, 2, 3, 64)])
@pytest.mark.parametrize("lens,new,window", [([3000, 1500, 70, 5], [70, 33, 70, 5], 0), ([3000, 1500, 70, 5], [70, 33, 70, 5], 700),
                                             ([4097], [300], 0), ([200], [200], 64)])
def test_prompts_whose_keys_are_split(D, Hk, group, page, lens, new, window):
    # a wide table and few row blocks: the keys go to several CTAs, some of which see none
    p, c, table = _filled(lens, Hk, D, page, seed=sum(lens) + D, max_pages=-(-8192 // page))
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = _rows(cu[-1] + 2, Hk * group, D, 13)
    a = _check_attention(c, table, q, cu, lens, max(new), window=window)
    b = _check_attention(c, table, q, cu, lens, max(new), window=window)
    assert torch.equal(a, b)


def test_prompt_rows_with_extreme_steps_and_scales():
    # value steps six decades apart, logits that keep growing, and both signs of the scale
    H, D, page, n = 1, 128, 16, 700
    p, c, table = _filled([n], H, D, page, seed=31)
    g = torch.Generator().manual_seed(1)
    k = torch.randn(n, H, D, generator=g) * torch.linspace(0.02, 3.0, n)[:, None, None]
    v = torch.randn(n, H, D, generator=g) * (10.0 ** (torch.arange(n) % 7 - 3))[:, None, None]
    pos = torch.arange(n)
    c.append(k.half().cuda(), v.half().cuda(), (table[0].long()[pos // page] * page + pos % page).cuda())
    for m in (1, 20, 120, 700):
        q = torch.randn(m, 4, D, generator=g).half()
        for scale in (0.088, -0.088, 1.5, 0.0):
            _check_attention(c, table, q, [0, m], [n], m, scale=scale)


def test_stored_zeros_are_attended_to():
    # slots that were never written (all bytes zero): keys and values of zero, an even average
    for m in (1, 100):
        p, c, table = _filled([300], 1, 64, 16, seed=2, poison=False)
        c.data.zero_()
        k = _rows(4, 1, 64, 3)
        at = torch.tensor([17, 100, 150, 299])
        c.append(k.cuda(), k.cuda(), (table[0].long()[at // 16] * 16 + at % 16).cuda())
        _check_attention(c, table, _rows(m, 2, 64, 1), [0, m], [300], m)


def test_two_caches_at_the_same_time():
    # calls on two streams, each with its stream's workspace, decode and prompt kernels mixed
    made = []
    for i, (lens, new) in enumerate([([900, 4000], [1, 1]), ([600, 333], [600, 200])]):
        p, c, table = _filled(lens, 2, 128, 32, seed=40 + i)
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        q = _rows(cu[-1], 8, 128, 41 + i).cuda()
        want, bound = ref.attention(q.cpu(), _bytes(c.data), table.numpy(), lens, cu, 32, 128 ** -0.5)
        made.append((c, q, torch.tensor(cu, dtype=torch.int32, device="cuda"), max(new), want, bound, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for o, (c, q, cu, most, _, _, s) in zip(outs, made):
            with torch.cuda.stream(s):
                o.append(c.attention(q, cu=cu, max_new=most))
    torch.cuda.synchronize()
    for o, (c, q, cu, most, want, bound, s) in zip(outs, made):
        for x in o:
            assert bool(((x.cpu().double() - want).abs() <= bound).all()) and torch.equal(x, o[0])


def test_captured_step_grows_the_cache():
    # reserve, store and attention in one graph: each replay adds a token to every request
    B, Hk, D, page = 3, 2, 64, 16
    p = awq.KV4Pages(40, page, B, 8)
    c = awq.KV4Cache(p, Hk, D)
    st = awq.new_status("cuda")
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(B, (4 + 2 * Hk) * D, dtype=torch.float16, device="cuda")
    q, k, v = qkv[:, : 4 * D].unflatten(1, (4, D)), qkv[:, 4 * D: (4 + Hk) * D], qkv[:, (4 + Hk) * D:]
    out = torch.zeros(B, 4, D, dtype=torch.float16, device="cuda")

    def step():
        slots, _, _ = p.reserve(new, B, status=st)
        c.append(k, v, slots, status=st)
        c.attention(q, out=out, status=st)
    step()   # outside the graph first
    p.release(new)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    tokens = []
    for i in range(37):
        x = _rows(B, 1, qkv.shape[1], 50 + i)[:, 0]
        tokens.append(x)
        qkv.copy_(x)
        g.replay()
        awq.raise_on_status(st)
        if i in (0, 15, 16, 36):
            assert p.lens.tolist() == [i + 1] * B and int(p.free_count) == 40 - B * -(-(i + 1) // page)
            table = p.block_table.cpu().numpy()
            cache = np.zeros_like(_bytes(c.data))
            for j, tk in enumerate(tokens):
                slots = [int(table[b, j // page]) * page + j % page for b in range(B)]
                ref.store(cache, tk[:, 4 * D: (4 + Hk) * D].reshape(B, Hk, D).numpy(),
                          tk[:, (4 + Hk) * D:].reshape(B, Hk, D).numpy(), slots, page)
            want, bound = ref.attention(x[:, : 4 * D].reshape(B, 4, D), cache, table, [i + 1] * B, [0, 1, 2, 3], page, D ** -0.5)
            assert bool(((out.cpu().double() - want).abs() <= bound).all())


def test_mixed_batches():
    # prompts, chunks and single tokens in one call: two kernels share the requests between them
    lens = [700, 33, 512, 1, 2000, 90, 0, 300, 64]
    new = [500, 1, 12, 1, 60, 90, 0, 13, 3]
    for D, Hk, group, page in ((128, 2, 4, 16), (64, 1, 7, 32)):
        p, c, table = _filled(lens, Hk, D, page, seed=D)
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        q = _rows(cu[-1] + 5, Hk * group, D, 17)
        _check_attention(c, table, q, cu, lens, max(new))
        _check_attention(c, table, q, cu, lens, max(new), window=100)
    # many requests of which a few have queries
    lens = [20 + i % 50 for i in range(600)]
    new = [0] * 600
    for i in range(0, 600, 37):
        new[i] = 1 + i % 19
    new[599], lens[599] = 60, 69
    p, c, table = _filled(lens, 1, 64, 16, seed=77)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    _check_attention(c, table, _rows(cu[-1], 4, 64, 3), cu, lens, 60)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_pages_before_the_window_may_be_gone(new):
    # a sliding window's user frees the pages that no query sees any more
    for page, window, n in ((16, 50, 500), (32, 64, 333), (128, 200, 1000)):
        p, c, table = _filled([n, 3 * page], 2, 64, page, seed=page)
        first = n - new - window + 1           # the first position that a query of request 0 sees
        gone = first // page
        assert gone > 0
        p.block_table[0, :gone] = -1
        q = _rows(2 * new, 8, 64, 5)
        _check_attention(c, table, q, [0, new, 2 * new], [n, 3 * page], new, window=window)


@pytest.mark.parametrize("fill", [0xFF, 0x80, 0x7F, 0x00])
@pytest.mark.parametrize("lens,new,window", [([4000, 900], [300, 90], 60), ([4000, 900], [300, 90], 0), ([2000, 33, 512], [60, 1, 12], 0),
                                             ([900, 4000], [1, 1], 0)])
def test_workspaces_may_hold_anything(lens, new, window, fill):
    # the grid of a prompt call is a bound on its row blocks: those that no request has are skipped, whatever the
    # workspace held where they would stand
    p, c, table = _filled(lens, 4, 128, 64, seed=sum(lens))
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = _rows(cu[-1], 8, 128, 23)
    around = torch.full((3, cu[-1], 8, 128), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.full((awq.kv4_attention_workspace_size(128),), fill, dtype=torch.uint8, device="cuda")
    st = awq.new_status("cuda")
    out = c.attention(q.cuda(), cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_new=max(new), window=window,
                      out=around[1], status=st, workspace=ws)
    awq.raise_on_status(st)
    want, bound = ref.attention(q, _bytes(c.data), table.numpy(), lens, cu, 64, 128 ** -0.5, window)
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    assert bool((around[0] == 7.0).all()) and bool((around[2] == 7.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,new,max_pages", [
    ([40, 1, 300], [1, 1, 1], None), ([77, 9], [6, 3], None),          # few rows
    ([200, 90], [120, 40], None), ([300, 2], [300, 30], None),         # prompts, keys in one piece; queries before the first token
    ([1500, 700], [70, 33], 64), ([4000, 3], [90, 60], 64)])           # prompts whose keys are split
def test_queries_that_are_not_finite_show(bad, lens, new, max_pages):
    # an overflow upstream reaches the output of its own rows on every path, and no other row
    p, c, table = _filled(lens, 2, 128, 64, seed=sum(lens), max_pages=max_pages)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    clean = _rows(cu[-1], 8, 128, 29)
    want, bound = ref.attention(clean, _bytes(c.data), table.numpy(), lens, cu, 64, 128 ** -0.5)
    hit = torch.zeros(cu[-1], 8, dtype=torch.bool)
    for b in range(len(lens)):
        hit[cu[b], 3] = hit[cu[b + 1] - 1, 6] = True
    q = clean.clone()
    q[..., 5][hit] = bad
    st = awq.new_status("cuda")
    out = c.attention(q.cuda(), cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_new=max(new), status=st).cpu().double()
    awq.raise_on_status(st)
    sees = torch.cat([torch.arange(n - m, n) >= 0 for n, m in zip(lens, new)])
    gone = hit & sees[:, None]
    assert bool(out[gone].isnan().all())
    assert bool(((out - want).abs() <= bound)[~gone].all())


@pytest.mark.parametrize("written", [0, 1, 40])
@pytest.mark.parametrize("m,max_pages", [(1, None), (100, None), (100, 64)])
def test_whole_tiles_of_stored_zeros(written, m, max_pages):
    # runs of slots that were never written, longer than a key tile, before and between written ones
    n, page = 700, 64
    p, c, table = _filled([n], 1, 128, page, seed=5, poison=False, max_pages=max_pages)
    c.data.zero_()
    at = torch.arange(written) * 11 + 230
    k = _rows(written, 1, 128, 3)
    if written:
        c.append(k.cuda(), k.cuda(), (table[0].long()[at // page] * page + at % page).cuda())
    q = _rows(m, 2, 128, 1)
    out = _check_attention(c, table, q, [0, m], [n], m)
    if not written:
        assert not out.any()
    _check_attention(c, table, q, [0, m], [n], m, window=150)


@pytest.mark.parametrize("m", [1, 3, 60])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_infinite_logits_of_a_single_key_show(m, bad):
    # one cached token whose codes make the infinite query's logit -inf in one head and +inf in the other
    p, c, table = _filled([1], 1, 64, 16, seed=1)
    k = torch.zeros(1, 1, 64, dtype=torch.float16)
    k[..., 5], k[..., 9] = -2.0, 2.0
    c.append(k.cuda(), torch.ones_like(k).cuda(), (table[0, :1].long() * 16).cuda())
    q = _rows(m, 2, 64, 1)
    q[-1, 0, 5] = q[-1, 1, 9] = bad
    st = awq.new_status("cuda")
    out = c.attention(q.cuda(), cu=torch.tensor([0, m], dtype=torch.int32, device="cuda"), max_new=m, status=st)
    awq.raise_on_status(st)
    assert bool(out[-1].isnan().all()) and not out[:-1].any()   # the earlier queries stand before the first token


def test_wide_tables_and_long_chunks():
    # the bounds of a server: 256 rows of 65536 tokens, a chunk of up to 2048 tokens among single ones
    B, Hk, D, page = 256, 8, 64, 16
    lens = [33 + i % 40 for i in range(B)]
    new = [1] * B
    new[7], lens[7] = 130, 700
    new[100] = 0
    p, c, table = _filled(lens, Hk, D, page, seed=3, max_pages=4096)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    _check_attention(c, table, _rows(cu[-1], 32, D, 5), cu, lens, 2048)


@pytest.mark.parametrize("bad", [-1, -7, 12, 2**31 - 1])
@pytest.mark.parametrize("total_extra", [0, 5000])
def test_reserve_reports_bad_pages_and_does_not_follow_them(bad, total_extra):
    # a held page and a page on the stack that the cache does not have: their tokens have no slot, the others do
    page, table, free = 16, [[4, 1, -1, -1], [6, -1, -1, -1], [3, -1, -1, -1]], [0, 2, 5, 7]
    lens, add = [17, 9, 16], [20, 3, 18]       # request 0 goes on in page 1 and takes 7; 2 takes 5 and 2
    total = sum(add) + total_extra
    for where in ("none", "held", "free"):
        t, f = np.array(table, np.int32), np.array(free + [-1] * 8, np.int32)
        if where == "held":
            t[1, 0] = bad
        if where == "free":
            f[2] = bad
        want = list(ref.reserve(add, lens, t, f, 4, page, total))
        if where == "held":
            want[0][20:23] = -1
        if where == "free":
            want[0][23:39] = -1
            want[5][2, 1] = -1
        p = awq.KV4Pages(12, page, 3, 4, block_table=torch.from_numpy(t).cuda(), free_pages=torch.from_numpy(f).cuda(),
                         lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         free_count=torch.tensor([4], dtype=torch.int32, device="cuda"))
        st = awq.new_status("cuda")
        slots, pos, cu = p.reserve(torch.tensor(add, dtype=torch.int32, device="cuda"), total, status=st)
        assert int(st) == (awq.OK if where == "none" else awq.ERR_RANGE)
        for g, w, name in zip((slots, pos, cu, p.lens, p.free_count, p.block_table), want,
                              ("slots", "positions", "cu", "lens", "free_count", "table")):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), (where, name)


@pytest.mark.parametrize("B,page,most", [(1, 16, 40), (5, 32, 700), (300, 16, 90), (4096, 16, 3), (7, 256, 5000)])
def test_release_passes_over_pages_that_are_gone(B, page, most):
    # rows that have given back pages before their window, and rows that have not, in one call
    r = random.Random(B)
    held = [r.randint(0, most) for _ in range(B)]
    lens = [h * page - r.randint(0, page - 1) if h else 0 for h in held]
    gone = [r.choice([0, r.randint(0, h), max(h - 1, 0)]) for h in held]
    done = [int(r.random() < 0.6) for _ in range(B)]
    done[0] = 1
    num = sum(held) + 4
    order = list(range(num))
    r.shuffle(order)
    table = np.full((B, most + 1), -1, np.int32)
    free = order[sum(held):]
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at: at + h]
        free += table[b, : gone[b]].tolist()       # given back by their holder
        table[b, : gone[b]] = -1
        at += h
    if held[0] > gone[0] + 2:                      # and one out of the middle
        free.append(int(table[0, gone[0] + 1]))
        table[0, gone[0] + 1] = -1
    p = awq.KV4Pages(num, page, B, most + 1, block_table=torch.from_numpy(table).cuda(),
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     free_pages=torch.tensor(free + [-1] * (num - len(free)), dtype=torch.int32, device="cuda"),
                     free_count=torch.tensor([len(free)], dtype=torch.int32, device="cuda"))
    st = awq.new_status("cuda")
    p.release(torch.tensor(done, dtype=torch.int32, device="cuda"), status=st)
    awq.raise_on_status(st)
    back = [int(x) for b in range(B) if done[b] for x in table[b, : held[b]] if x >= 0]
    count = len(free) + len(back)
    assert int(p.free_count) == count
    assert p.free_pages[:count].tolist() == free + back
    assert p.lens.tolist() == [0 if d else n for d, n in zip(done, lens)]
    for b in range(B):
        if done[b]:
            table[b, : held[b]] = -1
    assert np.array_equal(p.block_table.cpu().numpy(), table)


def test_a_request_under_a_window_gives_its_pages_back_and_ends():
    # as a server runs it: tokens appended and attended to under a window, pages before it given back as they leave it
    page, window, D = 16, 40, 64
    p = awq.KV4Pages(8, page, 1, 40)               # 8 pages for a request of 33 pages: only with the window
    c = awq.KV4Cache(p, 1, D)
    st, gone, host = awq.new_status("cuda"), 0, np.zeros((40, 1, awq.kv4_page_bytes(page, D)), np.uint8)
    for i, m in enumerate([30] + [7] * 70):
        slots, pos, cu = p.reserve(torch.tensor([m], dtype=torch.int32, device="cuda"), m, status=st)
        k, v, q = _rows(m, 1, D, 3 * i), _rows(m, 1, D, 3 * i + 1), _rows(m, 2, D, 3 * i + 2)
        c.append(k.cuda(), v.cuda(), slots, status=st)
        out = c.attention(q.cuda(), cu=cu, max_new=m, window=window, status=st)
        awq.raise_on_status(st)
        ref.store(host, k.numpy(), v.numpy(), pos.tolist(), page)
        n = int(p.lens)
        if i % 10 == 0:
            want, bound = ref.attention(q, host, np.arange(40)[None], [n], [0, m], page, D ** -0.5, window)
            assert bool(((out.cpu().double() - want).abs() <= bound).all())
        while (gone + 1) * page <= n - window + 1:  # the next query stands at n and sees n - window + 1 on
            p.free_pages[p.free_count.long()] = p.block_table[0, gone]
            p.block_table[0, gone] = -1
            p.free_count += 1
            gone += 1
    assert gone > 20
    p.release(torch.ones(1, dtype=torch.int32, device="cuda"), status=st)
    awq.raise_on_status(st)
    assert int(p.free_count) == 8 and sorted(p.free_pages.tolist()) == list(range(8)) and int(p.lens) == 0
    assert bool((p.block_table == -1).all())


@pytest.mark.parametrize("bad", [-2, 6, 2**31 - 1, -2**31])
def test_release_refuses_pages_outside_the_cache(bad):
    table = torch.tensor([[4, -1, bad, 2], [1, 3, -1, -1]], dtype=torch.int32, device="cuda")
    p = awq.KV4Pages(6, 16, 2, 4, block_table=table, lens=torch.tensor([60, 20], dtype=torch.int32, device="cuda"),
                     free_pages=torch.tensor([0, 5, -1, -1, -1, -1], dtype=torch.int32, device="cuda"),
                     free_count=torch.tensor([2], dtype=torch.int32, device="cuda"))
    state = (p.block_table, p.lens, p.free_pages, p.free_count)
    before = [t.clone() for t in state]
    st = awq.new_status("cuda")
    p.release(torch.ones(2, dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE and all(torch.equal(a, b) for a, b in zip(before, state))
    st = awq.new_status("cuda")
    p.free_count.fill_(5)          # two pages would make seven of six
    p.release(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == awq.ERR_RANGE and p.lens.tolist() == [60, 20] and int(p.free_count) == 5
    st = awq.new_status("cuda")
    p.free_count.fill_(2)
    p.release(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), status=st)
    awq.raise_on_status(st)
    assert p.free_pages.tolist()[:4] == [0, 5, 1, 3] and int(p.free_count) == 4
