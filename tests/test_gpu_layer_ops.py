"""GPU tests of the decoder-layer operators against plain 64-bit references
(tests/layer_ref.py, whose bounds follow the number formats)."""
import math

import numpy as np
import pytest
import torch

import wl_synth
from tests import layer_ref as ref
from tests.parity import assert_canaries, guarded_empty

pytestmark = pytest.mark.gpu

E4, BF = torch.float8_e4m3fn, torch.bfloat16
F64 = torch.float64


def _randn(seed, *s):
    return torch.randn(*s, generator=wl_synth.make_generator(seed))


def _within(got, want, bound, what=""):
    d = (got.to(F64).cpu() - want).abs()
    assert torch.isfinite(d).all(), what
    worst = (d / bound.clamp(min=1e-300)).max()
    assert bool((d <= bound).all()), f"{what}: {float(worst):.3g} times the bound"


# ------------------------------------------------------------------ append --
def _append_case(wl, gpu, lens, n, q_heads, kv, dim, page, dtype, x, rot, interleaved, counts=None, seed=0, positions=None,
                 amplitude=1.0, base=10000.0, spoil=None):
    """Runs wl_rope_append and checks q_out, the written rows, and that nothing else of the cache moved."""
    pg = ref.Paged(wl, gpu, lens, n, kv, dim, page, dtype, counts, seed)
    B = len(lens)
    q, k, v = _randn(seed + 1, B, n, q_heads, dim), _randn(seed + 2, B, n, kv, dim) * 3, _randn(seed + 3, B, n, kv, dim)
    if spoil:
        spoil(q, k, v)
    q, k, v = (t.to(x) for t in (q, k, v))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    rope = wl.RopeTable(ref.phases_of([f / (2 * math.pi) for f in freq]).to(gpu), interleaved, amplitude) if rot else None
    pos = positions if positions is not None else torch.tensor(lens)[:, None] + torch.arange(n)
    buf, q_out, pad = guarded_empty((B, n, q_heads, dim), BF, gpu)
    before = [t.view(torch.uint8 if dtype == E4 else torch.int16).cpu().clone() for t in (pg.cache.k, pg.cache.v)]
    wl.wl_rope_append(q.to(gpu), k.to(gpu), v.to(gpu), None if positions is None else positions.to(gpu, torch.int32), rope, pg.cache,
                      pg.seqs, q_out=q_out)
    torch.cuda.synchronize()
    assert_canaries(buf, pad)

    def turned(t):
        t = t.to(F64).view(B * n, -1, dim)
        return (ref.rotate(t, pos.reshape(-1), freq, interleaved, amplitude) if rot else t).view(B, n, -1, dim)

    # angle 2^-32 turn and sincospi, two products, a sum: 2^-21 of the pair's size
    def slack(t):
        t = t.to(F64).abs() * abs(amplitude)
        return t.amax(-1, keepdim=True).expand_as(t) * 2.0 ** -20 if rot else torch.zeros_like(t)

    counts = counts or [n] * B
    want = turned(q)
    for b in range(B):
        want[b, counts[b]:] = 0
    fin = torch.isfinite(want)
    _within(torch.where(fin, q_out.cpu().to(F64), 0.0), torch.where(fin, want, 0.0),
            ref.bf16_slack(torch.where(fin, want, 0.0)) + torch.where(fin, slack(q), 0.0) + 1e-40, "q")
    assert not torch.isfinite(q_out.cpu()[~fin].float()).any()
    written = torch.zeros(pg.pool, page, dtype=torch.bool)
    codes = {"k": pg.cache.k.cpu(), "v": pg.cache.v.cpu()}
    scales = {"k": pg.cache.k_scale.cpu(), "v": pg.cache.v_scale.cpu()}
    for name, val, sl in (("k", turned(k), slack(k)), ("v", v.to(F64), torch.zeros_like(v, dtype=F64))):
        for b in range(B):
            for i in range(counts[b]):
                p, t = pg.at(b, lens[b] + i)
                written[p, t] = True
                c, s = codes[name][p, :, t].float().to(F64), scales[name][p, :, t].to(F64)
                for h in range(kv):
                    r = val[b, i, h]
                    if not torch.isfinite(r).all():
                        assert torch.isnan(s[h]) and (c[h] == 0).all()
                        continue
                    if dtype == BF:
                        assert s[h] == 1
                        _within(c[h], r, ref.bf16_slack(r) + sl[b, i, h] + 1e-40, name)
                        continue
                    amax, near = float(r.abs().max()), float(sl[b, i, h].max())
                    sc = float(s[h])
                    if amax == 0:
                        assert sc == 1 and (c[h] == 0).all()
                        continue
                    assert math.frexp(sc)[0] == 0.5 and amax - near <= 448 * sc
                    assert sc == 2.0 ** -126 or amax + near > 224 * sc
                    # half a step of 4 significant bits, of the smallest step 2^-9 below 2^-6
                    e = torch.frexp(r / sc)[1].clamp(min=-5)
                    step = torch.ldexp(torch.ones_like(r), e - 5) * sc
                    _within(c[h] * sc, r, step * (1 + 2.0 ** -20) + sl[b, i, h], name)
                    if rot == 0:
                        assert (s[h].float() == ref.row_scale(r[None])[0])
                        assert torch.equal(codes[name][p, h, t].view(torch.uint8), ref.e4m3_codes(r[None].float(), s[h:h + 1].float())[0].view(torch.uint8))
    for old, now in zip(before, (pg.cache.k, pg.cache.v)):
        now = now.view(old.dtype).cpu()
        keep = ~written[:, None].expand(-1, kv, -1)
        assert torch.equal(old[keep], now[keep]), "a row outside the call was written"
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("x", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,rot,interleaved", [
    (256, 256, False), (256, 128, True), (128, 128, False), (128, 36, False), (80, 80, False), (80, 22, True), (16, 16, False),
    (16, 2, True), (48, 30, False), (112, 0, False)])
def test_append_layouts(wl, gpu, dtype, x, dim, rot, interleaved):
    _append_case(wl, gpu, [0, 5, 130], 3, 4, 2, dim, 16, dtype, x, rot, interleaved, seed=dim + rot)


@pytest.mark.parametrize("n,lens,counts,page,kv,group", [
    (1, [0], None, 1, 1, 1), (1, [63, 64], None, 64, 1, 4), (7, [13, 0, 47], [0, 7, 3], 48, 3, 1), (130, [65], None, 32, 1, 2),
    (5, [0, 0], [0, 0], 16, 2, 3), (33, [1, 2, 3], [33, 32, 1], 7, 16, 2)])
def test_append_sequences(wl, gpu, n, lens, counts, page, kv, group):
    for dtype in (E4, BF):
        _append_case(wl, gpu, lens, n, kv * group, kv, 64, page, dtype, BF, 64, False, counts, seed=n)


def test_append_positions_far_out_and_amplitude(wl, gpu):
    """Explicit positions (a tree's, negative, beyond 2^24) and a scaled amplitude."""
    pos = torch.tensor([[0, 1, 1, 2, -5, 131071], [1 << 20, 1 << 24, (1 << 24) + 1, 99999999, 7, 7]])
    _append_case(wl, gpu, [3, 9], 6, 2, 1, 128, 16, E4, torch.float32, 128, False, seed=3, positions=pos, amplitude=1.2079, base=1e6)
    _append_case(wl, gpu, [3, 9], 6, 2, 1, 128, 16, BF, torch.float32, 96, True, seed=4, positions=pos, base=500.0)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_append_extreme_rows(wl, gpu, dtype):
    """Zero rows, subnormals, huge values, rows at the scale's edge, NaN and infinities."""
    def spoil(q, k, v):
        k[0, 0, 0], v[0, 0, 0] = 0.0, 0.0
        v[0, 1, 0] = 1e-38 * torch.randn(64, generator=wl_synth.make_generator(1))
        v[0, 2, 0], v[0, 2, 0, 5] = 1.0, 448.0
        v[0, 3, 0], v[0, 3, 0, 5] = 1.0, -450.0
        v[0, 4, 0, 7], k[0, 4, 0, 9] = math.nan, math.inf
        v[0, 5, 0, 3] = -math.inf
        v[0, 6, 0] = 3e38
        v[0, 7, 0] = 2.0 ** -149
        q[0, 8, 1, 2] = math.nan
        v[0, 9, 0, 1:] *= 2.0 ** -12
    _append_case(wl, gpu, [2], 10, 2, 1, 64, 16, dtype, torch.float32, 0, False, seed=8, spoil=spoil)


def test_append_from_strided_rows_without_q_and_on_a_stream(wl, gpu):
    """k and v as column ranges of one wider matrix; no q; a stream that is not the current one."""
    pg = ref.Paged(wl, gpu, [4, 20], 3, 2, 64, 16, E4, seed=5)
    wide = _randn(6, 6, 8 + 2 * 128 + 8).to(BF).to(gpu)
    k, v = wide[:, 8:136], wide[:, 136:264]
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    assert wl.wl_rope_append(None, k, v, None, None, pg.cache, pg.seqs, stream=side) is None
    side.synchronize()
    vals = {"k": k, "v": v}
    for name, codes, scales in (("k", pg.cache.k, pg.cache.k_scale), ("v", pg.cache.v, pg.cache.v_scale)):
        for b in range(2):
            for i in range(3):
                p, t = pg.at(b, pg.lens[b] + i)
                r = vals[name][b * 3 + i].view(2, 64).float().cpu()
                sc = ref.row_scale(r)
                assert torch.equal(scales[p, :, t].cpu(), sc)
                assert torch.equal(codes[p, :, t].cpu().view(torch.uint8), ref.e4m3_codes(r, sc).view(torch.uint8))


def test_positions_without_a_page_are_skipped_and_reported(wl, gpu):
    pg = ref.Paged(wl, gpu, [14, 3], 4, 1, 64, 16, E4, seed=5)
    pages = pg.table.clone()
    pages[0, 1] = pg.pool  # past the pool
    pages[1, 0] = -1
    cache = wl.KVCache.empty(pg.pool, 1, 16, 64, device=gpu)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x11)
    seqs = wl.CacheSeqs(pages.to(gpu), pg.seqs.len, 4)
    x = torch.ones(8, 64, dtype=BF, device=gpu)
    wl.wl_rope_append(None, x, x, None, None, cache, seqs)
    assert wl.wl_device_status() == wl.WL_ERR_INVALID_ARG and "page" in wl.wl_last_error()
    assert wl.wl_device_status() == wl.WL_OK
    # only positions 14 and 15 of sequence 0 have a page
    rows = (cache.k.view(torch.uint8).cpu() != 0x11).any(-1).nonzero().tolist()
    assert sorted(rows) == sorted([[int(pages[0, 0]), 0, 14], [int(pages[0, 0]), 0, 15]])
    kk, _ = wl.wl_cache_read(cache, seqs)
    assert wl.wl_device_status() == wl.WL_ERR_INVALID_ARG
    kk = kk.float().cpu()
    assert (kk[0, :2] == 1).all() and (kk[0, 2:] == 0).all() and (kk[1] == 0).all()
    out = wl.wl_tree_attention(x.view(2, 4, 1, 64), cache, wl.CacheSeqs(pages.to(gpu), torch.tensor([16, 0], dtype=torch.int32, device=gpu), 4))
    assert wl.wl_device_status() == wl.WL_ERR_INVALID_ARG
    assert torch.isfinite(out[1].float()).all() and (out[1] == 0).all()


# -------------------------------------------------------------------- read --
@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,n,counts,kv,dim,page", [
    ([0], 1, None, 1, 16, 1), ([0, 33, 100], 37, [37, 0, 5], 2, 80, 16), ([7], 300, None, 1, 256, 48), ([64, 1], 65, None, 3, 128, 64)])
def test_read(wl, gpu, dtype, out, lens, n, counts, kv, dim, page):
    pg = ref.Paged(wl, gpu, lens, n, kv, dim, page, dtype, counts, seed=n)
    shape = (len(lens), n, kv, dim)
    (bk, k, pad), (bv, v, _) = guarded_empty(shape, out, gpu), guarded_empty(shape, out, gpu)
    wl.wl_cache_read(pg.cache, pg.seqs, dt=out, outs=(k, v))
    assert_canaries(bk, pad)
    assert_canaries(bv, pad)
    for b in range(len(lens)):
        c = pg.counts[b]
        for name, got in (("k", k), ("v", v)):
            assert torch.equal(got[b, :c].cpu(), pg.rows(name, b, lens[b], c).float().to(out))
            assert (got[b, c:] == 0).all()
    assert wl.wl_device_status() == wl.WL_OK


def test_nan_rows_read_back_as_nan(wl, gpu):
    cache = wl.KVCache.empty(2, 1, 16, 32, device=gpu)
    z = dict(dtype=torch.int32, device=gpu)
    seqs = wl.CacheSeqs(torch.zeros(1, 1, **z), torch.zeros(1, **z), 2)
    x = torch.ones(2, 32, dtype=BF, device=gpu)
    x[1, 3] = math.inf
    wl.wl_rope_append(None, x, x, None, None, cache, seqs)
    k, v = wl.wl_cache_read(cache, seqs, dt=torch.float32)
    assert (k[0, 0] == 1).all() and torch.isnan(k[0, 1]).all() and torch.isnan(v[0, 1]).all()


# --------------------------------------------------------------- attention --
def _attend_case(wl, gpu, lens, n, q_heads, kv, dim, page, dtype, counts=None, mask="tree", seed=0, peak=2.0, scale=None, pg=None,
                 stream=None):
    pg = pg or ref.Paged(wl, gpu, lens, n, kv, dim, page, dtype, counts, seed)
    B = len(lens)
    q = (_randn(seed + 1, B, n, q_heads, dim) * peak).to(BF)
    if isinstance(mask, str):
        mask = ref.tree_masks(B, n, seed) if mask == "tree" else None
    buf, out, pad = guarded_empty(q.shape, BF, gpu)
    qd, md = q.to(gpu), None if mask is None else mask.to(gpu)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream(gpu))
    wl.wl_tree_attention(qd, pg.cache, pg.seqs, mask=md, scale=scale, out=out, stream=stream)
    torch.cuda.synchronize()
    assert_canaries(buf, pad)
    want, bound = ref.attention(pg, q, mask, scale if scale is not None else dim ** -0.5)
    _within(out, want, bound + 1e-40, f"lens {lens} n {n} heads {q_heads}/{kv} dim {dim} page {page} {dtype}")
    assert (out.cpu()[want == 0] == 0).all()
    assert wl.wl_device_status() == wl.WL_OK
    return out


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("lens,n", [([0], 1), ([1], 1), ([127, 128, 129], 1), ([1000], 3), ([40, 300], 17)])
def test_attention_lengths(wl, gpu, dtype, dim, lens, n):
    _attend_case(wl, gpu, lens, n, 4, 2, dim, 16, dtype, seed=dim + n)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("q_heads,kv", [(1, 1), (4, 1), (7, 1), (3, 3), (32, 16), (20, 4)])
@pytest.mark.parametrize("n", [1, 5, 64])
def test_attention_heads(wl, gpu, dtype, q_heads, kv, n):
    _attend_case(wl, gpu, [70, 0], n, q_heads, kv, 128 if kv > 3 else 256, 32, dtype, seed=q_heads + n)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 100, 256])
def test_attention_pages(wl, gpu, dtype, page):
    _attend_case(wl, gpu, [page - 1, 3 * page, 261], 9, 2, 1, 64, page, dtype, seed=page)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_attention_ragged_counts_and_chain(wl, gpu, dtype):
    _attend_case(wl, gpu, [0, 5, 200, 129], 12, 8, 2, 128, 16, dtype, counts=[0, 12, 1, 7], seed=1)
    _attend_case(wl, gpu, [0, 5, 200, 129], 64, 2, 1, 128, 16, dtype, counts=[64, 63, 0, 33], seed=2, mask="chain")


@pytest.mark.parametrize("dtype", [E4, BF])
def test_attention_empty_rows(wl, gpu, dtype):
    """Masks that leave a row nothing (no context, no bit), bits beyond the count, all bits."""
    m = torch.tensor([[0, 1, 0, 7, -1], [0, 0, 0, 0, 0], [-1, 1 << 62, 4, 2, 16]], dtype=torch.int64)
    _attend_case(wl, gpu, [0, 0, 33], 5, 4, 2, 64, 16, dtype, counts=[5, 5, 3], seed=3, mask=m)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_attention_rows_that_are_masked_do_not_leak(wl, gpu, dtype):
    """A drafted token with NaN k and v spoils only the tokens that see it."""
    pg = ref.Paged(wl, gpu, [37], 4, 1, 64, 16, dtype, seed=4)
    mask = torch.tensor([[1, 2, 5, 10]], dtype=torch.int64)  # 0; 1; 0,2; 1,3
    p, t = pg.at(0, 37 + 1)
    for name in ("k", "v"):  # what wl_rope_append stores for a row with a NaN
        codes, scale = getattr(pg.cache, name), getattr(pg.cache, name + "_scale")
        codes.view(torch.uint8)[p, :, t] = 0
        scale[p, :, t] = math.nan
    q = (_randn(7, 1, 4, 4, 64)).to(BF)
    out = wl.wl_tree_attention(q.to(gpu), pg.cache, pg.seqs, mask=mask.to(gpu)).float().cpu()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 3]).all()
    getattr(pg, "vs")[p, :, t] = 1.0
    getattr(pg, "ks")[p, :, t] = 1.0
    pg.k.view(torch.uint8)[p, :, t] = 0
    pg.v.view(torch.uint8)[p, :, t] = 0
    want, bound = ref.attention(pg, q, mask, 64 ** -0.5)
    for i in (0, 2):
        _within(out[0, i], want[0, i], bound[0, i], "a token that does not see the NaN")
    # a NaN or an infinity in one query stays with that query
    q[0, 2, 1, 5], q[0, 0, 2, 1] = math.nan, math.inf
    out = wl.wl_tree_attention(q.to(gpu), pg.cache, pg.seqs, mask=mask.to(gpu)).float().cpu()
    assert torch.isnan(out[0, 2, 1]).all() and torch.isnan(out[0, 0, 2]).all()
    ok = [(0, 0), (0, 1), (0, 3), (2, 0), (2, 2), (2, 3)]
    for i, h in ok:
        _within(out[0, i, h], want[0, i, h], bound[0, i, h], "a query beside a NaN")


@pytest.mark.parametrize("dtype", [E4, BF])
def test_attention_scores_of_all_sizes(wl, gpu, dtype):
    """Flat, peaked and rising scores; keys and values of very different rows; large negative scores."""
    for peak in (0.0, 0.05, 30.0, 300.0):
        _attend_case(wl, gpu, [700], 6, 4, 1, 128, 16, dtype, seed=11, peak=peak)
    # scores that rise along the sequence: the running maximum moves in every tile
    for sign in (1.0, -1.0):
        pg = ref.Paged(wl, gpu, [1500], 2, 1, 64, 16, dtype, seed=12)
        for j in range(1502):
            p, t = pg.at(0, j)
            for name, s in (("k", "ks"), ("v", "vs")):
                x = torch.randn(1, 64, generator=wl_synth.make_generator(j))
                if name == "k":
                    x = x * 0.1 + sign * j / 100.0
                sc = ref.row_scale(x) if dtype == E4 else torch.ones(1)
                getattr(pg, s)[p, :, t] = sc
                getattr(pg, name)[p, :, t] = ref.e4m3_codes(x, sc) if dtype == E4 else x.to(BF)
        pg.upload(wl)
        _attend_case(wl, gpu, [1500], 2, 4, 1, 64, 16, dtype, seed=13, pg=pg, peak=1.0)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_attention_one_token_outweighs_a_long_tail(wl, gpu, dtype):
    """A token with a far larger score beside 20000 equal small ones whose sum counts."""
    L = 20000
    pg = ref.Paged(wl, gpu, [L], 1, 1, 32, 64, dtype, seed=14)
    one = torch.ones(32)
    for name, s in (("k", "ks"), ("v", "vs")):
        x = torch.zeros(pg.pool, 1, 64, 32)
        if name == "v":
            x[:] = 1.0
        p, t = pg.at(0, 3)
        x[p, 0, t] = one if name == "k" else -one
        sc = torch.where(x.abs().amax(-1) > 0, 2.0 ** -8, 1.0) if dtype == E4 else torch.ones(x.shape[:3])
        getattr(pg, s)[:] = sc
        getattr(pg, name).copy_(ref.e4m3_codes(x, sc) if dtype == E4 else x.to(BF))
    pg.upload(wl)
    for gap in (6.0, 9.0, 11.0, 13.0):
        q = torch.full((1, 1, 1, 32), 1.0, dtype=BF)
        out = wl.wl_tree_attention(q.to(gpu), pg.cache, pg.seqs, scale=gap / 32).float().cpu()
        w = math.exp(-gap) * L
        want = (w - 1) / (w + 1)
        # weights of 8 bits (2^-8 of each side) and 2^-22 of the largest for each of the others
        assert abs(float(out[0, 0, 0, 0]) - want) <= 2 * 2.0 ** -8 + L * 2.0 ** -22, (gap, float(out[0, 0, 0, 0]), want)


def test_attention_scale_and_stream_and_workspace(wl, gpu):
    side = torch.cuda.Stream(gpu)
    _attend_case(wl, gpu, [300, 40], 5, 4, 2, 64, 16, E4, seed=21, scale=-0.3, stream=side)
    _attend_case(wl, gpu, [300, 40], 5, 4, 2, 64, 16, E4, seed=22, scale=0.0)
    pg = ref.Paged(wl, gpu, [300, 40], 5, 2, 64, 16, E4, seed=23)
    q = _randn(24, 2, 5, 4, 64).to(BF).to(gpu)
    ws = torch.full((wl.wl_tree_attention_workspace_bytes(2, 5, 4, 2, 64),), 0xFF, dtype=torch.uint8, device=gpu)
    a = wl.wl_tree_attention(q, pg.cache, pg.seqs, workspace=ws)
    b = wl.wl_tree_attention(q, pg.cache, pg.seqs, workspace=ws)
    c = wl.wl_tree_attention(q.view(10, 256), pg.cache, pg.seqs)
    assert torch.equal(a, b) and torch.equal(a.view(10, 256), c)


def test_attention_follows_lengths_in_a_graph(wl, gpu):
    """The call reads lengths, counts and pages when it runs: a captured graph serves growing contexts."""
    pg = ref.Paged(wl, gpu, [500, 300], 2, 1, 64, 16, BF, seed=30, extra_pages=2)
    q = _randn(31, 2, 2, 4, 64).to(BF)
    qd = q.to(gpu)
    ws = torch.empty(wl.wl_tree_attention_workspace_bytes(2, 2, 4, 1, 64), dtype=torch.uint8, device=gpu)
    out = torch.empty_like(qd)
    s = torch.cuda.Stream(gpu)
    s.wait_stream(torch.cuda.current_stream(gpu))
    wl.wl_tree_attention(qd, pg.cache, pg.seqs, out=out, workspace=ws, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wl.wl_tree_attention(qd, pg.cache, pg.seqs, out=out, workspace=ws, stream=s)
    for lens in ([500, 300], [3, 299], [0, 130]):
        pg.lens = lens
        pg.seqs.len.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, bound = ref.attention(pg, q, None, 64 ** -0.5)
        _within(out, want, bound + 1e-40, f"graph {lens}")


def test_many_sequences_and_a_long_context(wl, gpu):
    """More (sequence, head) pairs than SMs, very uneven lengths; then one long context."""
    g = np.random.RandomState(3)
    lens = [int(v) for v in g.randint(0, 400, 90)]
    lens[7] = 3000
    _attend_case(wl, gpu, lens, 2, 4, 2, 64, 16, E4, seed=40, counts=[int(v) for v in g.randint(0, 3, 90)])
    _attend_case(wl, gpu, [30011], 1, 2, 1, 32, 128, E4, seed=41)
    _attend_case(wl, gpu, [30011], 1, 2, 1, 32, 128, BF, seed=42)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("n,group", [(1, 2), (9, 2), (20, 2)])
def test_many_long_contexts(wl, gpu, dtype, n, group):
    """More tiles than a CTA sums in tensor memory at a time (64 tiles, 8192 positions), in units that one CTA
    has whole and in units that several share."""
    lens, kv, dim, page = [9000] * 10 + [60001] * 5, 8, 32, 64
    B, G = len(lens), group
    per = -(-(max(lens) + n) // page)
    g = torch.Generator(device=gpu)
    g.manual_seed(n)
    pages = torch.randperm(B * per, generator=g, device=gpu).to(torch.int32).view(B, per).contiguous()
    mk = lambda std: (torch.randn(B * per, kv, page, dim, generator=g, device=gpu) * std).to(dtype)  # noqa: E731
    one = torch.ones(B * per, kv, page, device=gpu)
    vs = torch.exp2(torch.randint(-3, 4, one.shape, generator=g, device=gpu).float()) if dtype == E4 else one
    cache = wl.KVCache(mk(1.0), mk(1.0), one, vs)
    seqs = wl.CacheSeqs(pages, torch.tensor(lens, dtype=torch.int32, device=gpu), n)
    q = (torch.randn(B, n, kv * G, dim, generator=g, device=gpu) * 2).to(BF)
    out = wl.wl_tree_attention(q, cache, seqs)
    assert wl.wl_device_status() == wl.WL_OK
    for b in (0, 3, 9, 10, 14):
        L = lens[b] + n
        at = pages[b].long()
        k, v = ((x[at].to(torch.float32).double() * s[at][..., None].double()).permute(1, 0, 2, 3).reshape(kv, -1, dim)[:, :L]
                for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        see = torch.arange(L, device=gpu)[None] <= lens[b] + torch.arange(n, device=gpu)[:, None]
        for h in (0, 3, kv * G - 1):
            kk, vv, qq = k[h // G], v[h // G], q[b, :, h].double()
            sc = torch.where(see, qq @ kk.T * dim ** -0.5, -math.inf)
            p = torch.softmax(sc, -1)
            want = p @ vv
            ds = float((qq.abs() @ kk.abs().T).max()) * dim ** -0.5 * 2.0 ** -20
            heavy = torch.stack([(p[i][:, None] * vv.abs()).amax(0) for i in range(n)])
            bound = (2.0 ** -8 + 4 * ds) * (p @ vv.abs()) + 2.0 ** -22 * L * heavy + 2.0 ** -8 * want.abs()
            assert bool(((out[b, :, h].double() - want).abs() <= bound).all()), (b, h)


def test_offsets_past_32_bits(wl, gpu):
    """A cache of over 2^32 bytes, used at its far end by all three operators."""
    pages, page, dim = 140000, 128, 256  # 4.6e9 bytes of codes
    cache = wl.KVCache.empty(pages, 1, page, dim, device=gpu)
    z = dict(dtype=torch.int32, device=gpu)
    seqs = wl.CacheSeqs(torch.tensor([[pages - 1, pages - 3]], **z), torch.zeros(1, **z), 200)
    x = _randn(50, 200, dim).to(BF)
    xd = x.to(gpu)
    wl.wl_rope_append(None, xd, xd, None, None, cache, seqs)
    k, v = wl.wl_cache_read(cache, seqs, dt=torch.float32)
    sc = ref.row_scale(x.float())
    want = ref.e4m3_codes(x.float(), sc).double() * sc.double()[:, None]
    assert torch.equal(k[0, :, 0].cpu().double(), want) and torch.equal(v, k)
    q = _randn(51, 1, 1, 1, dim).to(BF)
    one = wl.CacheSeqs(seqs.pages, torch.full((1,), 199, **z), 1)
    out = wl.wl_tree_attention(q.to(gpu), cache, one).cpu().double().view(-1)
    p = torch.softmax(want @ q.view(-1).double() / 16, 0)
    assert ((out - p @ want).abs() <= 2.0 ** -7 * (p @ want.abs()) + 200 * 2.0 ** -22 * want.abs().max()).all()
    assert wl.wl_device_status() == wl.WL_OK


# -------------------------------------------------------------------- norm --
DT = {"b": torch.bfloat16, "f": torch.float32}


def _norm_case(wl, gpu, T, H, kinds="bbb", gate="channel", post=True, pre=True, has_y=True, alpha=1.0, beta=0.5, eps=1e-6, off=1.0,
               seed=0, inplace=False, edit=None):
    y = (_randn(seed, T, H) * 0.7).to(DT[kinds[0]]) if has_y else None
    x = (_randn(seed + 1, T, H) * 3).to(DT[kinds[1]])
    if edit:
        edit(y, x)
    wp, wq = (_randn(seed + 2, H) * 0.1 if post else None), (_randn(seed + 3, H) * 0.1 if pre else None)
    g = None if gate == "none" else torch.rand(*((T, H) if gate == "token" else (H,)), generator=wl_synth.make_generator(seed)).to(DT[kinds[0]])
    d = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    bx, xo, pad = guarded_empty((T, H), DT[kinds[1]], gpu)
    bh, h, _ = guarded_empty((T, H), DT[kinds[2]], gpu)
    xd = x.to(gpu)
    gx, gh = wl.wl_norm_residual(d(y), xd, d(wp), d(wq), d(g), alpha, beta, eps, off, x_out=xd if inplace else xo,
                                 h_dt=DT[kinds[2]], h=h if pre else None)
    torch.cuda.synchronize()
    assert_canaries(bx, pad)
    assert_canaries(bh, pad)
    wx, wh, sx, sh = ref.norm_residual(y, x, wp, wq, g, alpha, beta, eps, off)
    _within(gx, wx, sx + (ref.bf16_slack(wx) if kinds[1] == "b" else 0) + 1e-40, f"x' T {T} H {H} {kinds}")
    if pre:
        _within(gh, wh, sh + (ref.bf16_slack(wh) if kinds[2] == "b" else 0) + 1e-40, f"h T {T} H {H} {kinds}")
    else:
        assert gh is None


@pytest.mark.parametrize("kinds", ["bbb", "bff", "bfb", "fbf", "ffb", "fff", "bbf", "fbb"])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 264), (2, 1152), (5, 5376), (2, 16384), (1, 2056), (300, 4104)])
def test_norm_residual(wl, gpu, kinds, T, H):
    _norm_case(wl, gpu, T, H, kinds, gate=("none", "channel", "token")[(T + H // 8) % 3], seed=H)


@pytest.mark.parametrize("kw", [
    dict(post=False), dict(pre=False), dict(post=False, pre=False, gate="none"), dict(has_y=False, post=False, gate="none"),
    dict(has_y=False, post=False, gate="none", alpha=0.25), dict(alpha=-2.0, beta=3.0, off=0.0), dict(eps=0.1), dict(inplace=True),
    dict(inplace=True, kinds="bfb", gate="token"), dict(beta=0.0)])
def test_norm_residual_forms(wl, gpu, kw):
    _norm_case(wl, gpu, 4, 1152, **{"seed": 5, **kw})


def test_norm_rows_of_zeros_and_extremes(wl, gpu):
    def edit(y, x):
        y[0], x[0] = 0.0, 0.0
        y[1], x[1] = 1e-20, 0.0
        x[2] *= 1e15
        y[3] *= 1e15
    _norm_case(wl, gpu, 5, 264, "fff", seed=6, edit=edit)
    _norm_case(wl, gpu, 5, 264, "fff", seed=6, edit=edit, eps=1e-5, gate="token")


def test_norm_nan_stays_in_its_row(wl, gpu):
    y, x = _randn(1, 3, 64).to(gpu), _randn(2, 3, 64).to(gpu)
    w = torch.zeros(64, device=gpu)
    y[1, 5] = math.nan
    xo, h = wl.wl_norm_residual(y, x, w, w, w_offset=1.0, h_dt=torch.float32)
    assert torch.isnan(xo[1]).all() and torch.isnan(h[1]).all()
    assert torch.isfinite(xo[[0, 2]]).all() and torch.isfinite(h[[0, 2]]).all()


def test_norm_only_the_first_norm_leaves_x(wl, gpu):
    x = _randn(2, 3, 64).to(gpu)
    xo, h = wl.wl_norm_residual(None, x, w_pre=torch.ones(64, device=gpu))
    assert xo is x and h.dtype == torch.bfloat16


def test_python_refusals_on_the_gpu(wl, gpu):
    z = dict(dtype=torch.int32, device=gpu)
    cache = wl.KVCache.empty(4, 2, 16, 64, device=gpu)
    seqs = wl.CacheSeqs(torch.zeros(1, 4, **z), torch.zeros(1, **z), 3)
    x = torch.zeros(3, 128, dtype=BF, device=gpu)
    with pytest.raises(TypeError, match="v must be"):
        wl.wl_rope_append(x, x, x.float(), None, None, cache, seqs)
    with pytest.raises(ValueError, match="rows"):
        wl.wl_rope_append(None, x[:2], x[:2], None, None, cache, seqs)
    with pytest.raises(ValueError, match="positions"):
        wl.wl_rope_append(x, x, x, torch.zeros(2, **z), None, cache, seqs)
    with pytest.raises(wl.WLError, match="q_heads"):
        wl.wl_rope_append(torch.zeros(3, 192, dtype=BF, device=gpu), x, x, None, None, cache, seqs)
    with pytest.raises(wl.WLError, match="rot"):
        wl.wl_rope_append(x, x, x, None, wl.RopeTable.make(96, device=gpu), cache, seqs)
    with pytest.raises(ValueError, match="mask"):
        wl.wl_tree_attention(x, cache, seqs, mask=torch.zeros(2, dtype=torch.int64, device=gpu))
    with pytest.raises(wl.WLError, match="too small"):
        wl.wl_tree_attention(x, cache, seqs, workspace=torch.empty(256, dtype=torch.uint8, device=gpu)[:16])
    with pytest.raises(wl.WLError, match="n must"):
        wl.wl_tree_attention(torch.zeros(65, 128, dtype=BF, device=gpu), cache, wl.CacheSeqs(seqs.pages, seqs.len, 65))
    with pytest.raises(TypeError, match="q must"):
        wl.wl_tree_attention(x.float(), cache, seqs)
    with pytest.raises(ValueError, match="k_out"):
        wl.wl_cache_read(cache, seqs, outs=(x, x))
    with pytest.raises(ValueError, match="gate"):
        wl.wl_norm_residual(x, x, gate=torch.zeros(64, dtype=BF, device=gpu))
    with pytest.raises(TypeError, match="w_pre"):
        wl.wl_norm_residual(x, x, w_pre=x[0])
    with pytest.raises(wl.WLError, match="multiple of 8"):
        wl.wl_norm_residual(None, torch.zeros(2, 12, device=gpu), alpha=2.0)
    with pytest.raises(TypeError, match="float8"):
        wl.KVCache.empty(4, 2, 16, 64, dtype=torch.float16, device=gpu)
