"""Inputs of very different sizes side by side, in the decoder-layer operators:
what is said of one row must not come from another."""
import pytest
import torch

import wl_synth
from tests.test_gpu_attention_units import chain, check, filled, formula

pytestmark = pytest.mark.gpu
E4, BF = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("dim", [48, 128, 256])
@pytest.mark.parametrize("n,group", [(1, 3), (1, 16), (5, 4), (16, 4), (40, 2)])
def test_query_rows_of_very_different_sizes(wl, gpu, dtype, dim, n, group):
    """Each row of q keeps its bits beside rows up to 2^100 times larger or smaller (tests/layer_ref.py's bound,
    which knows no other row)."""
    lens, kv = [400, 37, 1500], 2
    cache, seqs = filled(wl, gpu, lens, n, kv, dim, 16, dtype, seed=dim + n)
    g = wl_synth.make_generator(n)
    for sizes in ((0, 10, 14, 17, 20, 24), (-30, 0, 1, 4), (0, 100), (-90, -60, -61)):
        e = torch.tensor(sizes)[torch.randint(0, len(sizes), (3, n, kv * group, 1), generator=g)]
        q = (2 * torch.randn(3, n, kv * group, dim, generator=g) * torch.exp2(e.float())).to(BF)
        q[1, 0, -1] = 0.0
        check(wl, cache, seqs, lens, q.to(gpu), what=f"{dtype} dim {dim} n {n} sizes {sizes}")
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("n,group", [(1, 4), (5, 4), (16, 4)])
def test_query_rows_of_zeros_beside_large_ones(wl, gpu, n, group):
    """Rows of zeros, and rows beyond a sequence's count, beside rows that differ and are all large or all small."""
    lens, kv, dim = [200, 37, 300], 2, 128
    cache, seqs = filled(wl, gpu, lens, n, kv, dim, 16, E4, seed=n)
    g = wl_synth.make_generator(n)
    for sizes in ((16, 24), (40, 60, 70), (110, 120), (-60, -40), (-100, -120, -110)) + tuple((s, s + 6) for s in range(4, 20)):
        e = torch.tensor(sizes)[torch.randint(0, len(sizes), (3, n, kv * group, 1), generator=g)]
        e[:, :, ::group] = sizes[0]
        if sizes[0] in range(4, 20):  # of one exponent
            q = torch.randint(0, 2, (3, n, kv * group, dim), generator=g) * 2.0 - 1.0
        else:
            q = torch.randn(3, n, kv * group, dim, generator=g)
        q = (q * torch.exp2(e.float())).to(BF)
        q[:, :, 1::group] = q[:, :, ::group]
        full = wl.wl_tree_attention(q.to(gpu), cache, seqs)
        q[:, :, 1::group] = 0.0
        q = q.to(gpu)
        out = wl.wl_tree_attention(q, cache, seqs)
        # a power of two more or less changes no row's bits, so neither does what its neighbours are
        keep = torch.ones(kv * group, dtype=torch.bool)
        keep[1::group] = False
        assert torch.isfinite(full.float()).all() and torch.equal(out[:, :, keep], full[:, :, keep]), sizes
        # a row of zeros: the mean of v
        for b in range(3):
            want, bound = formula(cache, seqs, q, b, chain(lens, b, n, gpu), dim ** -0.5)
            assert bool(((out[b].double() - want).abs() <= bound)[:, ~keep].all()), sizes
        some = wl.CacheSeqs(seqs.pages, seqs.len, n, torch.tensor([n, 0, n // 2], dtype=torch.int32, device=gpu))
        part = wl.wl_tree_attention(q, cache, some)
        assert torch.equal(part[0], out[0]) and bool((part[1] == 0).all()) and bool((part[2, n // 2:] == 0).all())
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("dtype", [E4, BF])
def test_values_that_round_to_an_infinity(wl, gpu, dtype):
    """A finite value beyond the cache's type marks its row as one with an infinity: only queries that see it know."""
    edge = 3.3961776e38  # halfway from the largest bf16 number to the next power of two: rounds up
    cache = wl.KVCache.empty(4, 1, 16, 64, dtype, gpu)
    z = dict(dtype=torch.int32, device=gpu)
    seqs = wl.CacheSeqs(torch.arange(4, **z)[None], torch.zeros(1, **z), 40)
    k, v = (torch.randn(40, 64, generator=wl_synth.make_generator(i)) for i in (1, 2))
    v[38, 5], k[39, 7] = edge, -edge
    v[37, 9] = 3.3895e38  # below the middle: the largest bf16 number
    wl.wl_rope_append(None, k.to(gpu), v.to(gpu), None, None, cache, seqs)
    kk, vv = wl.wl_cache_read(cache, seqs, dt=torch.float32)
    scales = torch.stack((cache.k_scale, cache.v_scale)).view(2, -1).cpu()
    if dtype == BF:
        assert not torch.isinf(kk).any() and not torch.isinf(vv).any()
        assert torch.isnan(scales).nonzero().tolist() == [[0, 39], [1, 38]]
        assert torch.isnan(kk[0, 39]).all() and torch.isnan(vv[0, 38]).all() and float(vv[0, 37, 0, 9]) == float(torch.finfo(BF).max)
    else:  # codes hold such values; reading them back may pass the type's range
        assert torch.isfinite(scales[:, :40]).all()
    # tokens that see neither row: a result as without them
    seqs = wl.CacheSeqs(seqs.pages, torch.full((1,), 30, **z), 10)
    q = torch.randn(1, 10, 2, 64, generator=wl_synth.make_generator(3)).to(BF).to(gpu)
    mask = torch.tensor([[1 << i for i in range(10)]], dtype=torch.int64, device=gpu)
    out = wl.wl_tree_attention(q, cache, seqs, mask=mask)
    cache.v_scale[2, 0, 5:8], cache.k_scale[2, 0, 5:8] = 1.0, 1.0
    for x in (cache.k, cache.v):
        x.view(torch.uint8)[2, 0, 5:8] = 0
    see = torch.arange(40, device=gpu)[None] < 30
    see = see | (torch.arange(40, device=gpu)[None] == 30 + torch.arange(10, device=gpu)[:, None])
    want, bound = formula(cache, seqs, q, 0, see, 64 ** -0.5)
    assert bool(((out[0, :7].double() - want[:7]).abs() <= bound[:7]).all())
    if dtype == BF:
        assert torch.isnan(out[0, 8:]).all()


def test_rows_of_zeros_in_v_weigh_nothing(wl, gpu):
    """A row of zeros has scale 1, far above a small row's: heavy scores on it must not take the others' bits."""
    for dim, n, group in ((64, 1, 2), (128, 6, 4), (256, 1, 4), (256, 20, 4)):
        lens = [900, 3000]
        cache, seqs = filled(wl, gpu, lens, n, 1, dim, 16, E4, seed=dim)
        rows = cache.v_scale
        rows.mul_(2.0 ** -12)  # values of about 2^-12
        q = torch.ones(2, n, group, dim, dtype=BF, device=gpu)
        for b in range(2):
            for j in (0, 5, 133, 260, 513):
                p, t = int(seqs.pages[b, j // 16]), j % 16
                cache.v.view(torch.uint8)[p, 0, t] = 0x80 if j == 5 else 0
                rows[p, 0, t] = 1.0
                cache.k.view(torch.uint8)[p, 0, t] = 0x38  # ones
                cache.k_scale[p, 0, t] = 1.0
        # a score of 16 on the rows of zeros, small ones elsewhere (k has both signs)
        scale = 16.0 / dim
        out = wl.wl_tree_attention(q, cache, seqs, scale=scale)
        for b in range(2):
            want, bound = formula(cache, seqs, q, b, chain(lens, b, n, gpu), scale)
            worst = float(((out[b].double() - want).abs() / bound).max())
            assert worst <= 1, f"dim {dim} n {n} sequence {b}: {worst:.3g} times the bound"
            assert float((want.abs() / bound).median()) > 2  # the bound tells the result from none
    assert wl.wl_device_status() == wl.WL_OK


def test_all_of_v_zero_and_large_rows_of_scale_one(wl, gpu):
    lens, n, dim = [300, 40], 3, 128
    cache, seqs = filled(wl, gpu, lens, n, 2, dim, 16, E4, seed=1)
    q = torch.randn(2, n, 4, dim, generator=wl_synth.make_generator(1)).to(BF).to(gpu)
    live = ~torch.isnan(cache.v_scale)
    cache.v_scale[live] = 1.0  # codes up to 448, as they are
    check(wl, cache, seqs, lens, q, what="scale 1")
    cache.v.view(torch.uint8)[live] = 0
    out = wl.wl_tree_attention(q, cache, seqs)
    assert bool((out == 0).all())
    half = live.clone()
    half[:, :, 8:] = False
    cache.v.view(torch.uint8)[half] = 0x01  # the smallest code alone
    check(wl, cache, seqs, lens, q, what="smallest codes")


@pytest.mark.parametrize("dim,n,group", [(128, 1, 2), (256, 1, 4), (128, 8, 8)])
def test_runs_of_tiny_rows_in_v(wl, gpu, dim, n, group):
    """Rows of v near fp32's smallest numbers, by the tile, beside ordinary ones: the softmax's sum stays finite.

    A row counts as if its scale were 2^-104 at least, so what lies below 448 * 2^-104 may come out as large as that."""
    lens = [2500, 700]
    cache, seqs = filled(wl, gpu, lens, n, 1, dim, 16, E4, seed=dim + n)
    q = torch.randn(2, n, group, dim, generator=wl_synth.make_generator(n)).to(BF).to(gpu)
    plain = cache.v_scale.clone()
    for first, last in ((0, 512), (128, 256), (0, 2000)):
        cache.v_scale.copy_(plain)
        for b in range(2):
            at = seqs.pages[b, first // 16:min(last, lens[b]) // 16].long()
            cache.v_scale[at] = 2.0 ** -126
        out = wl.wl_tree_attention(q, cache, seqs)
        for b in range(2):
            want, bound = formula(cache, seqs, q, b, chain(lens, b, n, gpu), dim ** -0.5)
            worst = float(((out[b].double() - want).abs() / (bound + 448 * 2.0 ** -104)).max())
            assert worst <= 1, f"positions {first} to {last}, sequence {b}: {worst:.3g} times the bound"
    assert wl.wl_device_status() == wl.WL_OK


def test_empty_calls_are_refused_by_name(wl, gpu):
    """No tokens or no sequences: the library's own words, not a division by zero."""
    z = dict(dtype=torch.int32, device=gpu)
    cache = wl.KVCache.empty(4, 2, 16, 64, device=gpu)
    x = torch.zeros(0, 128, dtype=BF, device=gpu)
    for B, n, what in ((1, 0, "n must"), (0, 2, "batch must")):
        s = wl.CacheSeqs(torch.zeros(B, 4, **z), torch.zeros(B, **z), n)
        for call in (lambda: wl.wl_rope_append(x, x, x, None, None, cache, s), lambda: wl.wl_rope_append(None, x, x, None, None, cache, s),
                     lambda: wl.wl_tree_attention(x, cache, s), lambda: wl.wl_cache_read(cache, s)):
            with pytest.raises(wl.WLError, match=what):
                call()
