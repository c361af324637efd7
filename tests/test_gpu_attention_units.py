"""Tree attention where a thread block works on several units (sequence, kv
head, row tile) one after the other, against the formula in 64 bits on the GPU.
The bound is that of tests/layer_ref.py, by the number formats."""
import math

import pytest
import torch

import wl_synth
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
E4, BF = torch.float8_e4m3fn, torch.bfloat16


def filled(wl, gpu, lens, n, kv, dim, page, dtype, seed=0, spare=1):
    """A cache with rows of several sizes at random pages, NaN in every row that no sequence has."""
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    B = len(lens)
    per = -(-(max(lens) + n) // page)
    pool = B * per + spare
    pages = torch.randperm(pool, generator=g, device=gpu)[:B * per].to(torch.int32).view(B, per).contiguous()
    shape = (pool, kv, page, dim)
    size = torch.exp2(torch.randint(-3, 4, shape[:3], generator=g, device=gpu).float())
    k, v = torch.randn(shape, generator=g, device=gpu), torch.randn(shape, generator=g, device=gpu) * size[..., None]
    one = torch.ones(shape[:3], device=gpu)
    if dtype == E4:
        ks, vs = (torch.exp2(torch.ceil(torch.log2(t.abs().amax(-1) / 448))) for t in (k, v))
        cache = wl.KVCache((k / ks[..., None]).to(E4), (v / vs[..., None]).to(E4), ks, vs)
    else:
        cache = wl.KVCache(k.to(BF), v.to(BF), one, one.clone())
    total = torch.tensor(lens, device=gpu) + n
    used = torch.zeros(pool, page, dtype=torch.bool, device=gpu)
    at = torch.arange(per * page, device=gpu)[None].expand(B, -1).reshape(B, per, page)
    used[pages.long()] = at < total[:, None, None]
    dead = ~used[:, None].expand(-1, kv, -1)
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x.view(torch.uint8 if dtype == E4 else torch.int16)[dead] = 0x7F if dtype == E4 else 0x7FC0
        s[dead] = math.nan
    return cache, wl.CacheSeqs(pages, torch.tensor(lens, dtype=torch.int32, device=gpu), n)


def formula(cache, seqs, q, b, see, scale):
    """(out, bound) [n, q_heads, dim] in 64 bits of sequence b; see [n, positions]."""
    n, L = see.shape
    page, G = cache.page_size, q.shape[2] // cache.kv_heads
    # (a page outside the cache: any row stands in, see excludes it)
    at = seqs.pages[b, :-(-L // page)].long().clamp(0, cache.pages - 1)

    def rows(x, s):
        t = x[at].to(torch.float32).double() * s[at][..., None].double()
        return t.permute(1, 0, 2, 3).reshape(cache.kv_heads, -1, cache.dim)[:, :L]

    k, v = (torch.where(see.any(0)[None, :, None], t, 0.0) for t in (rows(cache.k, cache.k_scale), rows(cache.v, cache.v_scale)))
    k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    qq = q[b].double().transpose(0, 1)
    p = torch.softmax(torch.where(see, qq @ k.transpose(1, 2) * scale, -math.inf), -1)
    p = torch.where(see.any(-1)[:, None], p, 0.0)
    out = p @ v
    mag = torch.where(see, qq.abs() @ k.abs().transpose(1, 2) * abs(scale), 0.0).amax(-1, keepdim=True)
    spread = p @ v.abs()
    heavy = torch.stack([(p[:, i, :, None] * v.abs()).amax(1) for i in range(n)], 1)
    bound = (2.0 ** -8 + 4 * mag * 2.0 ** -20) * spread + 2.0 ** -22 * see.sum(-1)[:, None] * heavy + 2.0 ** -8 * out.abs() + 2.0 ** -133
    return out.transpose(0, 1), bound.transpose(0, 1)


def chain(lens, b, n, dev):
    j = torch.arange(lens[b] + n, device=dev)
    return j[None] <= lens[b] + torch.arange(n, device=dev)[:, None]


def check(wl, cache, seqs, lens, q, see=None, which=None, what=""):
    """The call against the formula, and against itself."""
    out = wl.wl_tree_attention(q, cache, seqs)
    again = wl.wl_tree_attention(q, cache, seqs)
    for b in which if which is not None else range(len(lens)):
        want, bound = formula(cache, seqs, q, b, chain(lens, b, seqs.n, q.device) if see is None else see(b), cache.dim ** -0.5)
        d = (out[b].double() - want).abs()
        worst = float((d / bound).max())
        assert worst <= 1, f"{what} sequence {b}: {worst:.3g} times the bound"
    assert torch.equal(out, again), what


def _q(gpu, B, n, heads, dim, seed):
    return (torch.randn(B, n, heads, dim, generator=wl_synth.make_generator(seed)) * 2).to(BF).to(gpu)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("n", [4, 8, 16, 33])  # 16, 32, 64 and 3 x 64 rows of a kv head
@pytest.mark.parametrize("page", [16, 64, 4])
def test_blocks_with_many_units(wl, gpu, dtype, dim, n, page):
    """Far more units than SMs, of 1 to 5 tiles, so that ranges begin at any tile of a unit."""
    B, kv, G = 80, 4, 4
    lens = [(37 * b * b + 11 * b) % (5 * 128 - n) for b in range(B)]
    lens[0], lens[1] = 0, 5 * 128 - n
    cache, seqs = filled(wl, gpu, lens, n, kv, dim, page, dtype, seed=n)
    check(wl, cache, seqs, lens, _q(gpu, B, n, kv * G, dim, n), what=f"{dtype} dim {dim} n {n} page {page}")
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("dtype,dim,n", [(BF, 256, 16), (BF, 256, 8), (BF, 200 // 16 * 16, 16), (E4, 256, 16)])
def test_blocks_with_units_of_one_length(wl, gpu, dtype, dim, n):
    """Units of 1, 2, 3 tiles only, and of one long one between short ones."""
    for lens in ([100] * 200, [200] * 120, [380 - n] * 90, [100] * 60 + [5000] + [100] * 60):
        cache, seqs = filled(wl, gpu, lens, n, 2, dim, 32, dtype, seed=len(lens))
        B = len(lens)
        check(wl, cache, seqs, lens, _q(gpu, B, n, 8, dim, 3), which=range(0, B, 7 if B < 121 else 11), what=f"{lens[0]} x {B}")
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("dtype,dim", [(BF, 256), (BF, 128), (E4, 256), (E4, 64)])
@pytest.mark.parametrize("n", [4, 8, 16])
@pytest.mark.parametrize("page", [16, 128, 4])
def test_pages_that_are_not_there_in_long_contexts(wl, gpu, dtype, dim, n, page):
    """Positions of an invalid page, in any tile, are seen by no query, reach nothing else, and are reported."""
    B, kv, G = 60, 4, 4
    lens = [700 + 13 * b for b in range(B)]
    cache, seqs = filled(wl, gpu, lens, n, kv, dim, page, dtype, seed=5)
    gone = [(3 * b + 1) % (600 // page) for b in range(B)]
    for b in range(B):
        seqs.pages[b, gone[b]] = (-1, cache.pages, 1 << 30, -2, -(1 << 31))[b % 5]

    def see(b):
        m = chain(lens, b, n, gpu)
        m[:, gone[b] * page:(gone[b] + 1) * page] = False
        return m

    check(wl, cache, seqs, lens, _q(gpu, B, n, kv * G, dim, 4), see, what=f"{dtype} dim {dim} n {n} page {page}")
    assert wl.wl_device_status() == wl.WL_ERR_INVALID_ARG
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("entry", [-2, -(1 << 31)])
def test_any_negative_page_is_reported(wl, gpu, entry):
    for dtype in (E4, BF):
        cache, seqs = filled(wl, gpu, [700, 30], 4, 2, 128, 16, dtype)
        seqs.pages[0, 3] = entry
        wl.wl_tree_attention(_q(gpu, 2, 4, 4, 128, 1), cache, seqs)
        assert wl.wl_device_status() == wl.WL_ERR_INVALID_ARG
        assert wl.wl_device_status() == wl.WL_OK
