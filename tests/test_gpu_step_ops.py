"""GPU tests of the operators between a step's last states and the next step
against their 64-bit forms."""
import math

import numpy as np
import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def ok(wl):
    assert wl.wl_device_status() == wl.WL_OK


# -------------------------------------------------------------- quantiser --
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group", [1, 128])
@pytest.mark.parametrize("rows,inner", [(1, 16), (1, 1152), (3, 144), (7, 128), (129, 400), (1300, 272), (5, 5376)])
def test_quant(wl, gpu, rows, inner, group, dt):
    x = torch.randn(rows, inner, generator=gen(rows + inner)) * torch.exp(3 * torch.randn(rows, 1, generator=gen(1)))
    x[0, :16] = 0.875 * 2.0 ** 9  # 448 itself
    x = x.to(dt)
    codes, scales = wl.wl_quant_f8(x.to(gpu), group=group)
    want, ws = ref.quant(x, group)
    assert np.array_equal(scales.double().cpu().numpy(), ws)
    assert np.array_equal(codes.float().double().cpu().numpy(), want)
    ok(wl)


def test_quant_extremes(wl, gpu):
    """Blocks of zeros, of the smallest and the largest numbers, with a NaN, with an infinity; strided rows."""
    x = torch.randn(9, 384, generator=gen(3))
    x[0, :128] = 0.0
    x[1, 128:256] = 1e-45
    x[2, :128] *= 1e-40
    x[3] = torch.finfo(F32).max
    x[4, 200] = math.nan
    x[5, 300] = -math.inf
    x[6, :128] = 2.0 ** -126 * 448
    x[7, :128] = torch.nextafter(torch.tensor(448.0), torch.tensor(500.0))
    wide = torch.zeros(9, 400)
    wide[:, :384] = x
    for group in (1, 128):
        codes, scales = wl.wl_quant_f8(wide.to(gpu)[:, :384], group=group)
        want, ws = ref.quant(x, group)
        assert np.array_equal(scales.double().cpu().numpy(), ws, equal_nan=True)
        assert np.array_equal(codes.float().double().cpu().numpy(), want)


# ---------------------------------------------------------------- product --
def _factors(T, inner, out, seed):
    g = gen(seed)
    kb = -(-inner // 128)
    x = (torch.randn(T, inner, generator=g) * 60).clamp(-448, 448).to(F8)
    w = (torch.randn(out, inner, generator=g) * 60).clamp(-448, 448).to(F8)
    xs = torch.exp(torch.randn(kb, T, generator=g))
    ws = torch.exp(torch.randn(kb, -(-out // 128), generator=g)) * 1e-3
    return x, xs, w, ws


# fp32 sums: a block's by the tensor cores (128 products of 8 significant bits, truncated to at least 24 bits an
# addition: 128 * 2^-23 of the sum of magnitudes), then one rounding of the two scales' product and two a block; the
# result's own rounding half a step.
def _check_product(y, x, xs, w, ws, dt):
    want = ref.product(x, xs, w, ws)
    mag = ref.product(x.float().abs(), xs.abs(), w.float().abs(), ws.abs())
    kb = xs.shape[0]
    tol = (128 * 2.0 ** -23 + (kb + 2) * 2.0 ** -23) * mag + torch.finfo(dt).eps / 2 * np.abs(want) * (1 + 1e-3)
    d = np.abs(y.double().cpu().numpy() - want)
    assert (d <= tol).all(), (float((d / tol).max()), np.unravel_index((d / tol).argmax(), d.shape))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,inner,out", [
    (1, 16, 1), (1, 128, 128), (1, 1152, 300), (2, 144, 129), (3, 2304, 64), (5, 256, 1153), (8, 640, 127), (15, 384, 257), (16, 1152, 256), (17, 272, 100),
    (31, 512, 513), (33, 1296, 131), (37, 6912, 65), (64, 128, 384), (65, 1152, 255), (96, 1152, 640), (127, 144, 385), (129, 400, 200),
    (200, 1152, 1000), (100, 272, 20001), (70, 1152, 19464), (300, 400, 9731), (1000, 144, 2500), (140, 2048, 19460), (1, 400, 9740), (3, 144, 21504), (8, 1296, 5376), (9, 128, 21501), (33, 272, 19336), (128, 144, 39000), (64, 1152, 30008), (1, 144, 262144), (257, 16, 9736), (256, 256, 256), (257, 640, 130), (300, 2048, 512), (513, 384, 700), (1, 21504, 40), (1025, 144, 72),
])
def test_product(wl, gpu, T, inner, out, dt):
    x, xs, w, ws = _factors(T, inner, out, T + inner + out)
    weight = wl.F8Weight(w.to(gpu), ws.to(gpu))
    y = torch.full((T, out), math.nan, dtype=dt, device=gpu)
    wl.wl_linear_f8(x.to(gpu), xs.to(gpu), weight, y=y, ydt=dt)
    _check_product(y, x, xs, w, ws, dt)
    again = wl.wl_linear_f8(x.to(gpu), xs.to(gpu), weight, ydt=dt)
    assert torch.equal(y, again)
    ok(wl)


def test_product_nan_scales_reach_their_rows_alone(wl, gpu):
    x, xs, w, ws = _factors(70, 400, 300, 5)
    xs[2, 7], ws[1, 2] = math.nan, math.inf
    y = wl.wl_linear_f8(x.to(gpu), xs.to(gpu), wl.F8Weight(w.to(gpu), ws.to(gpu)), ydt=F32).cpu()
    clean = torch.ones(70, 300, dtype=torch.bool)
    clean[7], clean[:, 256:] = False, False
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[:, 256:]).any()
    assert torch.isfinite(y[clean]).all()


def test_quantised_projection_is_near_the_projection(wl, gpu):
    """Both factors off by at most half an e4m3 step (2^-4 of the value, or 2^-10 of the scale for the smallest)."""
    g = gen(11)
    x, W = torch.randn(40, 1152, generator=g), torch.randn(500, 1152, generator=g) * 0.05
    y = wl.wl_linear_f8(*wl.wl_quant_f8(x.to(gpu)), wl.F8Weight.quantise(W.to(gpu)), ydt=F32).double().cpu()
    want, mag = x.double() @ W.double().T, x.double().abs() @ W.double().abs().T
    # random signs: far inside the bound of (2 * 2^-4 + 2^-8) mag; the smallest codes add 2^-10 * scale <= 2^-17 of a block's largest
    assert ((y - want).abs() <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -9) * mag).all()
    assert float((y - want).norm() / want.norm()) < 2 * 2.0 ** -4


# ----------------------------------------------------------- verification --
def _tree(B, n, seed):
    rs = np.random.RandomState(seed)
    m = np.zeros((B, n), np.uint64)
    for b in range(B):
        for i in range(n):
            m[b, i] = np.uint64(1 << i) | (m[b, i - 1 - rs.randint(0, min(i, 5))] if i else np.uint64(0))
    return torch.from_numpy(m.view(np.int64))


def _drafts(B, n, V, seed, ldt=F32, ddt=None, sigma=2.0, mask=None):
    """Logits, tokens likely enough to be accepted, draws, and (ddt) a draft distribution near the model's."""
    g = gen(seed)
    logits = (torch.randn(B * n, V, generator=g) * sigma).to(ldt)
    p = torch.softmax(logits.float(), -1)
    draft = None if ddt is None else torch.softmax(logits.float() + 0.5 * torch.randn(B * n, V, generator=g), -1).to(ddt)
    par = torch.tensor([ref.parents(None if mask is None else mask[b].numpy().view(np.uint64), n) for b in range(B)]).clamp(min=0)
    rows = (torch.arange(B)[:, None] * n + par).view(-1)
    src = p if draft is None else draft.float()
    tokens = torch.multinomial(src[rows], 1, generator=g).view(B, n).to(torch.int32)
    return logits, tokens, torch.rand(B, n, generator=g), draft


def _check_verify(wl, gpu, logits, tokens, uniforms, **kw):
    to = lambda t: t.to(gpu) if isinstance(t, torch.Tensor) else t  # noqa: E731
    got = wl.wl_verify(to(logits), to(tokens), to(uniforms), **{k: to(v) for k, v in kw.items()})
    want = ref.verify(logits, tokens, uniforms, **kw)
    for name, a, b in zip(("path", "accepted", "next"), got, want):
        a = a.cpu().numpy()
        assert np.array_equal(a, b), (name, np.nonzero(a != b), a[a != b][:5], b[a != b][:5])
    ok(wl)
    return want


@pytest.mark.parametrize("ddt", [None, F32, BF])
@pytest.mark.parametrize("ldt", [F32, BF])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (1, 1, 7), (3, 4, 2), (2, 8, 33), (5, 3, 1000), (1, 64, 129), (20, 5, 4099), (40, 2, 511), (160, 3, 300),
                                   (2, 6, 70001), (9, 33, 8195)])
def test_verify_chains(wl, gpu, B, n, V, ldt, ddt):
    a, t, u, d = _drafts(B, n, V, B + n + V, ldt, ddt)
    path, acc, _ = _check_verify(wl, gpu, a, t, u, draft=d, temperature=0.8)
    if B >= 20 and V > 100 and ddt is not None:  # a certain token of a flat row is accepted as rarely as it is drawn
        assert (acc > 1).any() and (acc < n).any()


@pytest.mark.parametrize("ldt", [F32, BF])
@pytest.mark.parametrize("B,n,V", [(30, 6, 4001), (3, 12, 60000)])
def test_verify_likely_tokens(wl, gpu, B, n, V, ldt):
    """Peaked rows, certain tokens: most are accepted."""
    a, t, u, _ = _drafts(B, n, V, 3 * V, ldt, None, sigma=6.0)
    _, acc, _ = _check_verify(wl, gpu, a, t, u)
    assert (acc > 1).any() and (acc < n).any()


@pytest.mark.parametrize("ddt", [None, F32])
@pytest.mark.parametrize("temp", [0.0, 0.3, 1.0, 2.5])
@pytest.mark.parametrize("B,n,V", [(1, 7, 50), (6, 24, 1003), (3, 64, 400), (30, 12, 64), (2, 20, 33000)])
def test_verify_trees(wl, gpu, B, n, V, temp, ddt):
    m = _tree(B, n, B * n)
    a, t, u, d = _drafts(B, n, V, n + V, F32, ddt, mask=m)
    _check_verify(wl, gpu, a, t, u, mask=m, draft=d, temperature=temp)


def test_verify_counts_temperatures_and_strides(wl, gpu):
    B, n, V = 24, 9, 777
    m = _tree(B, n, 3)
    a, t, u, d = _drafts(B, n, V, 4, BF, BF, mask=m)
    count = torch.arange(B, dtype=torch.int32) % (n + 3) - 1
    temp = torch.linspace(0.0, 2.0, B)
    temp[5], temp[6], temp[7] = 1e-7, math.nan, math.inf
    temp[8] = -1.0
    _check_verify(wl, gpu, a, t, u, mask=m, draft=d, count=count, temperature=temp)
    wide, dw = torch.zeros(B * n, V + 12, dtype=BF), torch.zeros(B * n, V + 5, dtype=BF)
    wide[:, 3:3 + V], dw[:, 1:1 + V] = a, d
    got = wl.wl_verify(wide.to(gpu)[:, 3:3 + V], t.to(gpu), u.to(gpu), mask=m.to(gpu), draft=dw.to(gpu)[:, 1:1 + V], count=count.to(gpu),
                       temperature=temp.to(gpu))
    for x, y in zip(got, ref.verify(a, t, u, m, count, d, temp)):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("ddt", [None, F32])
@pytest.mark.parametrize("temp", [0.0, 1.0])
def test_verify_masked_and_broken_rows(wl, gpu, temp, ddt):
    """Masked tokens, a row with one token left, rows with nothing, a NaN, an infinity; tokens outside the vocabulary."""
    B, n, V = 12, 4, 2050
    a, t, u, d = _drafts(B, n, V, 9, F32, ddt, sigma=1.0)
    a.view(B, n, V)[:, :, 5:1900] = -math.inf
    a.view(B, n, V)[:, :, 1950] = torch.finfo(F32).min
    a[1 * n], a[2 * n] = -math.inf, -math.inf
    a[2 * n, 77] = -3.0
    t[2, 1] = 77
    a[3 * n, 1999], a[4 * n, 3] = math.nan, math.inf
    a[5 * n:6 * n] = torch.finfo(F32).min
    a[6 * n + 1], t[6, 1], u[6, 1] = math.nan, int(a[6 * n].argmax()), 0.0
    t[7], t[8] = -1, V
    t[9, 1:] = 100  # masked
    t[10], t[11] = 2 ** 31 - 1, -2 ** 31
    if d is not None:
        d[6 * n] = 0.5
    _check_verify(wl, gpu, a, t, u, temperature=temp, draft=d)


def test_verify_all_tokens_rejected_and_repeated_tokens(wl, gpu):
    """Siblings that use up the row's tokens, and siblings with the same token: the second finds no weight left."""
    n, V = 6, 3
    m = torch.tensor([[1, 3, 5, 9, 17, 33]] * 4)
    a = torch.tensor([[0.0, 0.0, -math.inf]]).repeat(4 * n, 1)
    t = torch.tensor([[0, 0, 0, 1, 1, 2], [0, 1, 1, 1, 1, 1], [0, 2, 2, 0, 0, 1], [0, 0, 1, 0, 1, 2]], dtype=torch.int32)
    u = torch.full((4, n), 1 - 2.0 ** -24)
    u[1, 1:], u[1, 0], u[2, 0] = 0.5, 0.3, 0.0  # 0.5 * 2 < 1 is false
    _check_verify(wl, gpu, a, t, u, mask=m)


@pytest.mark.parametrize("V", [8, 4096, 65536])
def test_verify_draws_on_borders(wl, gpu, V):
    """Equal logits: every multiple of 1/V is a border, and the token after it is the one drawn."""
    B = 16
    j = torch.arange(B) * (V // B) if V >= B else torch.arange(B) % V
    a = torch.full((B, V), 1.5)
    _, _, nxt = _check_verify(wl, gpu, a, torch.zeros(B, 1, dtype=torch.int32), (j.float() / V)[:, None])
    assert np.array_equal(nxt, j.numpy())
    # a child on the border is rejected, just below it accepted
    t = torch.full((B, 2), V - 1, dtype=torch.int32)
    u = torch.full((B, 2), 1.0 / V)
    u[::2, 1] = float(np.nextafter(np.float32(1.0 / V), np.float32(0)))
    _, acc, _ = _check_verify(wl, gpu, a.repeat_interleave(2, 0), t, u)
    assert acc.tolist() == [2, 1] * (B // 2)


def test_verify_takes_the_temperature_as_given(wl, gpu):
    """0.3 in 64 bits: rounded to fp32 it would move the border of the first token past the draw."""
    V, t = 3270000, 0.3
    low = -15.0 * t
    a = torch.full((1, V), low)
    a[0, 0] = 0.0
    low = float(a[0, 1])

    def first(temp):  # the share of token 0
        return 1.0 / (1.0 + (V - 1) * math.exp(low / temp))

    lo, hi = sorted((first(t), first(float(np.float32(t)))))
    u = float(np.float32((lo + hi) / 2))
    assert lo < u < hi
    _, _, nxt = _check_verify(wl, gpu, a, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([[u]]), temperature=t)
    assert (nxt[0] == 0) == (u < first(t))


def test_verify_draws_outside_the_range(wl, gpu):
    a, t, u, _ = _drafts(6, 2, 300, 2)
    a[:, 290:] = -math.inf
    u[:, 0] = torch.tensor([0.0, 1.0, 2.0, 1 - 2.0 ** -24, -1.0, 0.5])
    u[:, 1] = torch.tensor([0.0, 1.0, 2.0, 1.0, -1.0, 0.5])
    _check_verify(wl, gpu, a, t, u)


def test_verified_tokens_are_spread_like_the_model(wl, gpu):
    """One draft from q, then the next token: over all drafts and a grid of draws, the first new token is the model's."""
    V, G = 5, 64
    p = torch.tensor([0.4, 0.05, 0.3, 0.05, 0.2])
    q = torch.tensor([0.1, 0.3, 0.2, 0.25, 0.15])
    grid = (torch.arange(G) + 0.5) / G
    tok = torch.arange(V).repeat_interleave(G * G)
    r, r0 = grid.repeat_interleave(G).repeat(V), grid.repeat(V * G)
    B = V * G * G
    t = torch.stack((torch.zeros_like(tok), tok), 1).to(torch.int32)
    _, acc, nxt = wl.wl_verify(p.log().expand(2 * B, V).contiguous().to(gpu), t.to(gpu), torch.stack((r0, r), 1).contiguous().to(gpu),
                               draft=q.expand(2 * B, V).contiguous().to(gpu))
    first = torch.where(acc.cpu() == 2, tok, nxt.cpu().long())
    got = torch.zeros(V, dtype=torch.float64).index_add_(0, first, (q[tok] / (G * G)).double())
    # a grid of G points puts a border off by at most half a step, for the test and for each of two borders of a token
    assert ((got - p.double()).abs() < 3.0 / G).all(), got


# -------------------------------------------------------------- page plan --
class _State:
    def __init__(self, pool, page, B, P, seed):
        rs = np.random.RandomState(seed)
        ids = rs.permutation(pool).astype(np.int32)
        self.page, self.B, self.P, self.pool = page, B, P, pool
        self.free, self.top = ids.copy(), pool
        self.pages, self.held = np.full((B, P), -1, np.int32), np.zeros(B, np.int32)


def _plan_both(wl, s, dev, pool, pages, held, length, count, n):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    room, slots = wl.wl_page_plan(pool, pages, held, i32(length), n, None if count is None else i32(count), slots=True)
    stack, want_pages, want_held, want_room, want_slots = ref.plan(s.free, s.top, s.page, s.pages, s.held, length, count, n)
    assert room.tolist() == want_room and held.tolist() == want_held
    assert pages.tolist() == want_pages
    assert int(pool.top) == len(stack) and pool.free[:len(stack)].tolist() == stack
    assert torch.equal(slots.cpu(), torch.from_numpy(want_slots))
    s.free[:len(stack)], s.top = stack, len(stack)
    s.pages, s.held = np.array(want_pages, np.int32), np.array(want_held, np.int32)


@pytest.mark.parametrize("B,P,page,n,pool", [(1, 1, 1, 1, 1), (1, 9, 16, 8, 5), (5, 12, 3, 7, 40), (64, 20, 16, 24, 700), (65, 6, 64, 1, 200),
                                             (300, 40, 8, 33, 6000), (1500, 7, 5, 2, 9000), (40, 64, 16, 700, 1200)])
def test_plan_over_steps(wl, gpu, B, P, page, n, pool):
    """Sequences grow, are cut back, end and begin again; the pool runs short in some steps; lengths pass the table."""
    rs = np.random.RandomState(B + P)
    s = _State(pool, page, B, P, B)
    dp = wl.PagePool(torch.tensor(s.free, device=gpu), torch.tensor([s.top], dtype=torch.int32, device=gpu), page)
    pages, held = torch.tensor(s.pages, device=gpu), torch.tensor(s.held, device=gpu)
    length = np.zeros(B, np.int64)
    for step in range(8):
        count = None if step == 3 else [int(v) for v in rs.randint(-1, n + 2, B)]
        _plan_both(wl, s, gpu, dp, pages, held, length.tolist(), count, n)
        taken = (s.pages >= 0).sum()
        assert taken + s.top == pool and len(set(s.pages[s.pages >= 0].tolist())) == taken
        length = np.maximum(0, length + rs.randint(0, n + 1, B))
        length[rs.rand(B) < 0.2] = 0
        if step == 5:
            length[::3] = -7
        if step == 6:
            length[::4] = P * page + 5
    ok(wl)


def test_plan_undone_restores_everything(wl, gpu):
    s = _State(500, 16, 50, 20, 1)
    dp = wl.PagePool(torch.tensor(s.free, device=gpu), torch.tensor([s.top], dtype=torch.int32, device=gpu), 16)
    pages, held = torch.tensor(s.pages, device=gpu), torch.tensor(s.held, device=gpu)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    a = [(37 * b) % 150 for b in range(50)]
    wl.wl_page_plan(dp, pages, held, i32(a))
    before = [t.clone() for t in (pages, held, dp.top)] + [dp.free[:int(dp.top)].clone()]
    room, slots = wl.wl_page_plan(dp, pages, held, i32([(91 * b) % 140 for b in range(50)]), 5)
    assert slots is None and room.min() >= 0
    wl.wl_page_plan(dp, pages, held, i32(a))
    for x, y in zip(before, (pages, held, dp.top, dp.free[:int(dp.top)])):
        assert torch.equal(x, y)


def test_plan_feeds_the_cache(wl, gpu):
    """Slots are the rows of a cache with one kv head: what wl_rope_append writes there is what the slots say."""
    B, n, page, dim = 3, 5, 4, 16
    dp = wl.PagePool.full(20, page, gpu)
    pages, held = torch.full((B, 6), -1, dtype=torch.int32, device=gpu), torch.zeros(B, dtype=torch.int32, device=gpu)
    length = torch.tensor([0, 3, 9], dtype=torch.int32, device=gpu)
    room, slots = wl.wl_page_plan(dp, pages, held, length, n, slots=True)
    cache = wl.KVCache.empty(20, 1, page, dim, BF, gpu)
    k = torch.randn(B * n, dim, generator=gen(1)).to(BF).to(gpu)
    wl.wl_rope_append(None, k, k, None, None, cache, wl.CacheSeqs(pages, length, n, room))
    assert torch.equal(cache.k.view(-1, dim)[slots.view(-1)], k)
    ok(wl)
