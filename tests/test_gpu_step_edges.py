"""Operators between a step's last states and the next step: clusters under load,
starved sequences, decisions near a border, scales at the ends of fp32."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_decoder import _near, _x
from tests.test_gpu_decoder_step import _with_head
from tests.test_gpu_step_ops import _factors

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("B", [65, 273, 1030])
def test_plans_of_clusters_on_a_busy_gpu(wl, gpu, B):
    """Plans on two streams beside a stream of products, so that a cluster's CTAs do not begin alike: all as one after another."""
    page, P, n, steps = 16, 30, 20, 12
    rs = np.random.RandomState(B)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    lengths = [rs.randint(0, P * page - n, B).tolist() for _ in range(steps)]
    dev_lengths = [i32(v) for v in lengths]
    a = torch.randn(4096, 4096, device=gpu, dtype=BF)
    streams = [torch.cuda.Stream(gpu) for _ in range(2)]
    pools = [wl.PagePool.full(B * P // 2, page, gpu) for _ in streams]
    pages = [i32(np.full((B, P), -1)) for _ in streams]
    held = [i32(np.zeros(B)) for _ in streams]
    torch.cuda.synchronize()
    got = [[], []]
    for step in range(steps):
        a @ a
        for k, st in enumerate(streams):
            got[k].append(wl.wl_page_plan(pools[k], pages[k], held[k], dev_lengths[step], n, slots=True, stream=st))
    torch.cuda.synchronize()
    free, top = list(range(B * P // 2))[::-1], B * P // 2
    table, have = [[-1] * P for _ in range(B)], [0] * B
    for step in range(steps):
        stack, table, have, room, slots = ref.plan(free, top, page, table, have, lengths[step], None, n)
        free, top = stack, len(stack)
        for k in range(2):
            assert got[k][step][0].tolist() == room and np.array_equal(got[k][step][1].cpu().numpy(), slots)
    for k in range(2):
        assert pages[k].tolist() == table and held[k].tolist() == have and pools[k].free[:top].tolist() == free


@pytest.mark.parametrize("temp", [0.0, 0.8])
def test_a_starved_sequence_keeps_its_token(wl, gpu, temp):
    """A sequence that waits two steps for pages goes on from the token that it had: states and tokens of a decoder whose
    sequences have pages of their own and sit the same steps out."""
    few, embed = _with_head(wl, gpu, 5, max_len=64)  # pages of 16: both prompts and one page
    own, _ = _with_head(wl, gpu, None, max_len=64)
    x = _x(gpu, 2, 32)
    h = few.prompt(x)
    assert torch.equal(h, own.prompt(x))
    tok = {d: d.logits(h, F32).argmax(-1).to(torch.int32) for d in (few, own)}
    first = tok[few].tolist()
    for k in range(6):
        if k == 2:
            done = torch.tensor([True, False], device=gpu)
            few.release(done), own.release(done)
        live = [1, 0] if k < 2 else [0, 1]
        count = torch.tensor(live, dtype=torch.int32, device=gpu)
        u = torch.rand(2, 1, generator=torch.Generator().manual_seed(k)).to(gpu)
        for d in (few, own):
            h = d.step(embed[tok[d].long()], 1, count=None if d is few and k < 2 else count)
            _, acc, token = d.verify(d.logits(h, F32), tok[d][:, None], u, temperature=temp)
            assert acc.tolist() == live and [t >= 0 for t in token.tolist()] == [v == 1 for v in live]
            assert d.next.tolist() == [int(token[b]) if live[b] else int(tok[d][b]) for b in range(2)]
            tok[d] = d.next
        if k < 2:
            assert few.room.tolist() == live and int(tok[few][1]) == first[1]
        assert torch.equal(tok[few], tok[own])
    assert few.len.tolist() == own.len.tolist() == [0, 36]
    assert wl.wl_device_status() == wl.WL_OK


def test_next_without_and_with_a_distribution(wl, gpu):
    """next is the token drawn where all sequences take part, and -1 where a row has no distribution."""
    dec, embed = _with_head(wl, gpu)
    h = dec.step(_x(gpu, 2, 1).view(2, -1), 1)
    logits = dec.logits(h, F32)
    logits[1, 7] = float("nan")
    tokens = torch.tensor([[3], [4]], dtype=torch.int32, device=gpu)
    _, acc, token = dec.verify(logits, tokens, torch.zeros(2, 1, device=gpu), temperature=0.0)
    assert acc.tolist() == [1, 1] and token.tolist() == dec.next.tolist() == [int(logits[0].argmax()), -1]


@pytest.mark.parametrize("tree", [False, True])
def test_a_step_fills_the_last_page_where_there_are_no_more(wl, gpu, tree):
    """A sequence of 30 in pages of 16, none left: a step of 5 takes its first two nodes, the next step none; once there is a
    page the sequence goes on as one that took the same tokens in a prompt."""
    dec, embed = _with_head(wl, gpu, 3, batch=1, max_len=64)
    ids = torch.randint(0, 500, (1, 30), generator=torch.Generator().manual_seed(1)).to(gpu)
    h = dec.prompt(embed[ids])
    dec.pool.top -= 1  # the last page is somebody else's for now
    assert int(dec.pool.top) == 0
    tok = int(dec.logits(h, F32).argmax())
    mask = depth = None
    if tree:  # 1, 2 and 3 follow the root, 4 follows 1
        mask = torch.tensor([[1, 3, 5, 9, 19]], device=gpu)
        depth = torch.tensor([[0, 1, 1, 1, 2]], dtype=torch.int32, device=gpu)
    tokens = torch.tensor([[tok, 7, 8, 9, 10]], dtype=torch.int32, device=gpu)
    h = dec.step(embed[tokens[0].long()], 5, mask, depth)
    assert dec.room.tolist() == [2]
    logits = dec.logits(h, F32)
    logits[0, 7] = 1e4  # node 1 is the likeliest, and so would be nodes 2 and 4 behind it, which are not there
    logits[1:, 8:11] = 1e4
    path, acc, token = dec.verify(logits, tokens, torch.zeros(1, 5, device=gpu), mask=mask, temperature=0.0)
    assert path.tolist() == [[0, 1, -1, -1, -1]] and acc.tolist() == [2] and token.tolist() == dec.next.tolist() == [8]
    assert dec.len.tolist() == [32] and dec.held.tolist() == [2]
    h = dec.step(embed[dec.next.long()], 1)
    assert dec.room.tolist() == [0]
    _, acc, token = dec.verify(dec.logits(h, F32), dec.next[:, None], torch.zeros(1, 1, device=gpu))
    assert acc.tolist() == [0] and token.tolist() == [-1] and dec.next.tolist() == [8] and dec.len.tolist() == [32]
    dec.pool.top += 1
    h = dec.step(embed[dec.next.long()], 1)
    assert dec.room.tolist() == [1]
    whole, _ = _with_head(wl, gpu, None, batch=1)
    text = ids[0].tolist() + [tok, 7, 8]
    # the same text, fed in other steps: up to the projections' accumulation order, as the decoder's other tests
    _near(h[0], whole.prompt(embed[torch.tensor([text], device=gpu)])[0], 0.1, "states")
    assert wl.wl_device_status() == wl.WL_OK


def test_verify_takes_the_mask_of_its_step(wl, gpu):
    """A tree verified without a mask is the step's tree, not a chain."""
    mask = torch.tensor([[1, 3, 5]] * 2, device=gpu)  # two children of the root
    depth = torch.tensor([[0, 1, 1]] * 2, dtype=torch.int32, device=gpu)
    tokens = torch.tensor([[1, 2, 3]] * 2, dtype=torch.int32, device=gpu)
    found = []
    for given in (mask, None):
        dec, embed = _with_head(wl, gpu)
        h = dec.step(embed[tokens.view(-1).long()], 3, mask, depth)
        logits = dec.logits(h, F32)
        logits[0::3, 3] = 1e4  # the second child
        got = dec.verify(logits, tokens, torch.zeros(2, 3, device=gpu), mask=given, temperature=0.0)
        found.append([t.tolist() for t in got] + [dec.len.tolist(), dec.step(embed[got[2].long()], 1).tolist()])
    assert found[0] == found[1] and found[0][0] == [[0, 2, -1]] * 2


def _near_borders(V, B, seed):
    """Stars of five children of which the first b % 5 are rejected against a draft distribution; then the next child's draw, or
    the next token's, lies beside a border, as near as fp32 goes, but 2^-29 of the row's sum at least.  Returns the arguments, what
    follows in 64 bits (accepted node or 0, next token) and how near each sequence comes to any border."""
    rs = np.random.RandomState(seed)
    n, t = 6, 0.8
    mask = np.array([[1 | 1 << i for i in range(n)]] * B, np.int64)
    logits = (2 * rs.randn(B * n, V)).astype(np.float32)
    draft = np.zeros((B * n, V), np.float32)
    tokens, draws, count = np.zeros((B, n), np.int32), np.full((B, n), 0.5, np.float32), np.zeros(B, np.int32)
    want, near = [], []

    def beside(x, ok):
        """An fp32 number in (0, 1) beside x, on a random side, the nearest of a series of growing steps for which ok."""
        side = 1 if rs.rand() < 0.5 else -1
        for k in range(120):
            v = np.float32(x + side * np.spacing(np.float32(x)) * 1.15 ** k)
            if (float(v) - x) * side > 0 and 0 < v < 1 and ok(float(v)):
                return v
        return None

    for b in range(B):
        z = logits[b * n].astype(np.float64)
        w = np.exp((z - z.max()) / t)
        p = np.exp(z + 0.7 * rs.randn(V))
        q32 = (p / p.sum()).astype(np.float32)
        draft[b * n] = q32
        q = q32.astype(np.float64)
        S0, R, least, got = w.sum(), w.copy(), np.inf, 0
        test_child = b % 2 == 0
        c = 1
        for _ in range(b % 5):
            S = R.sum()
            odds = R / (q * S)
            can = np.nonzero(odds < 0.97)[0]
            if len(can) == 0 or np.maximum(R - S * q, 0.0).sum() < 1e-3 * S0:
                break  # none can be rejected, or little would be left
            k = rs.choice(can)
            tokens[b, c], draws[b, c] = k, np.float32(0.5 * (odds[k] + 1))
            least = min(least, abs(float(draws[b, c]) * q[k] * S - R[k]) / S0)
            R = np.maximum(R - S * q, 0.0)
            c += 1
        S = R.sum()
        odds = R / (q * S)
        can = np.nonzero((odds > 0.01) & (odds < 0.99))[0]
        test_child = test_child and len(can) > 0
        if test_child:
            k = can[np.argsort(-q[can])[rs.randint(min(5, len(can)))]]  # of the likelier ones: the others' borders are far from fp32's numbers
            r = beside(odds[k], lambda v: abs(v * q[k] * S - R[k]) >= 2.0 ** -29 * S0)
            r = np.float32(0.5 * odds[k]) if r is None else r
            tokens[b, c], draws[b, c] = k, r
            least = min(least, abs(float(r) * q[k] * S - R[k]) / S0)
            if float(r) * q[k] * S < R[k]:
                got = c
                z = logits[b * n + c].astype(np.float64)
                R = np.exp((z - z.max()) / t)
            else:
                R = np.maximum(R - S * q, 0.0)
            c += 1
        P, S = np.cumsum(R), R.sum()
        scale = P[-1] if got else S0
        can = np.nonzero((R > 0.1 * S / V) & (P < 0.999 * S))[0]
        u = None
        if not test_child and len(can) > 0:
            u = beside(P[rs.choice(can)] / S, lambda v: np.abs(P - v * S).min() >= 2.0 ** -29 * scale)
        if u is None:
            i = int(np.argmax(R))
            u = np.float32((P[i] - 0.5 * R[i]) / S)
        draws[b, 0], count[b] = u, c
        least = min(least, np.abs(P - float(u) * S).min() / scale)
        want.append((got, int(np.nonzero((R > 0) & (P > float(u) * S))[0][0])))
        near.append(least)
    args = [torch.from_numpy(a) for a in (logits, tokens, draws, mask, count, draft)]
    return args, want, np.array(near)


@pytest.mark.parametrize("V,B", [(6, 1000), (40, 2000), (9001, 300)])
def test_decisions_beside_borders_after_rejections(wl, gpu, V, B):
    """Decisions are those of exact arithmetic where no border lies within 2^-29 of the row's sum, after rejections too."""
    (logits, tokens, draws, mask, count, draft), want, near = _near_borders(V, B, V)
    assert near.min() >= 2.0 ** -29 and (near < 2.0 ** -25).sum() > B // 8
    path, acc, nxt = wl.wl_verify(logits.to(gpu), tokens.to(gpu), draws.to(gpu), mask=mask.to(gpu), count=count.to(gpu), draft=draft.to(gpu),
                                  temperature=0.8)
    got = [(int(p[1]) if a == 2 else 0, t) for p, a, t in zip(path.tolist(), acc.tolist(), nxt.tolist())]
    wrong = [b for b in range(B) if got[b] != want[b]]
    assert not wrong, [(b, got[b], want[b], np.log2(near[b])) for b in wrong[:5]]


@pytest.mark.parametrize("T,inner,out", [(3, 272, 130), (20, 1152, 9741), (100, 272, 20008), (300, 400, 1000)])
def test_products_of_scales_at_the_ends_of_fp32(wl, gpu, T, inner, out):
    """A block is scaled by the product of its scales rounded to fp32: subnormal, zero or infinite where that is."""
    x, xs, w, ws = _factors(T, inner, out, T)
    kb = xs.shape[0]
    xs[:, 0], ws[:, 0] = 2.0 ** -126, 3e-4  # subnormal, 13 bits
    xs[0, 1] = 2.0 ** -149  # 0 with ws
    ws[kb - 1] *= 2.0 ** 40
    xs[kb - 1, 2] = 2.0 ** 120  # infinite
    y = wl.wl_linear_f8(x.to(gpu), xs.to(gpu), wl.F8Weight(w.to(gpu), ws.to(gpu)), ydt=F32).double().cpu().numpy()
    want, mag = np.zeros((T, out)), np.zeros((T, out))
    with np.errstate(over="ignore", invalid="ignore"):
        for k in range(kb):
            at = slice(128 * k, 128 * (k + 1))
            scale = (xs[k].numpy()[:, None] * np.repeat(ws[k].numpy(), 128)[None, :out]).astype(np.float64)  # rounded to fp32
            a, b = x[:, at].double().numpy(), w[:, at].double().numpy()
            want += (a @ b.T) * scale
            mag += (np.abs(a) @ np.abs(b).T) * scale
    assert np.isinf(mag[2]).all() and np.isfinite(np.delete(mag, 2, 0)).all()
    assert not np.isfinite(y[2]).any()
    live = np.ones(T, bool)
    live[2] = False
    # as the other products, and fp32's subnormal step for each block and the result
    tol = (128 * 2.0 ** -23 + (kb + 2) * 2.0 ** -23) * mag + 2.0 ** -24 * np.abs(want) + (kb + 1) * 2.0 ** -149
    assert (np.abs(y[live] - want[live]) <= tol[live]).all()
    assert y[0, :128].any()
    assert wl.wl_device_status() == wl.WL_OK


def test_an_infinite_temperature_keeps_masks_of_the_lowest_value(wl, gpu):
    """A temperature counts as 1e30 at most: what is masked by fp32's lowest value has no weight, the rest is as good as equal."""
    V, B = 300, 16
    a = torch.full((B, V), torch.finfo(F32).min)
    a[:, 40:104] = torch.linspace(-3, 3, 64)
    u = ((torch.arange(B) + 0.5) / B)[:, None].float()
    temp = torch.full((B,), float("inf"))
    temp[1::2] = 3e38
    _, _, nxt = wl.wl_verify(a.to(gpu), torch.zeros(B, 1, dtype=torch.int32, device=gpu), u.to(gpu), temperature=temp.to(gpu))
    assert nxt.tolist() == [40 + int(64 * (b + 0.5) / B) for b in range(B)]
