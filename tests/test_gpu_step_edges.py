"""Operators between a step's last states and the next step: clusters under load,
starved sequences, decisions near a border, scales at the ends of fp32."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_decoder import _near, _x
from tests.test_gpu_decoder_step import _with_head

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
