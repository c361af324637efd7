"""The decoder with a head and shared pages: step, logits, verification and page
plan together, against itself run another way."""
import pytest
import torch

import wl_synth
from tests import step_ref as ref
from tests.test_gpu_decoder import SH, _decoder, _near, _x

pytestmark = pytest.mark.gpu
VOCAB = 500


def _with_head(wl, gpu, pool_pages=None, batch=2, max_len=256, seed=0):
    """A decoder with a head, and the embeddings of its tokens."""
    from rank_weight_reconstruction_wl_gb300 import decoder

    d = _decoder(wl, gpu, batch=batch, max_len=max_len, seed=seed)
    g = wl_synth.make_generator(seed + 7)
    head = wl.F8Weight.quantise((torch.randn(VOCAB, SH["hidden"], generator=g) * 0.3).to(gpu))
    embed = torch.randn(VOCAB, SH["hidden"], generator=g).to(gpu)
    return decoder.Decoder(d.layers, d.norms, d.final, 2, d.rope, batch, max_len, 16, head=head, pool_pages=pool_pages), embed


def _prompt(dec, embed, T, seed=3):
    ids = torch.randint(0, VOCAB, (dec.batch, T), generator=wl_synth.make_generator(seed)).to(embed.device)
    return dec.prompt(embed[ids]), ids


def _checked(dec, h, tokens, uniforms, **kw):
    """dec.verify() of the step's logits, equal to the definition's in 64 bits."""
    logits = dec.logits(h, torch.float32)
    got = dec.verify(logits, tokens, uniforms, **kw)
    want = ref.verify(logits.cpu(), tokens.cpu(), uniforms.cpu(), **{k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    for a, b in zip(got, want):
        assert a.tolist() == b.tolist()
    return got


# States of a step against those of a prompt of the same tokens: up to the projections' accumulation order and the codes
# that a bf16 step of k moves, as the other tests of this decoder (0.1 of rms).  Which token is the likeliest may differ
# between the two where two logits are as near, so it is the step's own logits that the verification is held to.
@pytest.mark.parametrize("temp", [0.0, 0.8])
@pytest.mark.parametrize("pool", [None, 40])
def test_drafted_chains(wl, gpu, pool, temp):
    """Drafts that follow the model's likeliest tokens up to a place of their own, step after step; what is in the cache in
    the end is the prompt and the accepted tokens."""
    B, n = 2, 5
    dec, embed = _with_head(wl, gpu, pool)
    h, ids = _prompt(dec, embed, 30)
    text = [ids[b].tolist() for b in range(B)]
    tok = dec.logits(h, torch.float32).argmax(-1).to(torch.int32)
    some = 0
    for step in range(12):
        # the drafter: the model itself, a token at a time, on a decoder of its own
        tokens = tok[:, None].repeat(1, n)
        draft, _ = _with_head(wl, gpu, None, batch=1)
        for b in range(B):
            draft.len.zero_()
            draft._most = 0
            draft.prompt(embed[torch.tensor([text[b]], device=gpu)])
            for i in range(1, n):
                hd = draft.step(embed[tokens[b, i - 1].long()][None], 1)
                draft.accept()
                tokens[b, i] = int(draft.logits(hd, torch.float32).argmax())
            tokens[b, 1 + (step + 2 * b) % n:] = (tokens[b, 1 + (step + 2 * b) % n:] + 1) % VOCAB
        u = torch.rand(B, n, generator=wl_synth.make_generator(step)).to(gpu) * 0.5
        h = dec.step(embed[tokens.view(-1).long()], n)
        path, acc, tok = _checked(dec, h, tokens, u, temperature=temp)
        for b in range(B):
            some += int(acc[b]) > 1
            text[b] += tokens[b, :int(acc[b])].tolist()
    assert dec.len.tolist() == [len(v) for v in text] and some > 6
    h = dec.step(embed[tok.long()], 1)
    for b in range(B):
        whole, _ = _with_head(wl, gpu, None, batch=1)
        _near(h[b], whole.prompt(embed[torch.tensor([text[b] + [int(tok[b])]], device=gpu)])[0], 0.1, f"sequence {b}")
    assert wl.wl_device_status() == wl.WL_OK


def test_trees_keep_the_path_that_was_verified(wl, gpu):
    """Trees with the model's likeliest tokens on one branch, shared pages: the accepted path is what the cache holds after."""
    dec, embed = _with_head(wl, gpu, 30)
    h, ids = _prompt(dec, embed, 21)
    tok = dec.logits(h, torch.float32).argmax(-1).to(torch.int32)
    # node: 0 root; 1, 2 its children; 3, 4 of 2; 5 of 4.  The likely way is 0 2 4 5.
    par = [-1, 0, 0, 2, 2, 4]
    m = [0] * 6
    for i in range(6):
        m[i] = (1 << i) | (m[par[i]] if i else 0)
    mask = torch.tensor([m, m], device=gpu)
    depth = torch.tensor([[0, 1, 1, 2, 2, 3]] * 2, dtype=torch.int32, device=gpu)
    line = [tok]
    draft, _ = _with_head(wl, gpu)
    draft.prompt(embed[ids])
    for _ in range(3):
        hd = draft.step(embed[line[-1].long()], 1)
        draft.accept()
        line.append(draft.logits(hd, torch.float32).argmax(-1).to(torch.int32))
    tokens = torch.stack((tok, (line[1] + 1) % VOCAB, line[1], (line[2] + 3) % VOCAB, line[2], line[3]), 1).contiguous()
    h = dec.step(embed[tokens.view(-1).long()], 6, mask, depth)
    path, acc, nxt = _checked(dec, h, tokens, torch.zeros(2, 6, device=gpu), mask=mask, temperature=0.0)
    assert int(acc.max()) > 2
    h = dec.step(embed[nxt.long()], 1)
    for b in range(2):
        k = int(acc[b])
        text = ids[b].tolist() + tokens[b][path[b, :k].long()].tolist()
        assert int(dec.len[b]) == len(text)
        whole, _ = _with_head(wl, gpu, None, batch=1)
        _near(h[b], whole.prompt(embed[torch.tensor([text + [int(nxt[b])]], device=gpu)])[0], 0.1, f"sequence {b}")


def test_shared_pages_equal_own_pages(wl, gpu):
    """Sequences that end and begin again, in a pool smaller than batch * max_len: states as with pages of their own."""
    own, embed = _with_head(wl, gpu, batch=3)
    few, _ = _with_head(wl, gpu, 24, batch=3)  # 24 of 48 pages
    x = _x(gpu, 3, 70, seed=9)
    assert torch.equal(own.prompt(x), few.prompt(x))
    for k in range(6):
        x = _x(gpu, 3, 7, seed=20 + k).view(21, -1)
        count = torch.tensor([7, 3 + k % 4, 0 if k % 2 else 5], dtype=torch.int32, device=gpu)
        a, b = own.step(x, 7, count=count), few.step(x, 7, count=count)
        live = (torch.arange(7, device=gpu) < count[:, None]).view(-1)
        assert torch.equal(few.room, count) and torch.equal(a[live], b[live])
        own.accept(), few.accept()
        done = torch.tensor([False, k == 3, k == 2], device=gpu)
        own.release(done), few.release(done)
        assert torch.equal(own.len, few.len)
        used = (few.pages >= 0).sum(1)
        assert torch.equal(used.to(torch.int32), few.held) and int(used.sum()) + int(few.pool.top) == 24
    assert wl.wl_device_status() == wl.WL_OK


def test_where_pages_run_out(wl, gpu):
    """Of three sequences the pool has pages for two: the third takes no token until one of them ends."""
    dec, embed = _with_head(wl, gpu, 4, batch=3, max_len=64)
    x = _x(gpu, 3, 32).view(96, -1)
    dec.step(x, 32)
    assert dec.room.tolist() == [32, 32, 0]
    dec.accept()
    assert dec.len.tolist() == [32, 32, 0]
    h = dec.step(_x(gpu, 3, 1).view(3, -1), 1)
    assert dec.room.tolist() == [0, 0, 0]
    _, acc, nxt = dec.verify(dec.logits(h), torch.zeros(3, 1, dtype=torch.int32, device=gpu), torch.zeros(3, 1, device=gpu))
    assert acc.tolist() == [0, 0, 0] and nxt.tolist() == [-1, -1, -1] and dec.len.tolist() == [32, 32, 0]
    dec.release(torch.tensor([True, False, False], device=gpu))
    assert int(dec.pool.top) == 2
    dec.step(_x(gpu, 3, 20).view(60, -1), 20, count=torch.tensor([0, 5, 20], dtype=torch.int32, device=gpu))
    assert dec.room.tolist() == [0, 5, 0]
    dec.accept(torch.zeros(3, 20, dtype=torch.int64, device=gpu), torch.tensor([3, 5, 20], dtype=torch.int32, device=gpu))
    assert dec.len.tolist() == [0, 37, 0]
    with pytest.raises(ValueError, match="pages"):
        dec.prompt(_x(gpu, 3, 20))
    assert wl.wl_device_status() == wl.WL_OK


def test_refusals(wl, gpu):
    dec, embed = _with_head(wl, gpu)
    z = torch.zeros(2, 1, device=gpu)
    with pytest.raises(ValueError, match="needs a step"):
        dec.verify(torch.zeros(2, VOCAB, device=gpu), z.int(), z)
    h = dec.step(_x(gpu, 2, 1).view(2, -1), 1)
    with pytest.raises(ValueError, match="as the step's"):
        dec.verify(dec.logits(h), torch.zeros(2, 2, dtype=torch.int32, device=gpu), torch.zeros(2, 2, device=gpu))
    with pytest.raises(ValueError, match="done must be"):
        dec.release(torch.zeros(2, device=gpu))
    dec.head = None
    with pytest.raises(ValueError, match="needs a head"):
        dec.logits(h)
    with pytest.raises(ValueError, match="pool_pages"):
        _with_head(wl, gpu, 0)


def test_a_captured_speculative_step(wl, gpu):
    """Page plan, step, logits, verification and accept in one graph, replayed: the tokens and lengths of plain calls."""
    n, B = 4, 2

    def run(graph):
        dec, embed = _with_head(wl, gpu, 40)
        h, _ = _prompt(dec, embed, 18)
        tok = dec.logits(h, torch.float32).argmax(-1).to(torch.int32)
        tokens, u = torch.zeros(B, n, dtype=torch.int32, device=gpu), torch.zeros(B, n, device=gpu)
        outs = []

        def body():
            h = dec.step(embed[tokens.view(-1).long()], n)
            return dec.verify(dec.logits(h), tokens, u, temperature=0.7)

        def feed(k, tok):
            g = wl_synth.make_generator(50 + k)
            tokens[:, 0] = tok
            tokens[:, 1:] = torch.randint(0, VOCAB, (B, n - 1), generator=g).to(gpu)
            u.copy_(torch.rand(B, n, generator=g) * torch.tensor([1.0, 0.01, 0.01, 0.01]))

        feed(0, tok)
        _, acc, tok = body()
        outs.append((acc.tolist(), tok.tolist(), dec.len.tolist()))
        if graph:
            side = torch.cuda.CUDAGraph()
            with torch.cuda.graph(side):
                res = body()
        for k in range(1, 6):
            feed(k, tok)
            if graph:
                side.replay()
                _, acc, tok = res
                tok = tok.clone()
            else:
                _, acc, tok = body()
            outs.append((acc.tolist(), tok.tolist(), dec.len.tolist()))
        return outs

    assert run(True) == run(False)
    assert wl.wl_device_status() == wl.WL_OK
