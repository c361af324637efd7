"""The decoder-layer operators together: weightless layers with rotary positions,
a quantised cache, tree attention and norms (decoder.py), against the same
layer in 64 bits and against itself run another way."""
import math

import pytest
import torch

import wl_synth
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
SH = dict(hidden=192, q=256, kv=128, inter=320)  # 4 query heads and 2 kv heads of 64


def _decoder(wl, gpu, L=2, batch=2, max_len=256, dtype=torch.float8_e4m3fn, seed=0, rope=True):
    from rank_weight_reconstruction_wl_gb300 import decoder
    from rank_weight_reconstruction_wl_gb300.stack import build_layers

    layers = build_layers(L, L, 1, SH, 4, seed, gpu)
    g = wl_synth.make_generator(seed + 1)
    w = lambda: (0.1 * torch.randn(SH["hidden"], generator=g)).to(gpu)  # noqa: E731
    norms = [decoder.BlockNorms(w(), w(), w(), w()) for _ in range(L)]
    table = wl.RopeTable.make(64, 10000.0, device=gpu) if rope else None
    return decoder.Decoder(layers, norms, w(), 2, table, batch, max_len, 16, dtype)


def _x(gpu, B, T, seed=5):
    return torch.randn(B, T, SH["hidden"], generator=wl_synth.make_generator(seed)).to(gpu)


def _near(a, b, tol, what):
    a, b = a.double().cpu(), b.double().cpu()
    rms = float(b.pow(2).mean().sqrt())
    worst = float((a - b).abs().max()) / rms
    assert worst <= tol, f"{what}: {worst:.3g} of rms"


def _exact(dec, x):
    """The decoder in 64 bits on the CPU, a prompt of one sequence (no cache: k and v as they are)."""
    dec_w = lambda th: (th.s.double().cpu()[:, None] * th.W0.double().cpu() + th.U.double().cpu() @ th.V.double().cpu().T)  # noqa: E731
    T = x.shape[0]
    x = x.double().cpu()
    norm = lambda a, w: a / (a.pow(2).mean(-1, keepdim=True) + dec.eps).sqrt() * (1 + w.double().cpu())  # noqa: E731
    freq = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    for l, (th, nm) in enumerate(zip(dec.layers, dec.norms)):
        h = norm(x, nm.attn_pre)
        q, k, v = (h @ dec_w(t).T for t in (th.q, th.k, th.v))
        q, k, v = q.view(T, 4, 64), k.view(T, 2, 64), v.view(T, 2, 64)
        q, k = (ref.rotate(t, torch.arange(T), freq, False, 1.0) for t in (q, k))
        o = torch.empty(T, 4, 64, dtype=F64)
        for hd in range(4):
            s = (q[:, hd] @ k[:, hd // 2].T) / 8
            s = torch.where(torch.ones(T, T).tril().bool(), s, -math.inf)
            o[:, hd] = torch.softmax(s, -1) @ v[:, hd // 2]
        x = x + norm(o.view(T, 256) @ dec_w(th.o).T, nm.attn_post)
        h = norm(x, nm.mlp_pre)
        m = torch.nn.functional.gelu(h @ dec_w(th.gate).T, approximate="tanh") * (h @ dec_w(th.up).T)
        x = x + norm(m @ dec_w(th.down).T, nm.mlp_post)
    return norm(x, dec.final)


@pytest.mark.parametrize("T", [1, 20, 64, 100])
def test_prompt_against_64_bits(wl, gpu, T):
    """bf16 cache.  About ten bf16 roundings (2^-9 each, of terms as large as the
    states) lie between x and the result of two layers: 0.1 of rms is six sigma."""
    dec = _decoder(wl, gpu, batch=1, dtype=torch.bfloat16)
    x = _x(gpu, 1, T)
    h = dec.prompt(x)
    _near(h[0], _exact(dec, x[0])[-1], 0.1, f"T {T}")
    assert int(dec.len[0]) == T
    assert wl.wl_device_status() == wl.WL_OK


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
def test_chunks_equal_single_tokens(wl, gpu, dtype):
    """A prompt in chunks and token by token fill the cache with the same rows up
    to the projections' accumulation order (a bf16 step of k may move a code)."""
    x = _x(gpu, 2, 70)
    a, b = _decoder(wl, gpu, dtype=dtype), _decoder(wl, gpu, dtype=dtype)
    ha = a.prompt(x)
    for t in range(70):
        hb = b.step(x[:, t].contiguous(), 1)
        b.accept()
    _near(ha, hb, 0.1, "last state")
    assert torch.equal(a.len, b.len)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
def test_tree_paths_equal_chains(wl, gpu, dtype):
    """Each node of a drafted tree gets what a chain of its ancestors would have
    got; after accept() decoding goes on from the accepted path."""
    B, n = 2, 6
    x, tree, nxt = _x(gpu, B, 33, 6), _x(gpu, B, n, 7), _x(gpu, B, 1, 8)
    parent = [-1, 0, 0, 1, 2, 4]  # two branches: 0-1-3 and 0-2-4-5
    paths = []
    for i in range(n):
        p = [i]
        while parent[p[0]] >= 0:
            p.insert(0, parent[p[0]])
        paths.append(p)
    mask = torch.tensor([[sum(1 << j for j in p) for p in paths]] * B, dtype=torch.int64, device=gpu)
    depth = torch.tensor([[len(p) - 1 for p in paths]] * B, dtype=torch.int32, device=gpu)
    dec = _decoder(wl, gpu, dtype=dtype)
    dec.prompt(x)
    h = dec.step(tree.reshape(B * n, -1), n, mask, depth).view(B, n, -1).clone()
    path = paths[5]
    dec.accept(torch.tensor([path] * B, device=gpu))
    after = dec.step(nxt.reshape(B, -1), 1)
    for p in (paths[3], path):
        chain = _decoder(wl, gpu, dtype=dtype)
        chain.prompt(x)
        hc = chain.step(tree[:, p].reshape(B * len(p), -1).contiguous(), len(p)).view(B, len(p), -1)
        for at, node in enumerate(p):
            _near(h[:, node], hc[:, at], 0.1, f"node {node}")
        chain.accept()
    assert torch.equal(dec.len, chain.len)
    _near(after, chain.step(nxt.reshape(B, -1), 1), 0.1, "after the accepted path")
    assert wl.wl_device_status() == wl.WL_OK


def test_ragged_accept(wl, gpu):
    """Sequences accept different numbers of drafted tokens."""
    x, draft, nxt = _x(gpu, 2, 10, 9), _x(gpu, 2, 4, 10), _x(gpu, 2, 1, 11)
    dec = _decoder(wl, gpu)
    dec.prompt(x)
    dec.step(draft.reshape(8, -1), 4)
    dec.accept(torch.tensor([[0, 1, 2, 3]] * 2, device=gpu), torch.tensor([1, 3], dtype=torch.int32, device=gpu))
    assert dec.len.tolist() == [11, 13]
    h = dec.step(nxt.reshape(2, -1), 1)
    for b, k in ((0, 1), (1, 3)):
        one = _decoder(wl, gpu, batch=1)
        one.prompt(torch.cat((x[b:b + 1], draft[b:b + 1, :k]), 1))
        _near(h[b], one.step(nxt[b], 1)[0], 0.1, f"sequence {b}")


def test_refusals(wl, gpu):
    dec = _decoder(wl, gpu)
    with pytest.raises(ValueError, match="1 to 64"):
        dec.step(torch.zeros(130, SH["hidden"], device=gpu), 65)
    with pytest.raises(ValueError, match="needs a step"):
        dec.accept()


def test_a_sequence_does_not_pass_its_room(wl, gpu):
    """A step that would pass max_len is refused before anything runs; what fits goes on."""
    dec = _decoder(wl, gpu, max_len=32)
    x = _x(gpu, 2, 40)
    for T in (40, 33):
        with pytest.raises(ValueError, match=f"{T} of 32"):
            dec.prompt(x[:, :T])
    with pytest.raises(ValueError, match="100 of 32"):
        dec.prompt(_x(gpu, 2, 100))
    assert dec.len.tolist() == [0, 0]
    dec.prompt(x[:, :30])
    assert dec.len.tolist() == [30, 30]
    with pytest.raises(ValueError, match="33 of 32"):
        dec.step(x[:, :3].reshape(6, -1).contiguous(), 3)
    # one sequence takes two more, the other none: the room of each counts, not n
    some = torch.tensor([2, 0], dtype=torch.int32, device=gpu)
    dec.step(x[:, :3].reshape(6, -1).contiguous(), 3, count=some)
    dec.accept()
    assert dec.len.tolist() == [32, 30]
    with pytest.raises(ValueError, match="33 of 32"):
        dec.step(x[:, :1].reshape(2, -1).contiguous(), 1)
    dec.len.zero_()  # the sequences begin anew
    dec.prompt(x[:, :32])
    assert dec.len.tolist() == [32, 32] and wl.wl_device_status() == wl.WL_OK


def test_accept_counts_what_the_step_had(wl, gpu):
    """accept() after a ragged step counts the step's tokens, no more; paths may be padded with anything."""
    x, draft, nxt = _x(gpu, 2, 10, 9), _x(gpu, 2, 4, 10), _x(gpu, 2, 1, 11)
    had = torch.tensor([1, 3], dtype=torch.int32, device=gpu)
    last = []
    for how in ("plain", "more", "path"):
        dec = _decoder(wl, gpu)
        dec.prompt(x)
        dec.step(draft.reshape(8, -1), 4, count=had)
        if how == "plain":
            dec.accept()
        elif how == "more":
            dec.accept(count=torch.tensor([4, 9], dtype=torch.int32, device=gpu))
        else:
            dec.accept(torch.tensor([[0, 1 << 40, -9, 4], [0, 1, 2, 1 << 40]], device=gpu), had)
        assert dec.len.tolist() == [11, 13], how
        last.append(dec.step(nxt.reshape(2, -1), 1))
    assert torch.equal(last[0], last[1]) and torch.equal(last[0], last[2])
    assert wl.wl_device_status() == wl.WL_OK


def test_accept_refusals(wl, gpu):
    dec = _decoder(wl, gpu)
    dec.step(_x(gpu, 2, 3).reshape(6, -1), 3)
    for bad in (torch.zeros(2, 4), torch.zeros(1, 2), torch.zeros(2, 0), torch.zeros(2)):
        with pytest.raises(ValueError, match="path must be"):
            dec.accept(bad.long().to(gpu))
    dec.accept(torch.zeros(2, 1, dtype=torch.int64, device=gpu))  # the step is still there
    with pytest.raises(ValueError, match="at least one token"):
        dec.prompt(_x(gpu, 2, 1)[:, :0])


def test_a_captured_step_grows_the_sequences(wl, gpu):
    """Replays of one captured step and accept() give what calls give; the room is checked on the lengths they left."""
    x, buf = _x(gpu, 2, 60), torch.empty(2, SH["hidden"], device=gpu)
    called, replayed = _decoder(wl, gpu, max_len=64), _decoder(wl, gpu, max_len=64)
    for dec in (called, replayed):
        dec.prompt(x[:, :20])
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    with torch.cuda.stream(side):  # (what a first call sets up)
        buf.copy_(x[:, 20])
        replayed.step(buf, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        h = replayed.step(buf, 1)
        replayed.accept()
    for t in range(20, 60):
        buf.copy_(x[:, t])
        graph.replay()
        want = called.step(x[:, t].contiguous(), 1)
        called.accept()
        assert torch.equal(h, want), t
    assert replayed.len.tolist() == called.len.tolist() == [60, 60]
    with pytest.raises(ValueError, match="65 of 64"):
        replayed.step(x[:, :5].reshape(10, -1).contiguous(), 5)
    replayed.step(x[:, :4].reshape(8, -1).contiguous(), 4)
    assert wl.wl_device_status() == wl.WL_OK
