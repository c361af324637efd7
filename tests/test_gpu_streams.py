"""Calls on a stream that is not the current one: what they allocate belongs to
that stream, so that neither side's queued work can reach the other's block."""
import pytest
import torch

import wl_synth

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _late_write(shape, dtype, dev):
    """A block of this size goes back to the current stream's pool with a write to it still to come."""
    x = torch.empty(shape, dtype=dtype, device=dev)
    torch.cuda._sleep(100_000_000)  # some 50 ms
    x.fill_(7.0)
    return x.data_ptr()


def _check(gpu, call, shapes):
    """call(stream) -> tensors; equal with the current stream's and with a late write pending there."""
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for shape, dtype in shapes:
        _late_write(shape, dtype, gpu)
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    raw = call(side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(want, raw):
        assert torch.equal(a, b)


def _cache(wl, gpu, T=512, kv=8, dim=128):
    z = dict(dtype=torch.int32, device=gpu)
    cache = wl.KVCache.empty(T // 64, kv, 64, dim, device=gpu)
    seqs = wl.CacheSeqs(torch.arange(T // 64, **z)[None], torch.zeros(1, **z), T)
    k = torch.randn(T, kv * dim, generator=wl_synth.make_generator(1)).to(BF).to(gpu)
    return cache, seqs, k


def test_append_and_read_on_another_stream(wl, gpu):
    cache, seqs, k = _cache(wl, gpu)
    q = k[:, :1024].contiguous()
    _check(gpu, lambda st: [wl.wl_rope_append(q, k, k, None, None, cache, seqs, stream=st)], [((512, 1024), BF)])
    _check(gpu, lambda st: wl.wl_cache_read(cache, seqs, stream=st), [((1, 512, 8, 128), BF)] * 2)


def test_attention_on_another_stream(wl, gpu):
    cache, seqs, k = _cache(wl, gpu)
    wl.wl_rope_append(None, k, k, None, None, cache, seqs)
    z = dict(dtype=torch.int32, device=gpu)
    tree = wl.CacheSeqs(seqs.pages, torch.full((1,), 448, **z), 64)
    q = torch.randn(1, 64, 32, 128, generator=wl_synth.make_generator(2)).to(BF).to(gpu)
    nb = wl.wl_tree_attention_workspace_bytes(1, 64, 32, 8, 128)
    _check(gpu, lambda st: [wl.wl_tree_attention(q, cache, tree, stream=st)], [((1, 64, 32, 128), BF), ((nb,), torch.uint8)])


def test_norm_on_another_stream(wl, gpu):
    x = torch.randn(512, 1024, generator=wl_synth.make_generator(3)).to(gpu)
    w = torch.ones(1024, device=gpu)
    _check(gpu, lambda st: wl.wl_norm_residual(x, x, w, w, h_dt=torch.float32, stream=st), [((512, 1024), torch.float32)] * 2)


def test_projections_on_another_stream(wl, gpu):
    T, inp, out, r = 256, 1024, 1152, 8
    g = wl_synth.make_generator(4)
    x = wl_synth.draw_x(g, T, inp).to(gpu)
    th = [t.to(gpu) for t in _bundle(g, inp, out, r)]
    _check(gpu, lambda st: [wl.wl_linear(x, *th, stream=st)], [((T, out), BF)])
    _check(gpu, lambda st: wl.wl_qkv_fused(x, th, th, th, stream=st), [((T, out), BF)] * 3)
    _check(gpu, lambda st: [wl.wl_materialize(*th, stream=st)], [((out, inp), BF)])
    f = [t.float() for t in th]
    _check(gpu, lambda st: [wl.wl_linear(x.float(), *f, ydt=torch.float32, stream=st)], [((T, out), torch.float32)])
    back = [t.to(gpu) for t in _bundle(g, out, inp, r)]
    _check(gpu, lambda st: [wl.wl_mlp_geglu_fused(x, th, th, back, stream=st)], [((T, inp), BF)])
    Ws = [th[0], th[0] + th[0]]
    _check(gpu, lambda st: wl.wl_decompose_band(Ws, 4, stream=st),
           [((out, inp), BF), ((2, out), torch.float32), ((2, out, 4), BF), ((2, inp, 4), BF), ((inp, 12), torch.float32)])


def _bundle(g, inp, out, r):
    th = wl_synth.draw_theta(g, inp, out, r)
    return th.W0, th.s, th.U, th.V
