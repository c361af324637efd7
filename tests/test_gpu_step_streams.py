"""The operators between a step's last states and the next step on streams of
their own, at the same time, in graphs, and beside memory that is not theirs."""
import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_step_ops import F8, _drafts, _factors, gen
from tests.test_gpu_streams import _check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_quant_and_product_on_another_stream(wl, gpu):
    x = torch.randn(300, 1152, generator=gen(1)).to(BF).to(gpu)
    _check(gpu, lambda st: [t.float() for t in wl.wl_quant_f8(x, stream=st)] if st is None else _after(st, gpu, wl.wl_quant_f8(x, stream=st)),
           [((300, 1152), F8), ((9, 300), F32)])
    w = wl.F8Weight.quantise(torch.randn(640, 1152, generator=gen(2)).to(gpu))
    c, s = wl.wl_quant_f8(x)
    _check(gpu, lambda st: [wl.wl_linear_f8(c, s, w, stream=st)], [((300, 640), BF)])


def _after(st, gpu, outs):
    """The outputs in fp32, once the stream is through."""
    torch.cuda.synchronize(gpu)
    return [t.float() for t in outs]


def test_verify_and_plan_on_another_stream(wl, gpu):
    a, t, u, _ = (None if v is None else v.to(gpu) for v in _drafts(64, 5, 3001, 3, sigma=5.0))
    _check(gpu, lambda st: wl.wl_verify(a, t, u, stream=st), [((64, 5), torch.int32), ((64,), torch.int32), ((64,), torch.int32)])
    i32 = dict(dtype=torch.int32, device=gpu)

    def plan(st):
        pool = wl.PagePool.full(3000, 16, gpu)
        pages, held = torch.full((200, 20), -1, **i32), torch.zeros(200, **i32)
        length = torch.arange(200, **i32)
        torch.cuda.synchronize()
        room, slots = wl.wl_page_plan(pool, pages, held, length, 90, slots=True, stream=st)
        torch.cuda.synchronize()
        return [room, slots, pages, held]

    _check(gpu, plan, [((200,), torch.int32), ((200, 90), torch.int64)])


@pytest.mark.parametrize("T,inner,out", [(1, 1152, 20000), (40, 6912, 1152), (100, 1152, 40000), (600, 1152, 5000)])
def test_two_products_at_once(wl, gpu, T, inner, out):
    """The same call on two streams, many times over: each result is that of the call alone."""
    x, xs, w, ws = _factors(T, inner, out, 7)
    weight, x, xs = wl.F8Weight(w.to(gpu), ws.to(gpu)), x.to(gpu), xs.to(gpu)
    want = wl.wl_linear_f8(x, xs, weight)
    side = [torch.cuda.Stream(gpu) for _ in range(2)]
    torch.cuda.synchronize()
    got = [wl.wl_linear_f8(x, xs, weight, stream=side[k % 2]) for k in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert wl.wl_device_status() == wl.WL_OK


def test_two_verifications_at_once(wl, gpu):
    a, t, u, d = (v.to(gpu) for v in _drafts(12, 6, 40000, 5, BF, F32, sigma=3.0))
    want = wl.wl_verify(a, t, u, draft=d, temperature=0.7)
    side = [torch.cuda.Stream(gpu) for _ in range(3)]
    torch.cuda.synchronize()
    got = [wl.wl_verify(a, t, u, draft=d, temperature=0.7, stream=side[k % 3]) for k in range(12)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,inner,out", [(1, 144, 9741), (3, 1152, 24), (33, 400, 1160), (64, 128, 21504), (70, 272, 19336), (127, 144, 9736),
                                         (129, 256, 20008), (300, 400, 9731), (257, 1152, 5000)])
def test_product_writes_its_rows_alone(wl, gpu, T, inner, out, dt):
    """y in the middle of a buffer: what lies before and behind it stays."""
    x, xs, w, ws = _factors(T, inner, out, 3)
    pad = 4096
    buf = torch.full((2 * pad + T * out,), 7.0, dtype=dt, device=gpu)
    y = buf[pad:pad + T * out].view(T, out)
    wl.wl_linear_f8(x.to(gpu), xs.to(gpu), wl.F8Weight(w.to(gpu), ws.to(gpu)), y=y, ydt=dt)
    assert (buf[:pad] == 7.0).all() and (buf[pad + T * out:] == 7.0).all()
    want = torch.from_numpy(ref.product(x, xs, w, ws))
    assert float((y.double().cpu() - want).norm() / want.norm()) < 2 * torch.finfo(dt).eps + 1e-6


def test_small_outputs_write_their_rows_alone(wl, gpu):
    a, t, u, _ = (None if v is None else v.to(gpu) for v in _drafts(7, 3, 500, 8))
    buf = torch.full((7 * 3 + 7 + 7 + 64,), 99, dtype=torch.int32, device=gpu)
    wl.wl_verify(a, t, u, outs=(buf[8:29].view(7, 3), buf[37:44], buf[52:59]))
    for lo, hi in ((0, 8), (29, 37), (44, 52), (59, 99)):
        assert (buf[lo:hi] == 99).all()
    codes, scales = torch.full((6, 1152), 1.0, device=gpu).to(F8), torch.full((11, 4), 5.0, device=gpu)
    x = torch.randn(4, 1152, generator=gen(5)).to(gpu)
    wl.wl_quant_f8(x, outs=(codes[1:5], scales[1:10]))
    assert (codes[[0, 5]].float() == 1.0).all() and (scales[[0, 10]] == 5.0).all()


def test_a_captured_end_of_a_step(wl, gpu):
    """Quantiser, product and verification in a graph, replayed on other states and draws."""
    B, n, H, V = 3, 4, 272, 2000
    w = wl.F8Weight.quantise((torch.randn(V, H, generator=gen(1)) * 0.3).to(gpu))
    h, u = torch.zeros(B * n, H, dtype=BF, device=gpu), torch.zeros(B, n, device=gpu)
    tokens = torch.zeros(B, n, dtype=torch.int32, device=gpu)

    def step():
        logits = wl.wl_linear_f8(*wl.wl_quant_f8(h), w, ydt=F32)
        return logits, wl.wl_verify(logits, tokens, u, temperature=0.9)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        logits, res = step()
    for k in range(4):
        h.copy_(torch.randn(B * n, H, generator=gen(10 + k)).to(BF))
        u.copy_(torch.rand(B, n, generator=gen(20 + k)))
        u[:, 1:] *= 1e-3
        tokens.copy_(torch.randint(0, V, (B, n), generator=gen(30 + k)))
        g.replay()
        plain, want = step()
        assert torch.equal(logits, plain)
        assert all(torch.equal(p, q) for p, q in zip(res, want))
        exact = ref.verify(logits.cpu(), tokens.cpu(), u.cpu(), temperature=0.9)
        assert all(p.tolist() == q.tolist() for p, q in zip(res, exact))
