"""The operators between a step's last states and the next step where element
offsets pass 32 bits: the last rows of buffers of a few GB."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_step_ops import F8, _check_product, _drafts, _factors, gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_verify_rows_past_2_31_elements(wl, gpu):
    B, n, V = 64, 64, 600000
    logits = torch.empty(B * n, V, dtype=BF, device=gpu)
    assert B * n * V > 2 ** 31
    a, t, u, _ = _drafts(1, n, V, 3, BF, sigma=6.0)
    logits[-n:] = a.to(gpu)
    logits[:-n, 0] = float("nan")  # the other sequences have no distribution
    tokens, draws = torch.zeros(B, n, dtype=torch.int32, device=gpu), torch.zeros(B, n, device=gpu)
    tokens[-1], draws[-1] = t[0].to(gpu), u[0].to(gpu)
    path, acc, nxt = wl.wl_verify(logits, tokens, draws)
    want = ref.verify(a, t, u)
    assert path[-1].tolist() == want[0][0].tolist() and int(acc[-1]) == want[1][0] and int(nxt[-1]) == want[2][0]
    assert (acc[:-1] == 1).all() and (nxt[:-1] == -1).all()


def test_quant_rows_past_2_31_elements(wl, gpu):
    rows, inner = 65600, 32784
    assert rows * inner > 2 ** 31
    x = torch.empty(rows, inner, dtype=BF, device=gpu)
    last = torch.randn(3, inner, generator=gen(4)).to(BF)
    x[-3:] = last.to(gpu)
    codes, scales = wl.wl_quant_f8(x)
    want, ws = ref.quant(last, 1)
    assert np.array_equal(codes[-3:].float().double().cpu().numpy(), want)
    assert np.array_equal(scales[:, -3:].double().cpu().numpy(), ws)


@pytest.mark.parametrize("T,out", [(8200, 262144), (8200, 262145), (20, 110000000)])
def test_products_past_2_31_outputs(wl, gpu, T, out):
    """Pairs of SMs, with and without stores by boxes; few tokens and a weight of so many rows."""
    assert T * out > 2 ** 31
    x, xs, w, ws = _factors(T, 16, 128, 5)
    big = torch.empty(out, 16, dtype=F8, device=gpu)
    big.view(torch.uint8).zero_()
    big[-128:] = w.to(gpu)
    scales = torch.ones(1, -(-out // 128), device=gpu)
    y = wl.wl_linear_f8(x.to(gpu), xs.to(gpu), wl.F8Weight(big, scales))
    keep = slice(max(0, T - 200), T)
    _check_product(y[keep, -128:], x[keep], xs[:, keep], w, torch.ones(1, 1), BF)
    assert not y[keep, :-128].any()
    assert wl.wl_device_status() == wl.WL_OK
