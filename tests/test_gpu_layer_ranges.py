"""Inputs of very different sizes side by side, in the decoder-layer operators:
what is said of one row must not come from another."""
import pytest
import torch

import wl_synth
from tests.test_gpu_attention_units import check, filled

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
