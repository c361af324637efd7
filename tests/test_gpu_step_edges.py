"""Operators between a step's last states and the next step: clusters under load,
starved sequences, decisions near a border, scales at the ends of fp32."""
import numpy as np
import pytest
import torch

from tests import step_ref as ref

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
