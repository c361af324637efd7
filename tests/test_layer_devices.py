"""CPU checks of the binding: tensors of different devices, and a workspace that
is not on the GPU, are refused before anything is launched."""
import pytest
import torch

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


class _On(torch.Tensor):
    """A CPU tensor that passes for one of cuda:0 or, with `other`, of cuda:1 (checks only: nothing reads it)."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.get_device()))

    def get_device(self):
        return 0


class _Other(_On):
    def get_device(self):
        return 1


def on(*shape, dtype=BF, cls=_On):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


def _cache(wl, cls=_On):
    return wl.KVCache(on(4, 2, 16, 64, dtype=E4, cls=cls), on(4, 2, 16, 64, dtype=E4, cls=cls),
                      on(4, 2, 16, dtype=torch.float32, cls=cls), on(4, 2, 16, dtype=torch.float32, cls=cls))


def _seqs(wl, n=3, cls=_On, B=1):
    return wl.CacheSeqs(on(B, 4, dtype=torch.int32, cls=cls), on(B, dtype=torch.int32, cls=cls), n)


def _i32(*s, cls=_On):
    return on(*s, dtype=torch.int32, cls=cls)


def test_handles_hold_one_device(wl):
    with pytest.raises(ValueError, match="one device"):
        wl.CacheSeqs(_i32(1, 4), _i32(1, cls=_Other), 3)
    with pytest.raises(ValueError, match="one device"):
        wl.CacheSeqs(_i32(1, 4), _i32(1), 3, _i32(1, cls=_Other))
    with pytest.raises(ValueError, match="one device"):
        wl.KVCache(on(4, 2, 16, 64), on(4, 2, 16, 64, cls=_Other), on(4, 2, 16, dtype=torch.float32), on(4, 2, 16, dtype=torch.float32))


def test_append_refuses_other_devices(wl):
    c, s, x, o = _cache(wl), _seqs(wl), on(3, 128), on(3, 128, cls=_Other)
    for q, k, v, name in ((None, o, x, "k must"), (None, x, o, "v must"), (o, x, x, "q must")):
        with pytest.raises(ValueError, match=name + " be on cuda:0"):
            wl.wl_rope_append(q, k, v, None, None, c, s)
    with pytest.raises(ValueError, match="q_out must be on"):
        wl.wl_rope_append(x, x, x, None, None, c, s, q_out=o)
    with pytest.raises(ValueError, match="positions must be on"):
        wl.wl_rope_append(None, x, x, _i32(3, cls=_Other), None, c, s)
    with pytest.raises(ValueError, match="rotary table must be on"):
        wl.wl_rope_append(None, x, x, None, wl.RopeTable(on(8, dtype=torch.int64, cls=_Other)), c, s)
    with pytest.raises(ValueError, match="sequences must be on"):
        wl.wl_rope_append(None, x, x, None, None, c, _seqs(wl, cls=_Other))


def test_read_and_attention_refuse_other_devices(wl):
    c, s, x, o = _cache(wl), _seqs(wl), on(3, 128), on(3, 128, cls=_Other)
    kv = on(1, 3, 2, 64)
    with pytest.raises(ValueError, match="v_out must be on"):
        wl.wl_cache_read(c, s, outs=(kv, on(1, 3, 2, 64, cls=_Other)))
    with pytest.raises(ValueError, match="sequences must be on"):
        wl.wl_cache_read(c, _seqs(wl, cls=_Other), outs=(kv, kv))
    with pytest.raises(ValueError, match="q must be on"):
        wl.wl_tree_attention(o, c, s)
    with pytest.raises(ValueError, match="mask must be on"):
        wl.wl_tree_attention(x, c, s, mask=on(1, 3, dtype=torch.int64, cls=_Other))
    with pytest.raises(ValueError, match="out must be on"):
        wl.wl_tree_attention(x, c, s, out=o)
    with pytest.raises(ValueError, match="sequences must be on"):
        wl.wl_tree_attention(x, c, _seqs(wl, cls=_Other), out=x)


def test_attention_refuses_a_workspace_that_the_kernel_cannot_use(wl):
    c, s, x = _cache(wl), _seqs(wl), on(3, 128)
    nb = wl.wl_tree_attention_workspace_bytes(1, 3, 2, 2, 64)
    with pytest.raises(ValueError, match="workspace must be a CUDA"):
        wl.wl_tree_attention(x, c, s, out=x, workspace=torch.zeros(nb, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be on"):
        wl.wl_tree_attention(x, c, s, out=x, workspace=on(nb, dtype=torch.uint8, cls=_Other))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        wl.wl_tree_attention(x, c, s, out=x, workspace=on(2 * nb, dtype=torch.uint8)[::2])
    with pytest.raises(TypeError, match="workspace"):
        wl.wl_tree_attention(x, c, s, out=x, workspace=nb)


def test_norm_refuses_other_devices(wl):
    x, o = on(3, 64), on(3, 64, cls=_Other)
    w, p = on(64, dtype=torch.float32), on(64, dtype=torch.float32, cls=_Other)
    for kw, name in ((dict(y=o), "y"), (dict(gate=on(64, cls=_Other)), "gate"), (dict(w_post=p), "w_post"), (dict(w_pre=p), "w_pre"),
                     (dict(x_out=o), "x_out"), (dict(h=o), "h")):
        a = dict(y=x, x=x, w_post=w, w_pre=w, x_out=x, h=x)
        a.update(kw)
        with pytest.raises(ValueError, match=f"{name} must be on cuda:0"):
            wl.wl_norm_residual(**a)
