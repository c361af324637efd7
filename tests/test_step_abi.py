"""CPU checks of the operators between a step's last states and the next step:
refusals before any launch, by the library and by the binding."""
import math

import pytest
import torch

from tests.test_layer_devices import _On, _Other, on

P = 1 << 20  # a fake, aligned device address: never dereferenced here
BF, F32, I32, I64, F8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


def _quant(wl, **kw):
    a = dict(x=P, stride=1152, dt=0, rows=4, inp=1152, group=1, codes=P, scales=P)
    a.update(kw)
    return wl.lib().wl_quant_f8(*[a[n] for n in ("x", "stride", "dt", "rows", "inp", "group", "codes", "scales")], None)


def _linear(wl, **kw):
    a = dict(x=P, xs=P, W=P, ws=P, y=P, T=4, inp=1152, out=100, dt=0)
    a.update(kw)
    return wl.lib().wl_linear_f8(*[a[n] for n in ("x", "xs", "W", "ws", "y", "T", "inp", "out", "dt")], None)


def _verify(wl, **kw):
    a = dict(logits=P, ls=1000, ldt=0, draft=P, ds=1000, ddt=1, tokens=P, u=P, mask=P, count=P, temps=0, temp=1.0, batch=3, n=4, vocab=1000,
             path=P, acc=P, next=P)
    a.update(kw)
    return wl.lib().wl_verify(*[a[n] for n in ("logits", "ls", "ldt", "draft", "ds", "ddt", "tokens", "u", "mask", "count", "temps", "temp", "batch", "n",
                                               "vocab", "path", "acc", "next")], None)


def _plan(wl, **kw):
    a = dict(free=P, top=P, pool=100, page=16, pages=P, held=P, len=P, count=P, batch=3, per=8, n=4, room=P, slots=P)
    a.update(kw)
    return wl.lib().wl_page_plan(*[a[n] for n in ("free", "top", "pool", "page", "pages", "held", "len", "count", "batch", "per", "n", "room", "slots")],
                                 None)


BAD = {
    _quant: [(dict(dt=2), "dtype"), (dict(rows=0), "rows"), (dict(rows=(1 << 30) + 1), "rows"), (dict(inp=1160), "multiple of 16"), (dict(inp=0), "multiple of 16"),
             (dict(inp=(1 << 20) + 16), "multiple of 16"), (dict(group=64), "group"), (dict(group=0), "group"), (dict(stride=1144), "x_stride"),
             (dict(stride=1156), "x_stride"), (dict(x=0), "NULL"), (dict(codes=0), "NULL"), (dict(scales=0), "NULL"), (dict(x=P + 8), "16-byte"),
             (dict(codes=P + 8), "16-byte"), (dict(scales=P + 2), "4-byte")],
    _linear: [(dict(dt=2), "dtype"), (dict(T=0), "T must"), (dict(out=0), "out must"), (dict(inp=8), "multiple of 16"), (dict(inp=24), "multiple of 16"),
              (dict(x=0), "NULL"), (dict(xs=0), "NULL"), (dict(W=0), "NULL"), (dict(ws=0), "NULL"), (dict(y=0), "NULL"), (dict(W=P + 8), "16-byte"),
              (dict(y=P + 4), "16-byte"), (dict(xs=P + 2), "4-byte")],
    _verify: [(dict(ldt=2), "dtype 2"), (dict(ddt=3), "dtype 3"), (dict(batch=0), "batch"), (dict(batch=65537), "batch"), (dict(n=0), "n must"),
              (dict(n=65), "n must"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 24) + 1), "vocab"), (dict(logits=0), "NULL"), (dict(tokens=0), "NULL"),
              (dict(u=0), "NULL"), (dict(path=0), "NULL"), (dict(acc=0), "NULL"), (dict(next=0), "NULL"), (dict(ls=999), "stride"), (dict(ds=999), "stride"),
              (dict(logits=P + 1), "elements"), (dict(draft=P + 2), "elements"), (dict(mask=P + 4), "8-byte"), (dict(tokens=P + 2), "4-byte"),
              (dict(temps=P + 2), "4-byte"), (dict(temp=-0.5), "temperature"), (dict(temp=math.nan), "temperature"), (dict(temp=math.inf), "temperature")],
    _plan: [(dict(pool=0), "pool_pages"), (dict(pool=1 << 30), "pool_pages"), (dict(page=0), "page_size"), (dict(page=(1 << 20) + 1), "page_size"),
            (dict(batch=0), "batch"), (dict(batch=65537), "batch"), (dict(n=-1), "n must"), (dict(n=1 << 30), "n must"), (dict(per=0), "max_pages"),
            (dict(per=1 << 27), "max_pages"), (dict(page=1, per=1 << 29), "batch * max_pages"), (dict(free=0), "NULL"), (dict(top=0), "NULL"),
            (dict(pages=0), "NULL"), (dict(held=0), "NULL"), (dict(len=0), "NULL"), (dict(room=0), "NULL"), (dict(slots=P + 4), "8-byte"),
            (dict(count=P + 2), "4-byte")],
}


@pytest.mark.parametrize("call", list(BAD))
def test_refusals(wl, call):
    for kw, frag in BAD[call]:
        st = call(wl, **kw)
        msg = wl.wl_last_error()
        assert st == wl.WL_ERR_INVALID_ARG and frag in msg, (kw, st, msg)


def test_valid_arguments_fail_at_the_cuda_step_without_a_gpu(wl):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    for call in BAD:
        assert call(wl) == wl.WL_ERR_CUDA
    for kw in (dict(draft=0, ds=0), dict(mask=0, count=0), dict(temps=P, temp=math.nan), dict(temp=0.0)):
        assert _verify(wl, **kw) == wl.WL_ERR_CUDA
    for kw in (dict(n=0, slots=0), dict(count=0), dict(slots=0)):
        assert _plan(wl, **kw) == wl.WL_ERR_CUDA


def z(*shape, dtype=F32, cls=_On):
    return on(*shape, dtype=dtype, cls=cls)


def test_binding_refuses_types_shapes_and_devices(wl):
    x = z(4, 32, dtype=BF)
    with pytest.raises(ValueError, match="x must be a tensor"):
        wl.wl_quant_f8(z(32))
    with pytest.raises(ValueError, match="CUDA"):
        wl.wl_quant_f8(torch.zeros(4, 32), outs=(z(4, 32, dtype=F8), z(1, 4)))
    with pytest.raises(ValueError, match="dtype"):
        wl.wl_quant_f8(z(4, 32, dtype=I32))
    with pytest.raises(ValueError, match="row must be contiguous"):
        wl.wl_quant_f8(z(32, 4).t(), outs=(z(4, 32, dtype=F8), z(1, 4)))
    with pytest.raises(ValueError, match="scales must have shape"):
        wl.wl_quant_f8(x, outs=(z(4, 32, dtype=F8), z(4, 1)))
    with pytest.raises(ValueError, match="codes must be on cuda:0"):
        wl.wl_quant_f8(x, outs=(z(4, 32, dtype=F8, cls=_Other), z(1, 4)))
    with pytest.raises(TypeError, match="codes must be"):
        wl.F8Weight(z(8, 32), z(1, 1))
    with pytest.raises(ValueError, match="scales must have shape"):
        wl.F8Weight(z(200, 32, dtype=F8), z(2, 1))
    with pytest.raises(ValueError, match="one device"):
        wl.F8Weight(z(8, 32, dtype=F8), z(1, 1, cls=_Other))
    w = wl.F8Weight(z(200, 160, dtype=F8), z(2, 2))
    c, s = z(3, 160, dtype=F8), z(2, 3)
    for kw, err in ((dict(codes=z(3, 128, dtype=F8)), "codes must have shape"), (dict(scales=z(3, 2)), "scales must have shape"),
                    (dict(codes=z(3, 160, dtype=F8, cls=_Other)), "codes must be on"), (dict(scales=z(2, 3, cls=_Other)), "scales must be on"),
                    (dict(y=z(3, 200)), "y must be"), (dict(y=z(3, 200, dtype=BF, cls=_Other)), "y must be on"), (dict(ydt=I32), "dtype")):
        a = dict(codes=c, scales=s, weight=w)
        a.update(kw)
        with pytest.raises((ValueError, TypeError), match=err):
            wl.wl_linear_f8(**a)


def test_binding_refuses_verification_arguments(wl):
    good = dict(logits=z(6, 50), tokens=z(2, 3, dtype=I32), uniforms=z(2, 3), mask=z(2, 3, dtype=I64), count=z(2, dtype=I32), draft=z(6, 50, dtype=BF),
                temperature=z(2))
    for kw, err in ((dict(tokens=z(6, dtype=I32)), "tokens must be a tensor"), (dict(tokens=z(2, 3, dtype=I64)), "tokens must be"),
                    (dict(logits=z(5, 50)), "logits must have shape"), (dict(logits=z(6, 50, cls=_Other)), "logits must be on"),
                    (dict(logits=z(50, 6).t()), "logits: each row"), (dict(uniforms=z(3, 2)), "uniforms must have shape"),
                    (dict(uniforms=z(2, 3, dtype=torch.float64)), "uniforms must be"), (dict(mask=z(2, 3, dtype=I32)), "mask must be"),
                    (dict(count=z(3, dtype=I32)), "count must have"), (dict(draft=z(6, 49)), "draft must have shape"),
                    (dict(draft=z(6, 50, cls=_Other)), "draft must be on"), (dict(draft=3), "draft must be"), (dict(temperature=z(3)), "temperature must have"),
                    (dict(temperature=z(2, cls=_Other)), "temperature must be on"),
                    (dict(outs=(z(2, 3, dtype=I32), z(2, dtype=I32), z(3, dtype=I32))), "next must have shape")):
        a = dict(good)
        a.update(kw)
        with pytest.raises((ValueError, TypeError), match=err):
            wl.wl_verify(**a)


def test_binding_refuses_plan_arguments(wl):
    with pytest.raises(ValueError, match="free must be"):
        wl.PagePool(z(4, 4, dtype=I32), z(1, dtype=I32), 16)
    with pytest.raises(ValueError, match="top must have"):
        wl.PagePool(z(4, dtype=I32), z(2, dtype=I32), 16)
    with pytest.raises(ValueError, match="one device"):
        wl.PagePool(z(4, dtype=I32), z(1, dtype=I32, cls=_Other), 16)
    good = dict(pool=wl.PagePool(z(9, dtype=I32), z(1, dtype=I32), 16), pages=z(2, 4, dtype=I32), held=z(2, dtype=I32), len=z(2, dtype=I32), n=3,
                count=z(2, dtype=I32), room=z(2, dtype=I32))
    for kw, err in ((dict(pages=z(8, dtype=I32)), "pages must be a tensor"), (dict(pages=z(2, 4)), "pages must be"),
                    (dict(pages=z(2, 4, dtype=I32, cls=_Other)), "pages must be on"), (dict(held=z(3, dtype=I32)), "held must have"),
                    (dict(len=z(2, dtype=I64)), "len must be"), (dict(count=z(1, dtype=I32)), "count must have"),
                    (dict(room=z(3, dtype=I32)), "room must have"), (dict(slots=z(2, 3, dtype=I32)), "slots must be"),
                    (dict(slots=z(2, 4, dtype=I64)), "slots must have")):
        a = dict(good)
        a.update(kw)
        with pytest.raises((ValueError, TypeError), match=err):
            wl.wl_page_plan(**a)
