"""CPU checks of the decoder-layer entry points: argument refusals before any
launch, the rotary table, and the binding's shape checks."""
import ctypes as C
import math

import pytest
import torch

P = 1 << 20  # a fake, aligned device address: never dereferenced here


def _cache(wl, **kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, pages=16, kv_heads=2, page_size=16, dim=128, format=0)
    a.update(kw)
    return wl._Cache(*[a[n] for n in ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "dim", "format")])


def _seqs(wl, **kw):
    a = dict(pages=P, len=P, count=P, batch=3, max_pages=4, n=2)
    a.update(kw)
    return wl._Seqs(*[a[n] for n in ("pages", "len", "count", "batch", "max_pages", "n")])


def _refused(wl, st, frag, code=None):
    msg = wl.lib().wl_last_error().decode()
    assert st == (wl.WL_ERR_INVALID_ARG if code is None else code), (st, msg)
    assert frag in msg, msg


CACHE_BAD = [
    (dict(format=2), "cache format"), (dict(dim=24), "multiple of 16"), (dict(dim=0), "multiple of 16"),
    (dict(dim=272), "multiple of 16"), (dict(pages=0), "pages"), (dict(page_size=0), "page_size"),
    (dict(kv_heads=0), "kv_heads"), (dict(k=0), "must not be NULL"), (dict(v_scale=0), "must not be NULL"),
    (dict(k=P + 8), "16-byte"), (dict(k_scale=P + 2), "4-byte"),
]
SEQS_BAD = [
    (dict(batch=0), "batch"), (dict(batch=65537), "batch"), (dict(n=0), "n must"), (dict(max_pages=0), "max_pages"),
    (dict(max_pages=1 << 30), "max_pages"), (dict(pages=0), "must not be NULL"), (dict(len=0), "must not be NULL"),
    (dict(count=P + 1), "4-byte"),
]


def _append(wl, cache=None, seqs=None, **kw):
    a = dict(q=P, k=P, v=P, q_out=P, heads=4, qs=512, ks=256, vs=256, dt=0, pos=P, rot=128, phase=P)
    a.update(kw)
    return wl.lib().wl_rope_append(a["q"], a["k"], a["v"], a["q_out"], a["heads"], a["qs"], a["ks"], a["vs"], a["dt"], a["pos"],
                                   wl._Rope(a["phase"], a["rot"], 0, 1.0), cache or _cache(wl), seqs or _seqs(wl), None)


def _read(wl, cache=None, seqs=None, ko=P, vo=P, dt=0):
    return wl.lib().wl_cache_read(cache or _cache(wl), seqs or _seqs(wl), ko, vo, dt, None)


def _attend(wl, cache=None, seqs=None, **kw):
    a = dict(q=P, heads=4, mask=P, scale=0.1, out=P, ws=P, nb=1 << 40)
    a.update(kw)
    return wl.lib().wl_tree_attention(a["q"], a["heads"], a["mask"], a["scale"], cache or _cache(wl), seqs or _seqs(wl), a["out"],
                                      a["ws"], a["nb"], None)


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_bad_caches_and_sequences(wl, call):
    for kw, frag in CACHE_BAD:
        _refused(wl, call(wl, cache=_cache(wl, **kw)), frag)
    for kw, frag in SEQS_BAD:
        _refused(wl, call(wl, seqs=_seqs(wl, **kw)), frag)


@pytest.mark.parametrize("kw,frag", [
    (dict(q=0), "both"), (dict(q_out=0), "both"), (dict(k=0), "k and v"), (dict(v=0), "k and v"), (dict(q=P + 8), "16-byte"),
    (dict(heads=3), "q_heads"), (dict(heads=0), "q_heads"), (dict(qs=516), "q_stride"), (dict(qs=504), "q_stride"),
    (dict(ks=248), "k_stride"), (dict(vs=260), "v_stride"), (dict(dt=2), "dtype"), (dict(pos=P + 2), "positions"),
    (dict(rot=7), "rot"), (dict(rot=130), "rot"), (dict(rot=-2), "rot"), (dict(phase=0), "phase"), (dict(phase=P + 4), "phase"),
])
def test_append_refusals(wl, kw, frag):
    _refused(wl, _append(wl, **kw), frag)


@pytest.mark.parametrize("kw,frag", [(dict(ko=0), "k_out"), (dict(vo=P + 8), "v_out"), (dict(dt=3), "dtype")])
def test_read_refusals(wl, kw, frag):
    _refused(wl, _read(wl, **kw), frag)


def test_attention_refusals(wl):
    for kw, frag in ((dict(q=0), "q and out"), (dict(out=P + 8), "16-byte"), (dict(heads=5), "q_heads"), (dict(mask=P + 4), "mask"),
                     (dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale")):
        _refused(wl, _attend(wl, **kw), frag)
    _refused(wl, _attend(wl, seqs=_seqs(wl, n=65)), "n must be in [1, 64]")
    _refused(wl, _attend(wl, ws=0), "workspace", wl.WL_ERR_WORKSPACE)
    _refused(wl, _attend(wl, ws=P + 128), "workspace", wl.WL_ERR_WORKSPACE)
    need = wl.wl_tree_attention_workspace_bytes(3, 2, 4, 2, 128)
    _refused(wl, _attend(wl, nb=need - 1), "too small", wl.WL_ERR_WORKSPACE)


def test_attention_workspace_sizes(wl):
    f = wl.wl_tree_attention_workspace_bytes
    assert f(3, 2, 4, 2, 128) > 0
    for bad in ((0, 2, 4, 2, 128), (3, 0, 4, 2, 128), (3, 65, 4, 2, 128), (3, 2, 5, 2, 128), (3, 2, 4, 2, 100), (3, 2, 4, 2, 272)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw,frag", [
    (dict(T=0), "T must"), (dict(H=12), "multiple of 8"), (dict(H=0), "multiple of 8"), (dict(H=16392), "multiple of 8"),
    (dict(x=0), "x must"), (dict(xo=0), "x_out"), (dict(y=0), "need y"), (dict(wpre=0), "w_pre"), (dict(gs=1151), "gate_stride"),
    (dict(gs=1156), "gate_stride"), (dict(ydt=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"),
    (dict(h=P + 4), "16-byte"), (dict(y=0, gate=0, wpost=0, xo=0, h=0), "x_out and h"),
])
def test_norm_refusals(wl, kw, frag):
    a = dict(y=P, gate=P, gs=0, x=P, wpost=P, wpre=P, xo=P, h=P, T=4, H=1152, eps=1e-6, ydt=0)
    a.update(kw)
    st = wl.lib().wl_norm_residual(a["y"], a["gate"], a["gs"], a["x"], a["wpost"], a["wpre"], a["xo"], a["h"], a["T"], a["H"], 1.0,
                                   1.0, a["eps"], 0.0, a["ydt"], 0, 0, None)
    _refused(wl, st, frag)


def test_valid_arguments_fail_at_the_cuda_step_without_a_gpu(wl):
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    for call in (_append, _read, _attend):
        assert call(wl) == wl.WL_ERR_CUDA
    assert _append(wl, q=0, q_out=0) == wl.WL_ERR_CUDA
    assert _append(wl, rot=0, phase=0, pos=0) == wl.WL_ERR_CUDA


# ------------------------------------------------------------ rotary table --
def _turns(ph):
    return [(int(p) & ((1 << 64) - 1)) / 2.0 ** 64 for p in ph]


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (256, 1e6), (6, 500.0)])
def test_plain_phases(wl, rot, base):
    ph, amp = wl.rope_phases(rot, base)
    assert amp == 1.0 and len(ph) == rot // 2
    for i, t in enumerate(_turns(ph)):
        assert t == pytest.approx(base ** (-2.0 * i / rot) / (2 * math.pi), rel=1e-14)


def test_scaled_phases(wl):
    rot, base, f = 128, 1e6, 8.0
    plain = _turns(wl.rope_phases(rot, base)[0])
    lin, amp = wl.rope_phases(rot, base, "linear", f)
    assert amp == 1.0 and all(a == pytest.approx(b / f, rel=1e-13) for a, b in zip(_turns(lin), plain))
    wide = _turns(wl.rope_phases(rot, base, "base", f)[0])
    assert wide[0] == pytest.approx(plain[0], rel=1e-13) and wide[-1] == pytest.approx(plain[-1] / f, rel=1e-11)
    ramp, amp = wl.rope_phases(rot, base, "ramp", f, 8192.0)
    assert amp == pytest.approx(0.1 * math.log(f) + 1.0, rel=1e-6)
    for t, p in zip(_turns(ramp), plain):
        turns = p * 8192
        if turns > 33 * 1.6:
            assert t == pytest.approx(p, rel=1e-13)
        elif turns < 1 / 1.6:
            assert t == pytest.approx(p / f, rel=1e-13)
        else:
            assert p / f * (1 - 1e-12) <= t <= p * (1 + 1e-12)


@pytest.mark.parametrize("args", [(3, 1e4), (-2, 1e4), (258, 1e4), (64, 1.0), (64, math.inf), (64, 1e4, "linear", 0.5),
                                  (64, 1e4, "ramp", 2.0, 0.0), (64, 1e4, "ramp", 2.0, 100.0, 1.0, 2.0)])
def test_phase_refusals(wl, args):
    with pytest.raises(wl.WLError) as e:
        wl.rope_phases(*args)
    assert e.value.status == wl.WL_ERR_INVALID_ARG


def test_phase_unknown_scaling(wl):
    with pytest.raises(ValueError, match="scaling"):
        wl.rope_phases(64, 1e4, "other")


# ---------------------------------------------------------- binding checks --
def test_binding_refuses_cpu_tensors(wl):
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        wl.KVCache(k, k, s, s)
    with pytest.raises(TypeError, match="holds"):
        wl.KVCache(k.float(), k, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        wl.CacheSeqs(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="CUDA"):
        wl.RopeTable(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        wl.wl_norm_residual(None, torch.zeros(2, 8, dtype=torch.bfloat16))


class _Fake(torch.Tensor):
    """A CPU tensor that passes for a CUDA one (shape checks only)."""
    is_cuda = property(lambda self: True)


def test_token_row_strides(wl):
    f = wl._token_rows
    mk = lambda *s: torch.zeros(*s).as_subclass(_Fake)  # noqa: E731
    assert f(mk(6, 64), "x", torch.float32, 6, 64) == 64
    assert f(mk(6, 4, 16), "x", torch.float32, 6, 64) == 64
    assert f(mk(6, 200)[:, 8:72], "x", torch.float32, 6, 64) == 200
    assert f(mk(2, 3, 10, 16)[:, :, 2:6], "x", torch.float32, 6, 64) == 160
    assert f(mk(2, 1, 10, 16)[:, :, 2:6], "x", torch.float32, 2, 64) == 160
    assert f(mk(1, 10, 16)[:, 2:6], "x", torch.float32, 1, 64) == 64
    with pytest.raises(ValueError, match="same distance"):
        f(mk(2, 4, 4, 16)[:, :3], "x", torch.float32, 6, 64)
    with pytest.raises(ValueError, match="contiguous"):
        f(mk(6, 16, 4).transpose(1, 2), "x", torch.float32, 6, 64)
    with pytest.raises(ValueError, match="rows"):
        f(mk(6, 60), "x", torch.float32, 6, 64)
    with pytest.raises(TypeError, match="must be"):
        f(mk(6, 64), "x", torch.bfloat16, 6, 64)
