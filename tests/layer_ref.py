"""Plain 64-bit references of the decoder-layer operators (test code only):
rotary positions, quantised cache rows, tree attention, norm and residual,
written from their formulas on the CPU."""
import math

import numpy as np
import torch

import wl_synth

F64 = torch.float64


def phases_of(turns):
    """uint64 phases of turns per position, as the int64 tensor the table holds."""
    ph = [int(round(math.ldexp(t, 64))) % (1 << 64) for t in turns]
    return torch.tensor([p - (1 << 64) if p >> 63 else p for p in ph], dtype=torch.int64)


def rotate(x, positions, freq, interleaved, amplitude):
    """x [tokens, heads, dim] 64 bits, freq radians per position."""
    rot = 2 * len(freq)
    ang = positions.to(F64)[:, None] * torch.tensor(freq, dtype=F64)
    co, si = amplitude * torch.cos(ang)[:, None], amplitude * torch.sin(ang)[:, None]
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out = x.clone()
    out[..., a] = x[..., a] * co - x[..., b] * si
    out[..., b] = x[..., a] * si + x[..., b] * co
    return out


def e4m3_codes(x, scale):
    """fp32 rows / power-of-two scales as e4m3 values (exact arithmetic; torch's cast rounds to nearest even)."""
    return (x.double() / scale[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def row_scale(x):
    """The smallest 2^e, e >= -126, with max|row| <= 448 * 2^e; 1 for zero rows, NaN for non-finite ones."""
    out = torch.empty(x.shape[:-1], dtype=torch.float32)
    for at in np.ndindex(*x.shape[:-1]):
        r = x[at].double()
        if not torch.isfinite(r).all():
            out[at] = math.nan
            continue
        m = float(r.abs().max())
        e = -126
        if m > 0:
            e = max(-126, math.frexp(m)[1] - 11)
            while m > 448 * 2.0 ** e:
                e += 1
        out[at] = 2.0 ** e if m > 0 else 1.0
    return out


class Paged:
    """A paged cache with its sequences: host copies and GPU objects."""

    def __init__(self, wl, dev, lens, n, kv_heads, dim, page, dtype, counts=None, seed=0, spare=2, std=1.0, extra_pages=0):
        g = wl_synth.make_generator(seed)
        B = len(lens)
        per = max(1, -(-(max(lens) + n) // page)) + extra_pages
        self.pool = B * per + spare
        self.table = torch.randperm(self.pool, generator=g)[:B * per].to(torch.int32).view(B, per).contiguous()
        shape = (self.pool, kv_heads, page, dim)
        k, v = (torch.randn(shape, generator=g) * std for _ in range(2))
        v = v * torch.exp2(torch.randint(-3, 4, shape[:3], generator=g).float())[..., None]
        if dtype == torch.float8_e4m3fn:
            self.ks, self.vs = (torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1) / 448))) for x in (k, v))
            self.k, self.v = e4m3_codes(k, self.ks), e4m3_codes(v, self.vs)
        else:
            self.ks, self.vs = torch.ones(shape[:3]), torch.ones(shape[:3])
            self.k, self.v = k.to(dtype), v.to(dtype)
        self.lens, self.counts, self.n, self.page, self.dim, self.kv, self.dev = lens, counts or [n] * B, n, page, dim, kv_heads, dev
        # what lies outside the sequences is never to be used: NaN codes and scales
        used = torch.zeros(self.pool, page, dtype=torch.bool)
        for b in range(B):
            for j in range(lens[b] + self.counts[b]):
                used[int(self.table[b, j // page]), j % page] = True
        dead = ~used[:, None].expand(-1, kv_heads, -1)
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            if dtype == torch.float8_e4m3fn:
                x.view(torch.uint8)[dead] = 0x7F
            else:
                x[dead] = math.nan
            s[dead] = math.nan
        self.upload(wl, counts)

    def upload(self, wl, counts=None):
        d = self.dev
        self.cache = wl.KVCache(self.k.to(d), self.v.to(d), self.ks.to(d), self.vs.to(d))
        i32 = dict(dtype=torch.int32, device=d)
        self.seqs = wl.CacheSeqs(self.table.to(d), torch.tensor(self.lens, **i32), self.n,
                                 None if counts is None else torch.tensor(counts, **i32))

    def at(self, b, j):
        return int(self.table[b, j // self.page]), j % self.page

    def rows(self, name, b, first, count):
        """Values [count, kv, dim] in 64 bits of positions first.. of sequence b."""
        x, s = getattr(self, name), getattr(self, name + "s")
        out = torch.zeros(count, self.kv, self.dim, dtype=F64)
        for i in range(count):
            p, t = self.at(b, first + i)
            out[i] = x[p, :, t].to(torch.float32).to(F64) * s[p, :, t].to(F64)[:, None]
        return out


def tree_masks(B, n, seed, branch=3):
    """Ancestor masks [B, n] of random trees, as int64 words."""
    rs = np.random.RandomState(seed)
    m = np.zeros((B, n), np.uint64)
    for b in range(B):
        for i in range(n):
            par = i - 1 - rs.randint(0, min(i, branch) + 1)
            m[b, i] = (m[b, par] if par >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return torch.from_numpy(m.view(np.int64).copy())


def attention(pg, q, mask, scale):
    """(out, bound): the attention in 64 bits, and how far a result may be off.

    The bound follows the number formats, not a kernel: weights held in 8
    significant bits (each off by at most 2^-8 of itself, and by 2^-22 of the
    largest), scores off by 2^-20 of sum |q||k| scale (fp32 products of at most
    256 terms), and the output's rounding to bf16 (2^-9 of itself, 2^-134 near 0)."""
    B, n = len(pg.lens), pg.n
    Hq = q.shape[2]
    G = Hq // pg.kv
    out, bound = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    for b in range(B):
        m, L = pg.counts[b], pg.lens[b]
        if m == 0:
            continue
        k, v = pg.rows("k", b, 0, L + m), pg.rows("v", b, 0, L + m)
        see = torch.ones(m, L + m, dtype=torch.bool)
        for i in range(m):
            w = (2 << i) - 1 if mask is None else int(mask[b, i]) & ((1 << 64) - 1)
            for j in range(m):
                see[i, L + j] = bool((w >> j) & 1)
        for h in range(Hq):
            kk, vv, qq = k[:, h // G], v[:, h // G], q[b, :m, h].to(F64)
            for i in range(m):
                idx = see[i]
                if not idx.any():
                    continue
                s = (kk[idx] @ qq[i]) * scale
                p = torch.softmax(s, 0)
                o = p @ vv[idx]
                out[b, i, h] = o
                ds = float(((kk[idx].abs() @ qq[i].abs()) * abs(scale)).max()) * 2.0 ** -20
                av = vv[idx].abs()
                bound[b, i, h] = (2.0 ** -8 + 4 * ds) * (p @ av) + 2.0 ** -22 * (p[:, None] * av).max(0).values * int(idx.sum()) \
                    + 2.0 ** -8 * o.abs() + 2.0 ** -133
    return out, bound


def norm_residual(y, x, w_post, w_pre, gate, alpha, beta, eps, off):
    """(x', h, slack of x', slack of h) in 64 bits.

    Slack: fp32 sums of up to 64 squares a thread and 40 joins (2^-18 of the
    result of a norm at most), a few fp32 roundings of each term."""
    x = x.to(F64)
    u = torch.zeros_like(x)
    if y is not None:
        u = y.to(F64)
        if w_post is not None:
            u = u / (u.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (off + w_post.to(F64))
        if gate is not None:
            u = u * gate.to(F64)
    xp = alpha * x + beta * u
    sx = 2.0 ** -18 * ((alpha * x).abs() + (beta * u).abs())
    if w_pre is None:
        return xp, None, sx, None
    r = 1 / (xp.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    w = off + w_pre.to(F64)
    h = xp * r * w
    # an error of x' moves h directly and through the mean square
    sh = sx * r * w.abs() + h.abs() * ((sx * xp.abs()).sum(-1, keepdim=True) / xp.pow(2).sum(-1, keepdim=True).clamp(min=1e-300) + 2.0 ** -18)
    return xp, h, sx, sh


def bf16_slack(v):
    """Half a bf16 step at each value of v (64 bits)."""
    e = torch.frexp(v)[1].clamp(min=-125)
    return torch.ldexp(torch.ones_like(v), e - 9)
