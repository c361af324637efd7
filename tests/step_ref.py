"""Plain 64-bit forms of the operators between a step's last states and the
next step (numpy on the host)."""
import math

import numpy as np
import torch


def quant(x, group):
    """(values of the codes, scales [ceil(in/128), ceil(rows/group)]) of x [rows, in] in 64 bits."""
    x = x.double().cpu().numpy()
    T, K = x.shape
    scales = np.ones((-(-K // 128), -(-T // group)))
    codes = np.zeros_like(x)
    for k in range(scales.shape[0]):
        for g in range(scales.shape[1]):
            at = (slice(g * group, min(T, (g + 1) * group)), slice(128 * k, min(K, 128 * (k + 1))))
            blk = x[at]
            if not np.isfinite(blk).all():
                scales[k, g] = math.nan
                continue
            top = np.abs(blk).max()
            e = -126
            if top > 0:
                while top > 448 * 2.0 ** e:
                    e += 1
                scales[k, g] = 2.0 ** e
                v = blk / 2.0 ** e
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
                codes[at] = np.round(v / step) * step
    return codes, scales


def product(x, xs, w, ws):
    """x [T, K], w [out, K] codes, xs [kb, T], ws [kb, ob] scales: y [T, out] in 64 bits."""
    x, w, xs, ws = (t.double().cpu().numpy() for t in (x, w, xs, ws))
    y = np.zeros((x.shape[0], w.shape[0]))
    for k in range(xs.shape[0]):
        at = slice(128 * k, 128 * (k + 1))
        y += (x[:, at] * xs[k][:, None]) @ (w[:, at] * np.repeat(ws[k], 128)[:w.shape[0], None]).T
    return y


def parents(mask_row, n):
    out = []
    for i in range(n):
        up = (int(mask_row[i]) & ((1 << i) - 1)) if mask_row is not None else ((1 << i) >> 1)
        out.append(up.bit_length() - 1)
    return out


def verify(logits, tokens, uniforms, mask=None, count=None, draft=None, temperature=1.0):
    """(path, accepted, next) by the definition, one sequence after another."""
    B, n = tokens.shape
    lg = logits.double().cpu().numpy()
    tk, un = tokens.cpu().numpy(), uniforms.double().cpu().numpy()
    dr = None if draft is None else draft.double().cpu().numpy()
    mk = None if mask is None else mask.cpu().numpy().view(np.uint64)
    temps = temperature.double().cpu().numpy() if isinstance(temperature, torch.Tensor) else np.full(B, float(temperature))
    V = lg.shape[1]
    path, acc, nxt = np.full((B, n), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        c = n if count is None else min(max(int(count[b]), 0), n)
        if c == 0:
            continue
        par = parents(None if mk is None else mk[b], n)
        u, way, t = 0, [0], temps[b]
        while True:
            z = lg[b * n + u]
            if not (t == t) or np.isnan(z).any() or z.max() in (math.inf, -math.inf):
                break
            kids = [i for i in range(u + 1, c) if par[i] == u]
            went = -1
            if t < 1e-6:
                best = int(z.argmax())
                went = next((i for i in kids if tk[b, i] == best), -1)
                nxt[b] = best
            else:
                w = np.exp((z - z.max()) / t)
                R = w.copy()
                for i in kids:
                    k = int(tk[b, i])
                    if 0 <= k < V:
                        S = math.fsum(R)
                        q = 1.0 if dr is None else dr[b * n + u, k]
                        if un[b, i] * q * S < R[k]:
                            went = i
                            break
                    if dr is not None:
                        R = np.maximum(R - math.fsum(R) * dr[b * n + u], 0.0)
                    elif 0 <= k < V:
                        R[k] = 0.0
                if went < 0:
                    if not R.sum() > 0:
                        R = w
                    hit = np.nonzero((R > 0) & (np.cumsum(R) > un[b, 0] * math.fsum(R)))[0]
                    nxt[b] = hit[0] if len(hit) else np.nonzero(R > 0)[0][-1]
            if went < 0:
                break
            nxt[b] = -1
            u = went
            way.append(u)
        path[b, :len(way)], acc[b] = way, len(way)
    return path, acc, nxt


def plan(free, top, page_size, pages, held, length, count, n):
    """One step of the page plan on Python lists: (stack, pages, held, room, slots)."""
    stack = [int(v) for v in free[:top]]
    pages = [[int(v) for v in r] for r in pages]
    held = [int(v) for v in held]
    B, P = len(pages), len(pages[0])
    length = [max(0, int(v)) for v in length]
    count = [n if count is None else min(max(int(count[b]), 0), n) for b in range(B)]
    need = [min(P, -(-(a + c) // page_size)) for a, c in zip(length, count)]
    gone = []
    for b in range(B):
        for j in range(need[b], held[b]):
            gone.append(pages[b][j])
            pages[b][j] = -1
        held[b] = min(held[b], need[b])
    stack += gone[::-1]
    short = False
    room, slots = [], np.full((B, n), -1, np.int64)
    for b in range(B):
        want = need[b] - held[b]
        if want > 0 and (short or want > len(stack)):
            short = True
        else:
            while held[b] < need[b]:
                pages[b][held[b]] = stack.pop()
                held[b] += 1
        room.append(max(0, min(count[b], held[b] * page_size - length[b])))
        for i in range(room[b]):
            j = length[b] + i
            slots[b, i] = pages[b][j // page_size] * page_size + j % page_size
    return stack, pages, held, room, slots
