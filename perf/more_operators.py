"""Cases of the operators between a step's last states and the next step.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, or 64 where sums and borders need them) or, where ``own`` is true, by
the framework's calls.  ``exact`` gives the same from the definition in 64 bits.

Operators (case["op"]):
  quantise  rows or weights as 8-bit floats with a scale for each block of 128
  product   8-bit product of quantised rows and a quantised weight
  verify    drafted tokens accepted or rejected, and the next token, from given random numbers
  plan      pages taken and given back as sequences grow and shrink, and the slots of their new tokens
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the last state of one sequence (hidden 1152) on its way to the vocabulary: latency
        dict(name="quantise one token", op="quantise", rows=1, inner=1152, group=1, x="bf16"),
        # a prompt of the large set before a projection
        dict(name="quantise prompt", op="quantise", rows=4096, inner=5376, group=1, x="bf16"),
        # logits of one token: the weight's bytes
        dict(name="head one token", op="product", rows=1, inner=1152, outer=262144, y="f32"),
        # logits of a batch's drafted tokens: weight and logits
        dict(name="head drafted tokens", op="product", rows=96, inner=1152, outer=262144, y="bf16"),
        # few tokens, a long sum and an odd, small output: latency
        dict(name="projection odd", op="product", rows=37, inner=6912, outer=1153, y="f32"),
        # a prompt of the large set: compute
        dict(name="projection prompt", op="product", rows=4096, inner=5376, outer=21504, y="bf16"),
        # plain sampling of one sequence: latency
        dict(name="sample one token", op="verify", batch=1, n=1, vocab=262144, logits="f32", draft="none", temp=1.0, tree=False),
        # widest trees of a few sequences, greedy, odd vocabulary
        dict(name="verify wide trees greedily", op="verify", batch=4, n=61, vocab=100003, logits="f32", draft="none", temp=0.0,
             tree=True),
        # drafted chains with the drafter's distribution
        dict(name="verify chains", op="verify", batch=16, n=8, vocab=262144, logits="bf16", draft="f32", temp=0.8, tree=False),
        # a full batch's drafted trees, drafts without a distribution
        dict(name="verify trees", op="verify", batch=32, n=24, vocab=262144, logits="bf16", draft="none", temp=0.8, tree=True),
        # one sequence crosses into a new page and, its draft rejected, back: latency
        dict(name="plan one sequence", op="plan", batch=1, n=8, page=64, len=1020, churn=0),
        # prompts come in while other requests end
        dict(name="plan prompts", op="plan", batch=512, n=4096, page=16, len=8000, churn=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "verify", "verify", "verify", "plan"])
    if op == "quantise":
        inner = 16 * _log(rng, 1, 1344)
        return dict(op=op, rows=_log(rng, 1, max(2, min(8192, 4096 * 5376 // inner))), inner=inner, group=rng.choice([1, 1, 128]),
                    x=rng.choice(["bf16", "f32"]))
    if op == "product":
        inner, rows = 16 * _log(rng, 4, 1344), _log(rng, 1, 4096)
        most = min(300e6 / inner, 1e8 / rows, 4.0e11 / (inner * rows), 262144)
        return dict(op=op, rows=rows, inner=inner, outer=_log(rng, 8, max(16, most)), y=rng.choice(["bf16", "f32"]))
    if op == "verify":
        batch, vocab = _log(rng, 1, 64), _log(rng, 1000, 262144)
        draft = rng.choice(["none", "none", "f32", "bf16"])
        most = max(1, min(64, 32 * 24 * 262144 // (2 * batch * vocab)))
        return dict(op=op, batch=batch, n=_log(rng, 1, most), vocab=vocab, logits=rng.choice(["bf16", "f32"]), draft=draft,
                    temp=rng.choice([0.0] * (draft == "none") + [0.6, 0.8, 1.0, 1.25]), tree=draft == "none" and rng.random() < 0.7)
    batch = _log(rng, 1, 1000)
    return dict(op=op, batch=batch, n=_log(rng, 1, max(1, min(4096, 2000000 // batch))), page=rng.choice([1, 16, 32, 48, 64, 128]),
                len=_log(rng, 1, max(2, min(20000, 8000000 // batch))) - 1, churn=rng.choice([0, 0, 2, 3, 5]))


# ------------------------------------------------- what a case's data are --
# Trees, accepted lengths and request lengths are a case's own: a pass's work does not depend on the seed.
def _parents(c):
    """Parent of each node [batch][n]; a chain, or a tree whose nodes have up to four children."""
    out = []
    for b in range(c["batch"]):
        rs = np.random.RandomState(b + 1)
        p = [-1]
        for i in range(1, c["n"]):
            free = [j for j in range(max(0, i - 6), i) if p.count(j) < 4]
            p.append(int(free[rs.randint(len(free))]) if c["tree"] else i - 1)
        out.append(p)
    return out


def _way(c, b, parent):
    """The nodes that sequence b's draws accept: two thirds of the way down, on average, through changing children."""
    n, node, path = c["n"], 0, [0]
    stop = (5 * b + 2) % 6
    while True:
        kids = [i for i in range(1, n) if parent[i] == node]
        if not kids or len(path) > 1 + stop:
            return path
        node = kids[(b + len(path)) % len(kids)] if c["temp"] > 0 else kids[0]
        path.append(node)


def _requests(c):
    """(lengths before, lengths of the step, new tokens) of each sequence; of every `churn`, one ends and one begins."""
    before, after, count = [], [], []
    for b in range(c["batch"]):
        old = c["len"] - (b * c["len"]) // (2 * c["batch"])
        ends, begins = c["churn"] and b % c["churn"] == 0, c["churn"] and b % c["churn"] == 1
        before.append(0 if begins else old)
        after.append(0 if ends or begins else old)
        count.append(0 if ends else max(1, c["n"] - (b % 4) * c["n"] // 8))
    return before, after, count


# ---------------------------------------------------------------- prepare --
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    s = {"case": dict(c)}
    if c["op"] == "quantise":
        x = randn(c["rows"], c["inner"])
        s["x"] = (x * torch.exp(randn(c["rows"], 1))).to(_DT[c["x"]])
    elif c["op"] == "product":
        T, K, N = c["rows"], c["inner"], c["outer"]
        kb, ob = -(-K // 128), -(-N // 128)
        s["x"] = (randn(T, K) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["w"] = (randn(N, K) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["x_scale"] = torch.exp2(torch.floor(randn(kb, T)) - 8)  # powers of two, as the quantiser gives
        s["w_scale"] = torch.exp(0.3 * randn(kb, ob)) / (100 * math.sqrt(K))  # any, as checkpoints hold
        if own:
            import rank_weight_reconstruction_wl_gb300 as wl

            s["weight"] = wl.F8Weight(s["w"], s["w_scale"])
    elif c["op"] == "verify":
        _prepare_verify(s, c, g, randn, rand)
    else:
        before, after, count = _requests(c)
        B, page = c["batch"], c["page"]
        held = [-(-v // page) for v in before]
        per = max(1, max(max(held), max(-(-(a + n) // page) for a, n in zip(after, count))))
        pool = sum(max(h, -(-(a + n) // page)) for h, a, n in zip(held, after, count)) + 1009
        ids = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        at = np.concatenate(([0], np.cumsum(held)))
        idx = np.full((B, per), -1, np.int64)
        for b in range(B):
            idx[b, :held[b]] = np.arange(at[b], at[b + 1])
        idx = torch.from_numpy(idx).to(dev)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        s.update(pages=torch.where(idx < 0, -1, ids[idx.clamp(min=0)]).to(torch.int32).contiguous(), held=i32(held),
                 before=i32(before), after=i32(after), count=i32(count), top=i32([pool - int(at[-1])]),
                 free=torch.cat((ids[int(at[-1]):], torch.full((int(at[-1]),), -1, dtype=torch.int32, device=dev))))
        if own:
            import rank_weight_reconstruction_wl_gb300 as wl

            s["pool"] = wl.PagePool(s["free"], s["top"], page)
    return s


def _prepare_verify(s, c, g, randn, rand):
    """Logits of the drafted nodes; tokens and draws as a drafter and a random generator give them where the path of
    _way() is the one accepted (an accepted token of a draft q is spread like min(p, q), a rejected one like max(q - p, 0))."""
    B, n, V, dev = c["batch"], c["n"], c["vocab"], torch.device("cuda")
    parents = _parents(c)
    ways = [_way(c, b, parents[b]) for b in range(B)]
    s["logits"] = torch.empty(B * n, V, dtype=_DT[c["logits"]], device=dev)
    drafted = c["draft"] != "none"
    if drafted:
        s["draft"] = torch.zeros(B * n, V, dtype=_DT[c["draft"]], device=dev)
    s["tokens"] = torch.zeros(B, n, dtype=torch.int32, device=dev)
    u = rand(B, n)
    temp = c["temp"] if c["temp"] > 0 else 1.0
    ramp = -1.2 * torch.log(torch.arange(1, V + 1, device=dev, dtype=torch.float32))
    for b in range(B):
        near = ramp[torch.randperm(V, generator=g, device=dev)]
        l = (near + 1.5 * randn(n, V)).to(_DT[c["logits"]])  # the contexts of one sequence share some of their likely tokens
        s["logits"][b * n:(b + 1) * n] = l
        accepted = torch.tensor([i in ways[b] for i in range(n)], device=dev)
        if n == 1:
            continue
        par = torch.tensor(parents[b][1:], device=dev)
        if drafted:
            p = torch.softmax(l.float() / temp, -1)
            q = torch.softmax((l.float() + 0.7 * randn(n, V)) / temp, -1).to(_DT[c["draft"]])
            s["draft"][b * n:(b + 1) * n] = q
            pp, qq = p[par], q.float()[par]
            t = torch.multinomial(torch.where(accepted[1:, None], torch.minimum(pp, qq), (qq - pp).clamp(min=0)), 1, generator=g)
            ratio = (pp.gather(1, t) / qq.gather(1, t)).clamp(max=1)[:, 0]
            u[b, 1:] = torch.where(accepted[1:], u[b, 1:] * ratio, ratio + (1 - ratio) * u[b, 1:])
        else:
            # the drafter's best tokens of the parent, best first; greedy: the target's own best where accepted
            best = torch.topk(l.float() if c["temp"] == 0 else l.float() + 0.5 * randn(n, V), 6, -1).indices
            place = torch.tensor([sum(parents[b][j] == parents[b][i] for j in range(1, i)) for i in range(1, n)], device=dev)
            if c["temp"] == 0:
                place = torch.where(accepted[1:], 0, place + 1)
            t = best[par].gather(1, place[:, None])
            p = torch.softmax(l.double() / temp, -1)[par].gather(1, t)[:, 0]
            gone = ((par[:, None] == par[None]).double().tril(-1) * p[None]).sum(1)  # the mass of the siblings tried before
            ratio = (p / (1 - gone)).clamp(max=1).float()
            u[b, 1:] = torch.where(accepted[1:], u[b, 1:] * ratio, ratio + (1 - ratio) * u[b, 1:])
        s["tokens"][b, 1:] = t[:, 0].to(torch.int32)
    s["uniforms"] = u.clamp(max=1 - 2.0 ** -24).contiguous()
    m = np.zeros((B, n), np.uint64)
    for b in range(B):
        for i in range(n):
            m[b, i] = (m[b, parents[b][i]] if i else np.uint64(0)) | np.uint64(1 << i)
    s["mask"] = torch.from_numpy(m.view(np.int64)).to(dev)  # bit j of row i: node j is node i or an ancestor of it
    s["parent"] = torch.tensor(parents, device=dev)


# ------------------------------------------------------------ plain forms --
def _plain_quantise(s, c):
    T, K, G = c["rows"], c["inner"], c["group"]
    tb, kb = -(-T // G), -(-K // 128)
    x = torch.nn.functional.pad(s["x"].float(), (0, kb * 128 - K, 0, tb * G - T)).view(tb, G, kb, 128)
    amax = x.abs().amax((1, 3))
    m, e = torch.frexp(amax)  # 448 is 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    sc = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    codes = (x / sc[:, None, :, None]).view(tb * G, kb * 128)[:T, :K].to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": sc.t().contiguous()}


def _plain_product(s, c):
    K, N = c["inner"], c["outer"]
    x = s["x"].float() * s["x_scale"].t().repeat_interleave(128, 1)[:, :K]
    w = s["w"].float() * s["w_scale"].t().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return torch.matmul(x, w.t()).to(_DT[c["y"]])


def _plain_verify(s, c):
    B, n, V = c["batch"], c["n"], c["vocab"]
    dev = s["tokens"].device
    logits = s["logits"].view(B, n, V)
    seq, node = torch.arange(B, device=dev), torch.arange(n, device=dev)
    at, level = (torch.zeros(B, dtype=torch.int64, device=dev) for _ in range(2))
    path = torch.full((B, n), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    tokens, draws, over = s["tokens"].long(), s["uniforms"].double(), s["parent"].clamp(min=0)
    best = logits.argmax(-1)  # the first of equal ones
    if c["temp"] == 0:
        for i in range(1, n):
            go = (s["parent"][:, i] == at) & (tokens[:, i] == best[seq, at])
            level = level + go
            at = torch.where(go, node[i], at)
            path[seq, level] = at.to(torch.int32)
        return {"path": path, "accepted": (level + 1).to(torch.int32), "next": best[seq, at].to(torch.int32)}
    # weights in 64 bits: the borders between tokens are closer than 32 bits hold
    top = logits.gather(2, best[..., None]).double()
    total = torch.exp((logits.double() - top) / c["temp"]).sum(-1)
    mine = torch.exp((logits[seq[:, None], over, tokens].double() - top[seq[:, None], over, 0]) / c["temp"])
    if "draft" in s:  # a chain: accepted up to the first rejection
        draft = s["draft"].view(B, n, V)
        go = draws * draft[seq[:, None], over, tokens].double() * total.gather(1, over) < mine
        level = go[:, 1:].long().cumprod(1).sum(1)
        at, path = level, torch.where(node <= level[:, None], node, -1).to(torch.int32)
        R = torch.exp((logits[seq, at].double() - top[seq, at]) / c["temp"])
        left = (R - total[seq, at][:, None] * draft[seq, at].double()).clamp(min=0)
        R = torch.where(((at < n - 1) & (left > 0).any(-1))[:, None], left, R)
    else:  # siblings' tokens differ
        gone, S = torch.zeros(B, n, dtype=torch.bool, device=dev), total[:, 0]
        for i in range(1, n):
            child = s["parent"][:, i] == at
            go = child & (draws[:, i] * S < mine[:, i])
            gone[:, i] = child & ~go
            level = level + go
            at = torch.where(go, node[i], at)
            path[seq, level] = at.to(torch.int32)
            S = torch.where(go, total[seq, at], torch.where(child, S - mine[:, i], S))
        R = torch.exp((logits[seq, at].double() - top[seq, at]) / c["temp"])
        gone = gone & (s["parent"] == at[:, None])
        R = R * torch.ones_like(R).scatter_reduce(1, tokens, (~gone).double(), "prod")
    upto = R.cumsum(-1)
    hit = (R > 0) & (upto > (draws[:, 0] * R.sum(-1))[:, None])
    first = torch.where(hit.any(-1), hit.byte().argmax(-1), V - 1 - (R > 0).flip(-1).byte().argmax(-1))
    return {"path": path, "accepted": (level + 1).to(torch.int32), "next": first.to(torch.int32)}


def _plain_plan(s, c, length, count):
    """One step of the plan in the state's buffers; the room of each sequence and the slots of its new tokens."""
    pages, held, free, top, page = s["pages"], s["held"], s["free"], s["top"], c["page"]
    B, P = pages.shape
    j = torch.arange(P, device=pages.device)
    need = torch.div(length + count + page - 1, page, rounding_mode="floor").clamp(max=P).long()
    have = held.long()
    back = (j >= need[:, None]) & (j < have[:, None])
    n_back = back.sum()
    k = torch.where(back, back.view(-1).long().cumsum(0).view(B, P) - 1, -1)
    spot = torch.where(back, top.long() + n_back - 1 - k, free.numel())  # the first page given back ends on top
    free.copy_(torch.cat((free, free[:1])).scatter(0, spot.view(-1), pages.view(-1))[:-1])
    up = top.long() + n_back
    want = (need - have).clamp(min=0)
    fits = (want.cumsum(0) <= up) & (want > 0)
    want = torch.where(fits, want, 0)
    first = want.cumsum(0) - want
    take = fits[:, None] & (j >= have[:, None]) & (j < need[:, None])
    at = (up - 1 - (first[:, None] + j - have[:, None])).clamp(0, free.numel() - 1)
    pages.copy_(torch.where(take, free[at], torch.where(back, -1, pages)))
    now = torch.where(fits, need, torch.minimum(have, need))
    held.copy_(now)
    top.copy_(up - want.sum())
    room = torch.minimum(now * page - length, count.long()).clamp(min=0)
    i = torch.arange(c["n"], device=pages.device)
    p = length[:, None].long() + i
    g = pages.long().gather(1, torch.div(p, page, rounding_mode="floor").clamp(max=P - 1))
    return room.to(torch.int32), torch.where(i < room[:, None], g * page + p % page, -1)


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "plan":
            # the step's pages, and back to the lengths before it
            room, slots = _plain_plan(s, c, s["after"], s["count"])
            _plain_plan(s, c, s["before"], torch.zeros_like(s["count"]))
            return {"room": room, "slots": slots, "pages": s["pages"], "held": s["held"], "top": s["top"]}
        return {"quantise": _plain_quantise, "product": _plain_product, "verify": _plain_verify}[c["op"]](s, c)
    import rank_weight_reconstruction_wl_gb300 as wl

    if c["op"] == "quantise":
        codes, scales = wl.wl_quant_f8(s["x"], group=c["group"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "product":
        return wl.wl_linear_f8(s["x"], s["x_scale"], s["weight"], ydt=_DT[c["y"]])
    if c["op"] == "verify":
        path, accepted, token = wl.wl_verify(s["logits"], s["tokens"], s["uniforms"], mask=s["mask"] if c["tree"] else None,
                                             draft=s.get("draft"), temperature=c["temp"])
        return {"path": path, "accepted": accepted, "next": token}
    room, slots = wl.wl_page_plan(s["pool"], s["pages"], s["held"], s["after"], c["n"], s["count"], slots=True)
    wl.wl_page_plan(s["pool"], s["pages"], s["held"], s["before"])
    return {"room": room, "slots": slots, "pages": s["pages"], "held": s["held"], "top": s["top"]}


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] == "quantise":
        n = c["rows"] * c["inner"]
        return {"bytes": n * (size[c["x"]] + 1) + 4 * -(-c["rows"] // c["group"]) * -(-c["inner"] // 128), "flops": 2 * n}
    if c["op"] == "product":
        T, K, N = c["rows"], c["inner"], c["outer"]
        kb = -(-K // 128)
        return {"bytes": (T + N) * K + T * N * size[c["y"]] + 4 * kb * (T + -(-N // 128)), "flops": 2 * T * K * N}
    if c["op"] == "verify":
        rows = tried = 0  # logits rows of the accepted nodes, draft rows where a child was rejected
        for b, parent in enumerate(_parents(c)):
            way = _way(c, b, parent)
            rows += len(way)
            tried += way[-1] in parent
        V = c["vocab"]
        per = 4 + 4 + (8 if c["tree"] else 0) + 4
        return {"bytes": rows * V * size[c["logits"]] + tried * V * size[c["draft"]] + c["batch"] * (c["n"] * per + 8),
                "flops": 4 * rows * V + 3 * tried * V * (c["draft"] != "none")}
    before, after, count = _requests(c)
    moved = sum(abs(-(-(a + n) // c["page"]) - -(-o // c["page"])) for o, a, n in zip(before, after, count))
    return {"bytes": 2 * (8 * moved + 16 * c["batch"]) + 8 * c["batch"] * c["n"] + 4 * c["batch"], "flops": 2 * c["batch"] * c["n"]}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    c = case
    f64 = torch.float64
    s = prepare(case, seed)
    if c["op"] == "quantise":
        T, K, G = c["rows"], c["inner"], c["group"]
        codes = torch.empty(T, K, dtype=f64, device="cuda")
        scales = torch.empty(-(-K // 128), -(-T // G), dtype=f64, device="cuda")
        for k in range(scales.shape[0]):
            x = s["x"][:, 128 * k:128 * (k + 1)].to(f64)
            top = x.abs().amax(1)
            top = torch.stack([t.amax() for t in top.split(G)]) if G > 1 else top
            sc = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -110))) - 10)  # too small by up to four times
            for _ in range(3):
                sc = torch.where(top > 448 * sc, 2 * sc, sc)
            sc = torch.where(top > 0, sc, 1.0)
            scales[k] = sc
            v = x / sc.repeat_interleave(G)[:T, None]
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)  # e4m3: 3 bits after the first
            codes[:, 128 * k:128 * (k + 1)] = torch.round(v / step) * step
        return {"codes": codes, "scales": scales}
    if c["op"] == "product":
        y = torch.zeros(c["rows"], c["outer"], dtype=f64, device="cuda")
        ob = torch.arange(c["outer"], device="cuda") // 128
        for k in range(s["w_scale"].shape[0]):
            cut = slice(128 * k, min(128 * (k + 1), c["inner"]))
            x = s["x"][:, cut].to(f64) * s["x_scale"][k].to(f64)[:, None]
            y += x @ (s["w"][:, cut].to(f64) * s["w_scale"][k].to(f64)[ob, None]).t()
        return y
    if c["op"] == "plan":
        room, slots = _by_hand(s, c)
        return {"room": room, "slots": slots, "pages": s["pages"], "held": s["held"], "top": s["top"]}
    B, n, V = c["batch"], c["n"], c["vocab"]
    path, accepted, token = np.full((B, n), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    draws, tokens = s["uniforms"].double().cpu().numpy(), s["tokens"].cpu().numpy()
    for b, parent in enumerate(_parents(c)):
        rows = s["logits"][b * n:(b + 1) * n]
        node, way = 0, [0]
        while True:
            z = rows[node].to(f64)
            if c["temp"] > 0:
                p = torch.softmax(z / c["temp"], 0)
            else:  # all on the first of the largest
                p = torch.zeros_like(z)
                p[int((z == z.max()).nonzero()[0])] = 1.0
            went = False
            for i in [i for i in range(n) if i and parent[i] == node]:
                t = int(tokens[b, i])
                q = s["draft"][b * n + node].to(f64) if "draft" in s and c["temp"] > 0 else None
                have = float(p[t])
                if (c["temp"] == 0 and have == 1.0) or (c["temp"] > 0 and draws[b, i] * (1.0 if q is None else float(q[t])) < have):
                    node, went = i, True
                    way.append(i)
                    break
                if c["temp"] > 0:
                    if q is None:
                        p[t] = 0.0
                    else:
                        p = (p - q).clamp(min=0)
                    p = p / p.sum()
            if not went:
                break
        run_up = torch.cumsum(p, 0)
        found = ((p > 0) & (run_up > draws[b, 0] * float(run_up[-1]))).nonzero()
        token[b] = int(found[0] if len(found) else (p > 0).nonzero()[-1])
        path[b, :len(way)], accepted[b] = way, len(way)
    i32 = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return {"path": i32(path), "accepted": i32(accepted), "next": i32(token)}


def _by_hand(s, c):
    """The step's pages from a stack: pages given back go on it, the first on top, and new ones come off it."""
    _, after, count = _requests(c)
    stack = s["free"][:int(s["top"])].tolist()
    table = s["pages"].tolist()
    held, page = s["held"].tolist(), c["page"]
    need = [-(-(a + n) // page) for a, n in zip(after, count)]
    gone = [table[b][j] for b in range(c["batch"]) for j in range(need[b], held[b])]
    stack += gone[::-1]
    room, slots = [], np.full((c["batch"], c["n"]), -1, np.int64)
    for b in range(c["batch"]):
        mine = table[b][:min(held[b], need[b])]
        while len(mine) < need[b]:
            mine.append(stack.pop())
        room.append(count[b])
        at = after[b] + np.arange(count[b])
        if count[b]:
            slots[b, :count[b]] = np.array(mine, np.int64)[at // page] * page + at % page
    return torch.tensor(room, dtype=torch.int32, device="cuda"), torch.from_numpy(slots).cuda()
