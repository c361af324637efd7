"""CPU check of the kernels' source: no CTA touches a peer's shared memory before
a cluster barrier has told it that the peer has begun.  A store into a CTA that
has not begun may be lost or fault; which CTAs of a cluster begin late cannot be
arranged in a test on a GPU."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_weight_reconstruction_wl_gb300", "csrc")
TOUCH = re.compile(r"map_shared_rank\(|mapa\.shared::cluster")
BARRIER = re.compile(r"\bcl\.sync\(\)|\bcluster_wait\(\)|barrier\.cluster\.wait")
WORD = re.compile(r"\b([a-z_][a-z0-9_]*)\s*(?:<[^;{}()]*>)?\(")
KEYWORDS = {"if", "for", "while", "switch", "return", "sizeof", "alignof", "asm", "static_assert"}


def functions(path):
    """(name, body, is a kernel) of each function: its braces stand in the first column, or all of it on one line."""
    lines = [re.sub(r"//.*", "", ln.rstrip("\n")) for ln in open(path)]
    out = []
    for i, line in enumerate(lines):
        one = re.match(r"[a-z_].*\)\s*\{(.*)\}\s*$", line)
        if line != "{" and not one:
            continue
        head = [line.split("{")[0]] if one else []
        for above in [] if one else reversed(lines[:i]):
            if not above.strip() or above[0] in "}#" or above.endswith(";"):
                break
            head.insert(0, above)
        head = " ".join(ln for ln in head if not ln.startswith("template"))
        names = [w for w in WORD.findall(head) if not w.startswith("__")]
        if not names:
            continue
        body = one[1] if one else "\n".join(lines[i + 1:next(j for j in range(i + 1, len(lines)) if lines[j].startswith("}"))])
        out.append((names[0], body, "__global__" in head))
    return out


def calls(body):
    return [w for w in WORD.findall(body) if w not in KEYWORDS]


def sources():
    shared = [f for p in glob.glob(os.path.join(CSRC, "*.cuh")) for f in functions(p)]
    return {os.path.basename(p): shared + functions(p) for p in glob.glob(os.path.join(CSRC, "*.cu"))}


def closure(funcs, pattern):
    """Names of the functions whose body, or that of a function they call, matches."""
    found = {n for n, body, _ in funcs if pattern.search(body)}
    while True:
        more = {n for n, body, _ in funcs if n not in found and found & set(calls(body))}
        if not more:
            return found
        found |= more


def first(body, pattern, names):
    at = [m.start() for m in pattern.finditer(body)] + [m.start() for m in WORD.finditer(body) if m[1] in names]
    return min(at, default=None)


def early(funcs):
    """Kernels that touch a peer, and those of them that do so before any cluster barrier."""
    touch, sync = closure(funcs, TOUCH), {n for n, body, _ in funcs if BARRIER.search(body)}
    seen, bad = set(), set()
    for name, body, kernel in funcs:
        at = first(body, TOUCH, touch)
        if not kernel or at is None:
            continue
        seen.add(name)
        # a function that has both is taken to have its barrier first if it is itself right
        both = {n for n, b, k in funcs if not k and n in touch and n in sync and first(b, BARRIER, sync) is not None
                and first(b, BARRIER, sync - {n}) < first(b, TOUCH, touch - {n})}
        b = first(body, BARRIER, sync)
        if b is None or (b > at or (b == at and WORD.match(body, at)[1] not in both)):
            bad.add(name)
    return seen, bad


@pytest.mark.parametrize("source", sorted(sources()))
def test_peers_are_touched_after_a_cluster_barrier(source):
    assert not early(sources()[source])[1]


def test_all_kernels_with_peers_are_looked_at():
    seen = set().union(*(early(f)[0] for f in sources().values()))
    assert {"page_plan_kernel", "verify_kernel", "linear_f8_kernel", "linear_f8_pair_kernel", "prefill_kernel"} <= seen, seen


def test_a_store_before_the_barrier_is_found():
    right = sources()["page_plan.cu"]
    wrong = [(n, b.replace("cluster_wait();", "", 1), k) for n, b, k in right]
    assert early(right)[1] == set() and early(wrong)[1] == {"page_plan_kernel"}
