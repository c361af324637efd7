"""CPU checks of the two-float exponentials and sums that decide a verification
(csrc/two_float.h, compiled here), against the host's widest floats."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_weight_reconstruction_wl_gb300", "csrc")

SRC = r"""
#include <algorithm>
#include <cstdio>
#include <random>

#include "two_float.h"

using namespace wl;

int main()
{
    float table[64];
    double tabs = 0;
    for (int j = 0; j < 32; ++j) {
        table[j] = kExp2High[j], table[32 + j] = kExp2Low[j];
        tabs = std::max(tabs, (double)std::fabs(((long double)table[j] + table[32 + j]) / exp2l(j / 32.0L) - 1));
    }
    std::printf("table %.3g\n", tabs);
    const long double log2e = 1.442695040888963407359924681001892137L;
    std::mt19937_64 g(1);
    std::uniform_real_distribution<double> un(0, 1);
    const double edge[] = {1, 4, 16, 32, 99};
    double worst[5] = {0}, low[5] = {0};
    for (long i = 0; i < 3000000; ++i) {
        const int k = i % 5;
        const double t = std::exp(un(g) * 6 - 3), y0 = edge[k] * (k ? 0.25 + 0.75 * un(g) : un(g));
        const float m = (float)((un(g) - 0.5) * std::exp(un(g) * 8 - 2)), l = (float)(m - y0 / 1.4426950408889634 * t);
        const long double y = ((long double)l - (long double)m) * (log2e / (long double)t), e = exp2l(y);
        if (l > m || y < -99) continue;
        const FF a = weight(l, m, ff_of(1.4426950408889634 / t), table);
        worst[k] = std::max(worst[k], (double)std::fabs(((long double)a.h + a.l - e) / e));
        low[k] = std::max(low[k], (double)std::fabs(a.l / a.h));
    }
    for (int k = 0; k < 5; ++k) std::printf("weight%g %.3g\nlow%g %.3g\n", edge[k], worst[k], edge[k], low[k]);
    // ends: the largest logit itself, an infinite distance, a masked token
    const FF c = ff_of(1.4426950408889634 / 0.7);
    const float big = 3.4e38f, inf = big * 10.0f;
    std::printf("one %.3g\n", std::fabs((double)weight(3.25f, 3.25f, c, table).h - 1) + std::fabs((double)weight(3.25f, 3.25f, c, table).l));
    std::printf("none %.3g\n", (double)(weight(-big, big, c, table).h + weight(-inf, 5.0f, c, table).h + weight(-inf, -big, c, table).h));
    // long sums of equal terms: one lane's
    double sums = 0, rest = 0;
    for (int r = 0; r < 60; ++r) {
        const float m = (float)(un(g) * 8), l = (float)(m - 16.6 * un(g));
        const FF x = weight(l, m, ff_of(1.4426950408889634 / (0.3 + un(g))), table);
        FF acc{0.0f, 0.0f};
        for (int v = 0; v < 8192; ++v) {
            FF s{0.0f, 0.0f};
            for (int i = 0; i < 4; ++i) s = ff_add(s, x);
            acc = ff_sum(acc, s);
        }
        const long double want = ((long double)x.h + x.l) * 32768;
        sums = std::max(sums, (double)std::fabs(((long double)acc.h + acc.l - want) / want));
        // R - S q, S q up to R
        const float q = (float)(un(g) * (double)x.h);
        const FF S = ff_of(0.9 + 0.1 * un(g)), R = residual(x, q, S);
        const long double left = (long double)x.h + x.l - ((long double)S.h + S.l) * q;
        rest = std::max(rest, (double)std::fabs(((long double)R.h + R.l - left) / ((long double)x.h + x.l)));
    }
    std::printf("sums %.3g\nrest %.3g\n", sums, rest);
}
"""


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    d = tmp_path_factory.mktemp("ff")
    (d / "s.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-Wall", "-Werror", "-I", CSRC, str(d / "s.cpp"), "-o", str(d / "s")], check=True)
    out = subprocess.run([str(d / "s")], capture_output=True, text=True, check=True).stdout
    return {k: float(v) for k, v in (line.split() for line in out.splitlines())}


def test_table(found):
    """Two floats of a number in [1, 2): the low one's own half step is 2^-50 at most."""
    assert found["table"] <= 2.0 ** -49


@pytest.mark.parametrize("to", [1, 4, 16, 32])
def test_weights_down_to_2_to_the_minus_32(found, to):
    """Roundings that reach the result, in parts of it: the square's three (2^-14 (1 + 1 + 1 + 1/2) 2^-24 = 2^-36.2 if all went
    one way at |f| = 1/64), the next term of the series (2^-39.5), sums of low parts (2^-39): 2^-36."""
    assert found[f"weight{to}"] <= 2.0 ** -36


def test_weights_below(found):
    """There the low part of (l - m) c, up to 2^-17, enters without its square's half: 2^-35, and the above."""
    assert found["weight99"] <= 2.0 ** -34
    assert max(v for k, v in found.items() if k.startswith("low")) <= 2.0 ** -16


def test_ends(found):
    assert found["one"] == 0 and found["none"] == 0


def test_sums_and_residuals(found):
    """A normed running sum loses 2^-48 of itself at each of 8192 steps: 2^-35 if all went one way; a residual is off by the
    roundings of its low parts, 2^-17 2^-24 of the weight and a few of 2^-24 2^-24."""
    assert found["sums"] <= 2.0 ** -35
    assert found["rest"] <= 2.0 ** -40
