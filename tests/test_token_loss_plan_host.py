"""The plan of the cross entropy over a vocabulary, on the host: which tiles, pieces and
passes sizes lead to, and bounds that the kernels rely on."""
import shutil
import subprocess

import pytest

from padding_free_pair_amd.build import CSRC
from token_cases import LOSS_PLANS

PROGRAM = r"""
#include <cstdio>
#include "nt_token_loss_plan.hpp"
using namespace nt::token_loss;
int main() {
  long long T, V, C;
  int narrow;
  while (std::scanf("%lld %lld %lld %d", &T, &V, &C, &narrow) == 4) {
    const Plan f = forward_plan(T, V, C, narrow), b = backward_plan(T, V, C, narrow);
    const long long pieces = tiles_of(V, b.piece);
    std::printf("forward %d logits %d singles %d weights %d tokens %lld piece %lld pieces %lld "
                "last %lld padded %lld ldt %lld ldv %lld planes %lld w_most %d x_budget %lld "
                "WT %zu d %zu x_sums %zu w_sums %zu total %zu\n",
                f.logits.tile, b.logits.tile, b.singles.tile, b.weights.tile, (long long)b.tokens,
                (long long)b.piece, pieces, (long long)(V - (pieces - 1) * b.piece),
                (long long)b.padded, (long long)b.ldt, (long long)b.ldv, (long long)b.planes,
                b.w_most, (long long)b.x_budget, b.WT, b.d, b.x_sums, b.w_sums, b.total);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    made = subprocess.run([gxx, "-std=c++17", "-O1", f"-I{CSRC}", str(at / "plan.cpp"), "-o",
                           str(at / "plan")], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr

    def of(cases):
        lines = "".join(f"{T} {V} {C} {1 if dtype == 'bf16' else 0}\n" for T, V, C, dtype in cases)
        ran = subprocess.run([str(at / "plan")], input=lines, capture_output=True, text=True)
        assert ran.returncode == 0
        words = [line.split() for line in ran.stdout.splitlines()]
        return [dict(zip(w[::2], map(int, w[1::2]))) for w in words]

    return of


def test_cases_reach_what_they_are_for(plan):
    """A change of the cost rule that empties a case is seen here."""
    for (name, case), p in zip(LOSS_PLANS.items(), plan([c[:4] for c in LOSS_PLANS.values()])):
        for key, value in case[5].items():
            assert p[key] == value, (name, key, p)


def test_arrays_hold_their_pieces(plan):
    """Whole pieces and padded tokens, in arrays that do not meet, of bounded size."""
    cases = [(T, V, C, dtype) for dtype in ("bf16", "f32")
             for T in (1, 33, 256, 257, 1866, 8007, 65536, 65537, 200000)
             for V in (1, 33, 257, 4099, 32003, 131072, 2 ** 26) for C in (8, 384, 2048, 16384)]
    for case, p in zip(cases, plan(cases)):
        T, V, C, dtype = case
        es = 2 if dtype == "bf16" else 4
        rows = min(p["piece"], V)
        assert p["piece"] % 256 == 0 and 1 <= p["last"] <= p["piece"], case
        assert p["tokens"] <= min(T, 65536) and p["padded"] % 256 == 0, case
        assert p["tokens"] <= p["padded"] < p["ldt"] and p["piece"] < p["ldv"], case
        assert p["d"] - p["WT"] >= es * p["ldv"] * C, case
        assert p["x_sums"] - p["d"] >= es * p["planes"] * p["ldt"] * p["piece"], case
        assert p["w_sums"] - p["x_sums"] >= 4 * p["x_budget"] >= 4 * p["padded"] * C, case
        assert p["w_most"] == 1 or p["total"] - p["w_sums"] >= 4 * p["w_most"] * rows * C, case
        # loads count bytes from a tile's first row in 32 bits
        assert 256 * p["ldt"] * es < 2 ** 32 and 256 * p["ldv"] * es < 2 ** 32, case
        assert p["tokens"] * C * es <= 2 ** 32, case
