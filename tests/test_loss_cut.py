"""How the losses' rows are dealt out to CTAs (csrc/fo_loss_cut.h, compiled here by itself): on devices of few SMs, and
on ones whose SMs do not share clusters as the ones do that the kernels were measured on."""
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "overlapped_tensor_gemm_gb300", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")
pytestmark = pytest.mark.skipif(CXX is None, reason="needs a C++ compiler")

PROGRAM = r"""
#include <cstdio>
#include "fo_loss_cut.h"
int main() {
  fo::LossShape s;
  long long rows, groups;
  int waits, alone, exchange;
  while (std::scanf("%lld %lld %d %d %d %d %d %d %d %d %d %d %d %d", &rows, &groups, &s.chunk_groups, &s.threads, &waits,
                    &s.slots, &s.fit, &alone, &exchange, &s.places, s.teams, s.teams + 1, s.teams + 2, s.teams + 3) == 14) {
    s.rows = rows, s.groups = groups, s.waits = waits, s.reads_alone = alone, s.exchange = exchange;
    const fo::LossCut c = fo::loss_cut(s);
    std::printf("%d %d %lld\n", c.ctas, c.twice, static_cast<long long>(c.teams));
  }
}
"""
CHUNK, SLOTS, FIT = 2048, 6, 2  # groups of a copy; chunks that a CTA holds, and of a row where it is shared


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    at = tmp_path_factory.mktemp("cut")
    (at / "cut.cpp").write_text(PROGRAM)
    subprocess.run([CXX, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "cut.cpp"), "-o", str(at / "cut")], check=True)

    def call(shapes):
        text = "".join(" ".join(str(int(x)) for x in s) + "\n" for s in shapes)
        out = subprocess.run([str(at / "cut")], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(shapes)
        return got
    return call


def _shape(mode, rows, groups, sms, teams=None):
    policy = mode == "policy"
    places = sms * (1 if policy else 2)
    teams = teams or [places >> i for i in range(4)]
    return (rows, groups, CHUNK, 512 if policy else 256, policy, SLOTS, FIT, mode == "forward", mode != "backward", places,
            *teams)


def _random(n, seed, sms, clusters):
    rng = random.Random(seed)
    out = []
    for _ in range(n):
        mode, m = rng.choice(["policy", "forward", "backward"]), rng.choice(sms)
        places = m * (1 if mode == "policy" else 2)
        out.append((mode, _shape(mode, int(2 ** rng.uniform(0, 31)) - rng.randint(0, 1), int(2 ** rng.uniform(0, 20)) - 1, m,
                                 clusters(rng, places))))
    return out


@pytest.mark.parametrize("sms", [[1], [2, 3, 5, 7, 8, 10], [76, 132, 148, 152, 160]], ids=str)
def test_every_cut_can_be_launched(cut, sms):
    """Teams there are, of a size that the device holds, at most as many as fit, and a row that waits has room."""
    def clusters(rng, places):  # fewer than the SMs alone would give; sizes beyond some not at all
        most = rng.randint(1, 4)
        return [max(1, places >> i) if i == 0 else (max(0, (places >> i) - rng.randint(0, 4)) if i < most else 0)
                for i in range(4)]
    shapes = _random(3000, len(sms), sms, clusters)
    for (mode, s), (ctas, twice, teams) in zip(shapes, cut([s for _, s in shapes])):
        rows, groups, places, fits = s[0], s[1], s[9], s[10:]
        assert ctas in (1, 2, 4, 8) and teams >= 1
        fit = fits[ctas.bit_length() - 1]
        assert fit >= 1 and teams <= max(1, min(fit, rows)) and teams * ctas <= max(places, 1)
        chunks = -(-groups // CHUNK)
        if mode == "policy":
            assert twice or chunks <= ctas * SLOTS
        else:
            assert not twice


def test_the_measured_device_is_cut_as_before(cut):
    """Policy loss on 152 SMs of which 76, 36 and 15 clusters of 2, 4 and 8 fit: the rule as it was, with its constants."""
    def before(rows, groups):
        fit = lambda c: 152 * (152 if c <= 2 else 144 if c == 4 else 120) // 152 // c  # noqa: E731
        chunks, least, twice = -(-groups // CHUNK), 1, False
        while least < 8 and chunks > least * FIT:
            least *= 2
        if chunks > least * SLOTS:
            least, twice = 1, True
        ns, best, ctas = float(groups) * 32 * 152 / 6700.0, None, least
        c = least
        while c <= 8 and (c == least or groups >= c * 512):
            cost = -(-rows // fit(c)) * (ns / c + (700.0 if c > 1 else 500.0))
            if c == least or cost < best:
                ctas, best = c, cost
            c *= 2
        return ctas, int(twice), 1 if rows < 1 else min(rows, fit(ctas))
    rng = random.Random(5)
    sizes = [(rng.randint(0, 20000), rng.randint(0, 70000)) for _ in range(2000)]
    got = cut([_shape("policy", r, g, 152, [152, 76, 36, 15]) for r, g in sizes])
    assert got == [before(r, g) for r, g in sizes]
