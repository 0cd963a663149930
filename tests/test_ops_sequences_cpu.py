"""How the attention kernels read a sequence from the device's lengths and starts (attn_sequence, compiled for the host):
whatever the integers, no row belongs to two sequences and nothing lies outside the tensors."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r"""
#include <cstdio>
#include <vector>
#include "window_attn_common.cuh"
using namespace kvevict;
// a line: packed, batch, q_rows, k_rows, max_q, then the two arrays (batch + 1 starts, or batch lengths)
int main()
{
    int packed, batch, q_rows, k_rows, max_q;
    while (std::scanf("%d %d %d %d %d", &packed, &batch, &q_rows, &k_rows, &max_q) == 5) {
        std::vector<int> a(batch + packed), c(batch + packed);
        for (int &x : a) if (std::scanf("%d", &x) != 1) return 1;
        for (int &x : c) if (std::scanf("%d", &x) != 1) return 1;
        AttnProblem p{};
        p.batch = batch; p.q_rows = q_rows; p.k_rows = k_rows; p.max_q = max_q;
        if (packed) { p.q_starts = a.data(); p.k_starts = c.data(); }
        else { p.q_lens = a.data(); p.k_lens = c.data(); }
        bool sound = true;
        for (int b = 0; b < batch; ++b) {
            if (packed) sound = sound && !attn_falls(p, b);
            const AttnSeq s = attn_sequence(p, b, sound);
            std::printf("%d %d %d %d %d %d ", s.q0, s.n, s.k0, s.m, s.p0, s.bad ? 1 : 0);
        }
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def sequences(tmp_path_factory):
    d = tmp_path_factory.mktemp("seq")
    (d / "s.cu").write_text(SRC)
    from kv_cache_eviction_decode_gb300 import build
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(d / "s.cu"), "-o", str(d / "s")],
                   check=True)

    def run(packed, q_rows, k_rows, max_q, a, c):
        batch = len(a) - packed
        line = " ".join(map(str, [packed, batch, q_rows, k_rows, max_q, *a, *c]))
        out = subprocess.run([str(d / "s")], input=line, capture_output=True, text=True, check=True).stdout.split()
        v = [int(x) for x in out]
        return [dict(zip(("q0", "n", "k0", "m", "p0", "bad"), v[i:i + 6])) for i in range(0, len(v), 6)]
    return run


def test_sound_starts(sequences):
    got = sequences(1, 30, 40, 12, [2, 2, 12, 24, 30], [0, 5, 15, 15, 40])
    assert [(s["q0"], s["n"], s["k0"], s["m"], s["p0"], s["bad"]) for s in got] == \
        [(2, 0, 0, 5, 5, 0), (2, 10, 5, 10, 0, 0), (12, 12, 15, 0, -12, 0), (24, 6, 15, 25, 19, 0)]


@pytest.mark.parametrize("starts,whole", [([0, 20, 10, 15, 40], 0), ([0, 10, 5, 7, 20], 0), ([0, 5, 20, 3, 9, 30], 1)])
def test_a_start_that_goes_back_ends_the_batch(sequences, starts, whole):
    """The sequences before it are whole; its own and all behind it are left out, also those that start after their
    predecessor again, inside the rows of a sequence before."""
    got = sequences(1, 40, 40, 40, starts, starts)
    for b, s in enumerate(got):
        assert (s["q0"], s["n"], s["bad"]) == (starts[b], starts[b + 1] - starts[b], 0) if b <= whole else s["n"] == 0 and s["bad"], b


def test_any_starts_give_every_row_to_one_sequence(sequences):
    rng = random.Random(3)
    for _ in range(200):
        batch, rows = rng.randint(1, 8), rng.randint(1, 30)
        starts = [rng.randint(-4, rows + 4) for _ in range(batch + 1)]
        if rng.random() < 0.5:
            starts.sort()
            if batch > 1 and rng.random() < 0.7:
                i = rng.randrange(batch + 1)
                starts[i] = rng.randint(-4, rows + 4)
        ks = [rng.choice([rng.randint(-9, 60), 2**31 - 1, -2**31]) for _ in range(batch + 1)]
        owner = {}
        for b, s in enumerate(sequences(1, rows, 50, rng.randint(0, rows), starts, ks)):
            assert s["n"] >= 0 and s["m"] >= 0 and s["q0"] >= 0 and s["k0"] >= 0 and s["k0"] + s["m"] <= 50
            for r in range(s["q0"], s["q0"] + s["n"]):
                assert r < rows and r not in owner, (starts, b, owner.get(r))
                owner[r] = b


def test_rows_of_a_cut_sequence_keep_their_positions(sequences):
    """Queries beyond max_q or the tensor are left out at their end of the sequence: the others stay where m keys and
    the given number of queries put them, and see no later key."""
    (s,) = sequences(1, 30, 30, 20, [0, 30], [0, 30])
    assert (s["q0"], s["n"], s["m"], s["p0"], s["bad"]) == (0, 20, 30, 0, 1)
    (s,) = sequences(1, 30, 80, 30, [0, 50], [0, 80])
    assert (s["n"], s["p0"], s["bad"]) == (30, 30, 1)
    (s,) = sequences(1, 30, 20, 30, [-7, 10], [0, 20])      # its first seven queries are not there
    assert (s["q0"], s["n"], s["p0"], s["bad"]) == (0, 10, 10, 1)
    (s,) = sequences(0, 8, 40, 8, [11], [40])
    assert (s["n"], s["p0"], s["bad"]) == (8, 29, 1)
    for packed, a in ((1, [0, 2**31 - 1]), (0, [2**31 - 1]), (1, [-2**31, 2**31 - 1])):
        s = sequences(packed, 8, 40, 8, a, [0, 40] if packed else [40])[0]
        assert s["n"] == 8 and s["p0"] == -2**30 and s["bad"]
