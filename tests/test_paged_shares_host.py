"""How the attention over pages shares a call's tiles out to CTAs: the product's own arithmetic (mp_paged.cuh),
compiled for the host."""
import random
import subprocess

import pytest

HEAD = r"""
#include <cstdio>
#include <vector>
#include "mp_paged.cuh"
using namespace mp;
"""

# shares of a total: every tile belongs to one CTA, found again from the tile, and a cluster's ranks
SHARES = HEAD + r"""
int main() {
    const int totals[] = {1, 2, 7, 151, 152, 153, 303, 305, 1000, 10007, 123456789, (1 << 30) + (1 << 22),
                          2147483647 - 304, 2147483647};
    for (int total : totals)
        for (int ctas : {1, 2, 152, 304}) {
            PArgs a = {};
            a.ctas = ctas;
            const Shares s(a, total);
            if (s.n != (ctas < total ? ctas : total) || s.first(0) != 0 || s.first(s.n) != total) return 1;
            for (int c = 0; c < s.n; ++c) {
                const int lo = s.first(c), hi = s.first(c + 1);
                if (hi <= lo || hi - lo > (total - 1) / s.n + 1) return 2;
                const int at[] = {lo, lo + (hi - lo) / 2, hi - 1};
                for (int t : at)
                    if (s.of(t) != c) return 3;
            }
        }
    PArgs a = {};
    a.ctas = 152;
    if (Shares(a, 0).n != 0) return 4;
    puts("ok");
}
"""

# a batch: every CTA's walk from where its run begins, and the CTAs that a unit's states are joined from
WALK = HEAD + r"""
int main() {
    PArgs a = {};
    std::vector<int> lengths;
    int with_lengths;
    while (scanf("%d %d %d %d %d %d %d", &a.B, &a.Hkv, &a.chunks, &a.n, &a.ctas, &a.tile_shift, &with_lengths) == 7) {
        lengths.assign(a.B, 0);
        for (int& x : lengths)
            if (scanf("%d", &x) != 1) return 1;
        a.pages.lengths = with_lengths ? lengths.data() : nullptr;
        struct Tile { int b, unit, t, tiles; };
        std::vector<Tile> all;
        for (int b = 0; b < a.B; ++b)
            for (int u = 0; u < a.Hkv * a.chunks; ++u)
                for (int t = 0; t < tiles_of(a, length_of(a, b)); ++t)
                    all.push_back({b, u, t, tiles_of(a, length_of(a, b))});
        const int total = static_cast<int>(all.size());
        const Shares s(a, total);
        int seen = 0;
        for (int c = 0; c < s.n; ++c) {
            const Tile& from = all[s.first(c)];
            Walk w = {s.first(c + 1) - s.first(c), from.b, from.unit, from.t, from.tiles, length_of(a, from.b)};
            if (w.left < 1) return 2;
            for (int parts = 0; w.left > 0; ++parts) {
                const int here = w.here();
                if (here < 1 || w.t + here > w.tiles) return 3;
                // a unit that this CTA has not to itself: the rest of one, or the beginning of one; and the
                // CTAs that the join finds for it are those that have its tiles
                const bool whole = here == w.tiles;
                if (!whole && w.t > 0 && parts > 0) return 4;
                const int t0 = seen - w.t, c0 = s.of(t0), c1 = s.of(t0 + w.tiles - 1);
                if (c < c0 || c > c1 || whole != (c0 == c1)) return 5;
                for (int k = 0; k < here; ++k, ++seen) {
                    const Tile& x = all[seen];
                    if (x.b != w.b || x.unit != w.unit || x.t != w.t + k || x.tiles != w.tiles ||
                        w.len != length_of(a, x.b))
                        return 6;
                }
                w.next(a, here);
            }
        }
        if (seen != total) return 7;
    }
    puts("ok");
}
"""


def _run(tmp_path, source, text=""):
    from lsh_sampled_sparse_gb300.build import NVCC_FLAGS, nvcc
    (tmp_path / "a.cu").write_text(source)
    subprocess.run([nvcc(), *NVCC_FLAGS, str(tmp_path / "a.cu"), "-o", str(tmp_path / "a")], check=True)
    r = subprocess.run([str(tmp_path / "a")], input=text, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.returncode


def test_shares_cover_the_tiles_once(tmp_path):
    _run(tmp_path, SHARES)


@pytest.mark.parametrize("shift,ctas", [(7, 152), (5, 304), (7, 3)])
def test_runs_cover_every_unit_of_a_batch(tmp_path, shift, ctas):
    rng = random.Random(shift + ctas)
    text = ""
    for case in range(120):
        B, Hkv, chunks = rng.choice([1, 2, 5, 33, 300]), rng.choice([1, 2, 3, 8]), rng.choice([1, 1, 2, 3])
        n = rng.choice([1, 31, 32, 33, 128, 129, 1000, 5000])
        used = [rng.choice([0, 1, n, rng.randint(-5, n + 7), rng.randint(0, n)]) for _ in range(B)]
        if case % 5 == 0:
            used = [0] * B
            used[rng.randrange(B)] = n
        text += f"{B} {Hkv} {chunks} {n} {ctas} {shift} {case % 4 != 0:d} " + " ".join(map(str, used)) + "\n"
    _run(tmp_path, WALK, text)
