"""The form and launch that a shape of the MXFP4 product takes (host code of csrc/mx_forms.h,
compiled here with the host's compiler)."""
import os
import shutil
import subprocess

import pytest

from mx_walks import EVERY, FORMS, WALKS
from quantized_prefill_gemm_amd import build as qbuild

CXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(CXX is None, reason="g++ not available")

MAIN = r"""
#include <stdio.h>
#include "mx_forms.h"
using namespace qpg;
int main()                       // lines of rows S E N K; dense: E 0
{
    long long rows, S, E, N, K;
    while (scanf("%lld %lld %lld %lld %lld", &rows, &S, &E, &N, &K) == 5) {
        const Form form = E ? experts_form(rows, S, E, N, K) : choose(1, rows, N);
        const FormShape f = form_shape(form);
        const long long tiles = E ? experts_row_tiles(S, E, f.bm) : (rows + f.bm - 1) / f.bm;
        const StreamGrid g = f.per_cu ? StreamGrid{0, 0} : stream_grid(tiles * ((N + f.bn - 1) / f.bn));
        printf("%d %d %d %d %d %lld %u %u\n", (int)form, f.bm, f.bn, f.threads, f.per_cu, tiles, g.x, g.y);
    }
}
"""


class Launch:
    def __init__(self, line, N):
        form, self.bm, self.bn, self.threads, self.per_cu, self.row_tiles, self.x, self.y = map(int, line.split())
        self.form, self.n_tiles = FORMS[form], -(-N // self.bn)
        self.tiles = self.row_tiles * self.n_tiles
        self.grid = min(self.tiles, 256 * self.per_cu) if self.per_cu else self.tiles


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    d = tmp_path_factory.mktemp("forms")
    (d / "forms.cpp").write_text(MAIN)
    exe = str(d / "forms")
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(qbuild.HERE, "csrc"), "-o", exe,
                    str(d / "forms.cpp")], check=True)

    def ask(*shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        return [Launch(line, s[3]) for line, s in zip(out, shapes)]
    return ask


def shape_of(counts, dropped, top_k, N, K):
    if top_k is None:
        return counts[0], 0, 0, N, K
    S = sum(counts) + dropped
    assert S % top_k == 0
    return S // top_k, S, len(counts), N, K


def name(case):
    form, counts, dropped, top_k, N, K = case
    return f"{form}-{sum(counts)}-{'dense' if top_k is None else len(counts)}-{N}-{K}"


@pytest.mark.parametrize("case", WALKS, ids=name)
def test_walks(launches, case):
    """More tiles that hold rows than workgroups: some walk on to a second."""
    form, counts, *rest = case
    one, = launches(shape_of(counts, *rest))
    assert one.form == form
    real = sum(-(-c // one.bm) for c in counts) * one.n_tiles
    assert real <= one.row_tiles * one.n_tiles and real > one.grid, (real, one.grid)


@pytest.mark.parametrize("case", EVERY, ids=name)
def test_every_form(launches, case):
    form, counts, *rest = case
    one, = launches(shape_of(counts, *rest))
    assert one.form == form


def test_walks_have_odd_and_even_steps():
    """Of every tiled form that walks (64 x 64: of experts alone, since its rule keeps the tiles of a
    dense shape below its grid), both for the dense product and for experts."""
    for form in FORMS[4:]:
        for dense in (True, False):
            steps = {-(-k // 256) % 2 for f, _, _, top_k, _, k in WALKS if f == form and (top_k is None) == dense}
            assert steps == (set() if dense and form == "T64" else {0, 1}), (form, dense)
        widths = {n % 2 for f, _, _, _, n, _ in WALKS if f == form}
        tails = {k // 32 % 4 != 0 for f, _, _, _, _, k in WALKS if f == form}
        assert widths == {0, 1} and True in tails, form


# The largest shapes that the entry points take: rows S E N K, E 0 the dense product.
LARGEST = [(2 ** 21, 2 ** 21, 8, 4096, 4096), (2 ** 23, 2 ** 23, 8, 1024, 1024), (2 ** 22, 2 ** 23, 64, 2048, 2048),
           (520, 0, 0, 2 ** 24 + 40, 32), (1, 0, 0, 2 ** 30 - 64, 32), (16, 0, 0, 2 ** 30 - 64, 32), (2 ** 30 - 64, 0, 0, 16, 32),
           (2 ** 15, 0, 0, 2 ** 20 - 1, 32), (2 ** 17, 2 ** 20, 1024, 2 ** 14, 2048), (2 ** 29, 2 ** 30, 1, 16, 64)]


@pytest.mark.parametrize("shape", LARGEST, ids=lambda s: "-".join(map(str, s)))
def test_largest_shapes_launch(launches, shape):
    """Every tile has a workgroup, and each side of the grid what a launch holds."""
    one, = launches(shape)
    if not one.per_cu:
        assert one.x * one.y >= one.tiles > one.x * (one.y - 1)
        assert one.x * one.threads < 2 ** 32 and one.y <= 65535 and one.x * one.y < 2 ** 32
    else:
        assert one.grid * one.threads < 2 ** 32


def test_random_shapes_launch(launches):
    import random
    rng, shapes = random.Random(5), []

    def log(high):
        return max(1, min(high, int(2 ** rng.uniform(0, high.bit_length()))))
    while len(shapes) < 4000:
        K = 32 * log(2 ** 19)
        E = rng.choice([0, log(1024)])
        most = (2 ** 35 - 2 ** 11) // K
        rows, N = log(most), log(max(1, most // max(E, 1)))
        S = rows * rng.randint(1, 8) if E else 0
        tiles = ((S + 15) // 16 + E if E else (rows + 15) // 16) * ((N + 15) // 16)
        if tiles >= 2 ** 31 or S > 2 ** 30 or (E and E * ((S + 15) // 16) >= 2 ** 31) or E * N * K > 2 ** 35 - 2 ** 11:
            continue
        shapes.append((rows, S, E, N, K))
    for shape, one in zip(shapes, launches(*shapes)):
        assert one.tiles < 2 ** 31, shape
        if not one.per_cu:
            assert one.x * one.y >= one.tiles > one.x * (one.y - 1), shape
            assert one.x * one.threads < 2 ** 32 and one.y <= 65535, shape
        else:
            assert shape[3] <= 2 ** 24, shape                     # what a tile's stores address
