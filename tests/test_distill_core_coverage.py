"""The GPU cases of the distillation reach every tile core of each product, in
its steady state, under the rule that the library chooses with (CPU)."""

import math

import distill_tile_rule as D
import test_gpu_distill as G
import tile_rule as R
from distill_core_cases import CORES

PRODUCTS = {"stats": "NT", "g": "NT", "dh": "NN", "dw": "TN"}


def _cases():
    for n, vocab, dim, _, dt, _, _, _, _, off, pad, *_ in G.CASES:
        yield n, vocab, dim, dt, not off and pad % 8 == 0
    mark = next(m for m in G.test_tile_cores.pytestmark if m.name == "parametrize")
    for n, vocab, dim, _, dt, off in mark.args[1]:
        yield n, vocab, dim, dt, not off
    for n, vocab, dim, _, dt, off, _ in CORES:
        yield n, vocab, dim, dt, not off


def test_every_core_of_every_product():
    seen = {p: set() for p in PRODUCTS}
    pieces, ragged = set(), set()
    for n, vocab, dim, dt, grid in _cases():
        chosen, count, cut = D.distill(n, vocab, dim, dt, grid)
        for p, (core, k) in chosen.items():
            per, _ = R.stage(core, PRODUCTS[p]) if core in R.SHAPES else (1, 0)
            if core not in R.SHAPES or math.ceil(k / per) > R.steady_stages(core, PRODUCTS[p]):
                seen[p].add(core)
        if dt == "bf16" and chosen["dh"][0] in R.SHAPES:
            piece, _ = D.pieces(n, vocab, dt)
            pieces.add((chosen["dh"][0], count > 1, cut > 1))
            if cut > 1 and (piece % D.share_of(piece, cut)) % 32:
                ragged.add(chosen["dh"][0])
    for p, layout in PRODUCTS.items():
        dma = R.SHAPES if layout != "TN" else R.SHAPES[:3]
        assert seen[p] == {*dma, "Any64", "Any128", "Split64", "Split128"}, p
    # dhidden in Half tiles: one piece and two, one share and more
    for count in (False, True):
        for cut in (False, True):
            assert ("Half", count, cut) in pieces
    assert "Half" in ragged


def test_a_size_of_the_timed_ranges_that_takes_half_tiles():
    assert D.distill(51, 160221, 4480, "bf16", True)[0]["dh"][0] == "Half"
