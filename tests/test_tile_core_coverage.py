"""The GPU cases of tile_core_cases.py reach every tile core, and the DMA
cores' steady loops, under the rule that the library chooses with (CPU)."""

import math

import tile_rule as R
from tile_core_cases import EXPERTS, LOSS

PRODUCTS = {"stats": "NT", "g": "NT", "dh": "NN", "dw": "TN"}


def _steady(core, layout, k):
    if core not in R.SHAPES:
        return True
    per, _ = R.stage(core, layout)
    return math.ceil(k / per) > R.steady_stages(core, layout)


def _cores(layout):
    dma = R.SHAPES if layout != "TN" else R.SHAPES[:3]
    return {*dma, "Any64", "Any128", "Split64", "Split128"}


def test_expert_cases_reach_every_core():
    seen = {layout: set() for layout in ("NN", "NT", "TN")}
    for layout, rows, experts, k, n, _, dt, off in EXPERTS:
        grid = not off and k % 8 == 0 and n % 8 == 0
        if layout == "TN":
            core, length = R.expert_wgrad(rows, experts, k, n, dt, grid), rows // experts
        else:
            core, length = R.expert_matmul(rows, experts, k, n, dt, grid, layout == "NT"), k
        if _steady(core, layout, length):
            seen[layout].add(core)
    for layout, cores in seen.items():
        assert cores == _cores(layout), layout


def test_loss_cases_reach_every_core():
    seen = {p: set() for p in PRODUCTS}
    joined = False
    for n, vocab, dim, dt, off in LOSS:
        chosen, pieces, splits = R.loss(n, vocab, dim, dt, not off and dim % 8 == 0)
        for product, (core, length) in chosen.items():
            if _steady(core, PRODUCTS[product], length):
                seen[product].add(core)
        # the last piece adds the fp32 sums of those before into dhidden itself
        joined |= pieces > 1 and splits == 1 and dt == "bf16"
    assert joined
    for product, cores in seen.items():
        assert cores == _cores(PRODUCTS[product]), product


def test_the_rule_reads_the_sources():
    assert [len(R.TABLES[t]) for t in ("NT", "NN", "TN", "AnyBf16", "AnyFp32")] == [4, 4, 3, 2, 2]
    for layout in ("NT", "NN", "TN"):
        for shape in R.SHAPES:
            per, slots = R.stage(shape, layout)
            assert per in (32, 64) and 2 <= slots <= 6
