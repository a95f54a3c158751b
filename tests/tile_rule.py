"""Which tile core a call of the loss or of the expert products takes, and how
many stages its sums have: the library's rule on the host, with the constants
read from its sources, so that a test can tell whether a core is reached."""

import math
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_newton_schulz_amd", "csrc")
SHAPES = ("Large", "Half", "Medium", "Thin")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _tables():
    text, out = _source("train_gemm.h"), {}
    for name, body in re.findall(r"constexpr ShapeCost kShape(\w+)\[\] = \{(.*?)\};", text, re.S):
        out[name] = [tuple(float(v) for v in row.split(","))
                     for row in re.findall(r"\{([^{}]+)\}", body)]
    return out


TABLES = _tables()


def _loss_constant(name):
    expr = re.search(name + r" = ([^;]+?)[;,]", _source("lm_loss.hip")).group(1)
    expr = re.sub(r"static_cast<\w+>\((\d+)\)", r"\1", expr)
    return int(eval(expr, {"__builtins__": {}}))  # digits, << and * only


def stage(shape, layout):
    """(k a stage, slots) of the DMA core's shapes, as their aliases say."""
    text = _source("train_gemm.h")
    args = re.search(r"using %sCore = DmaCore<PKS, QKS, (.*?)>;" % shape, text, re.S).group(1)
    k, slots = re.fullmatch(r"\d+, \d+, \d+, (.+), (.+)", args).groups()

    def value(t):
        choice = re.fullmatch(r"\(PKS \|\| QKS\) \? (\d+) : (\d+)", t)
        if choice is None:
            return int(t)
        return int(choice.group(2 if layout == "NT" else 1))

    return value(k), value(slots)


def steady_stages(shape, layout):
    """Stages from which the pipeline's steady loop runs."""
    _, slots = stage(shape, layout)
    return 4 if slots == 2 else 2 * slots


def _time(c, row_tiles, cols, k):
    bm, bn, per_cu, alone, full, fixed = c
    tiles = row_tiles * math.ceil(cols / bn)
    places = 256.0 * per_cu

    def once(n):
        load = min(1.0, max(0.0, (n - 128.0) / (places - 128.0)))
        return k / 64.0 * (alone + (full - alone) * load) + fixed

    if tiles >= 8.0 * places:
        return (tiles / places + 0.5) * once(places)
    whole = math.floor(tiles / places)
    rest = tiles - whole * places
    return whole * once(places) + (once(rest) if rest > 0 else 0.0)


def _pick(table, rows, cols, k):
    best, t = 0, 0.0
    for i, c in enumerate(TABLES[table]):
        e = _time(c, rows(int(c[0])), cols, k)
        if i == 0 or e < t:
            best, t = i, e
    return best


def core(layout, grid, dtype, rows, cols, k):
    """Name of the core: rows(bm) row tiles of bm rows, cols columns, sums of
    k; grid: operands and result on the 16-byte grid."""
    if dtype == "bf16" and grid:
        return SHAPES[_pick(layout, rows, cols, k)]
    side = (128, 64)[_pick("AnyBf16" if dtype == "bf16" else "AnyFp32", rows, cols, k)]
    return ("Any" if dtype == "bf16" else "Split") + str(side)


def _tiles(n):
    return lambda bm: float(math.ceil(n / bm))


def expert_matmul(rows, experts, k, n, dtype, grid, trans):
    def tiles(bm):
        groups = min(rows, experts)
        r = rows / groups
        return groups * (1.0 if r <= bm / 2 else r / bm + 0.6)
    return core("NT" if trans else "NN", grid, dtype, tiles, n, k)


def expert_wgrad(rows, experts, m, n, dtype, grid):
    return core("TN", grid, dtype, lambda bm: experts * float(math.ceil(m / bm)), n,
                rows // experts)


def loss(n, vocab, dim, dtype, grid):
    """{product: (core, length of its sums)} of a forward and a backward, and
    the number of pieces and splits."""
    size = 2 if dtype == "bf16" else 4
    step = _loss_constant("kPieceStep")
    least = int(re.search(r"kMinPiece = (\d+)", _source("lm_loss.hip")).group(1))
    piece = max(least, _loss_constant("kPieceBytes") // (size * n) // step * step)
    pieces = 1
    if piece >= vocab:
        piece = vocab
    else:
        pieces = math.ceil(vocab / piece)
        piece = math.ceil(math.ceil(vocab / pieces) / step) * step
        pieces = math.ceil(vocab / piece)
    most = re.search(r"kMaxSplits = (\d+), kMaxSplitsAny = (\d+)", _source("lm_loss.hip"))
    most = int(most.group(1 if dtype == "bf16" and dim % 8 == 0 else 2))
    tiles = math.ceil(n / 128) * math.ceil(dim / 128)
    splits = max(1, min(most, 512 // tiles, math.ceil(piece / 512)))
    share = math.ceil(math.ceil(piece / splits) / 64) * 64
    part = math.ceil(piece / splits)

    planes = 2 if dtype == "bf16" else 1

    def dh(bm):
        return float(math.ceil(n / bm) * splits)

    return {
        "stats": (core("NT", grid, dtype, _tiles(min(n, 16384)), vocab, dim), dim),
        "g": (core("NT", grid, dtype, _tiles(n), piece, dim), dim),
        "dh": (core("NN", grid, dtype, dh, dim, planes * part), min(share, piece)),
        "dw": (core("TN", grid, dtype, _tiles(piece), dim, planes * n), n),
    }, pieces, splits
