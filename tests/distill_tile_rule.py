"""Which tile core a distillation call's products take, how many shares
dhidden's sum is cut into, and the workspace that follows: the library's rule on
the host, beside tile_rule.py's for the vocabulary loss."""

import math
import re

import tile_rule as R


def _constant(name):
    return int(re.search(r"\b" + name + r" = (\d+)[,;]", R._source("distill.hip")).group(1))


def _round64(v):
    return math.ceil(v / 64) * 64


def share_of(piece, splits):
    """Rows of a share, as k_loss_dh takes them."""
    return _round64(math.ceil(piece / splits))


def laid(n, dim, dtype, backward):
    limit = _constant("kLayBackward" if backward else "kLayForward")
    return dtype == "bf16" and dim % 8 != 0 and n >= limit


def pieces(n, vocab, dtype):
    size = 2 if dtype == "bf16" else 4
    step = R._loss_constant("kPieceStep")
    least = int(re.search(r"kMinPiece = (\d+)", R._source("lm_loss.hip")).group(1))
    piece = max(least, R._loss_constant("kPieceBytes") // (size * n) // step * step)
    if piece >= vocab:
        return vocab, 1
    piece = math.ceil(math.ceil(vocab / math.ceil(vocab / piece)) / step) * step
    return piece, math.ceil(vocab / piece)


def splits(n, dim, piece, dtype):
    half = dtype == "bf16"
    table = "NN" if half and dim % 8 == 0 else "AnyBf16" if half else "AnyFp32"
    best, least = 1, 0.0
    for s in range(1, _constant("kMostSplits") + 1):
        if s > 1 and piece // s < 512:
            break
        t = 0.0
        for c in R.TABLES[table]:
            cols = math.ceil(dim / c[1])
            tiles = float(math.ceil(n / c[0]) * s * cols)
            even = tiles if c[2] == 1 or tiles <= 256 else math.ceil(tiles / 256) * 256.0
            e = R._time(c, even / cols, dim,
                        (2 if half else 1) * math.ceil(piece / s))
            t = e if t == 0.0 or e < t else t
        if s > 1:
            t += 8.0 * n * dim * s / 2.5e6 + 4.0
        if s == 1 or t < least:
            best, least = s, t
    return math.ceil(piece / share_of(piece, best))


def distill(n, vocab, dim, dtype, grid):
    """As tile_rule.loss; grid: operands and results start on the 16-byte grid
    and their rows follow each other without a gap."""
    room, on = dim, grid and dim % 8 == 0
    if laid(n, dim, dtype, True):
        room, on = math.ceil(dim / 8) * 8, True
    forward = (math.ceil(dim / 8) * 8, True) if laid(n, dim, dtype, False) else \
        (dim, grid and dim % 8 == 0)
    piece, count = pieces(n, vocab, dtype)
    cut = splits(n, room, piece, dtype)
    planes = 2 if dtype == "bf16" else 1
    return {
        "stats": (R.core("NT", forward[1], dtype, R._tiles(min(n, 16384)), vocab, forward[0]),
                  forward[0]),
        "g": (R.core("NT", on, dtype, R._tiles(n), piece, room), room),
        "dh": (R.core("NN", on, dtype, lambda bm: float(math.ceil(n / bm) * cut), room,
                      planes * math.ceil(piece / cut)), planes * min(share_of(piece, cut), piece)),
        "dw": (R.core("TN", on, dtype, R._tiles(piece), room, planes * n), planes * n),
    }, count, cut


def workspace(n, vocab, dim, top, dtype):
    """Bytes of distill_loss_workspace_size with backward, where the backward
    needs more than the forward."""
    align = lambda b: (b + 255) // 256 * 256  # noqa: E731
    size, planes = (2, 2) if dtype == "bf16" else (4, 1)
    is_laid = laid(n, dim, dtype, True)
    room = math.ceil(dim / 8) * 8 if is_laid else dim
    piece, count = pieces(n, vocab, dtype)
    cut = splits(n, room, piece, dtype)
    ldg = math.ceil(piece / 8) * 8
    ldg += 128 if ldg % 1024 == 0 else 0
    parts = [256, planes * n * ldg * size, n * room * size]
    if cut > 1 or count > 1 or is_laid:
        parts.append(cut * n * room * 4)
    parts += [n * top * 4, n * 4, n * 8]
    if is_laid:
        parts.append(vocab * room * 2)
    return sum(align(p) for p in parts)
