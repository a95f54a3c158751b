"""The shares that a distillation backward cuts dhidden's sum into (CPU): every
one holds rows of the table, and the workspace has fp32 sums for those alone."""

import math
import random

import pytest

import distill_tile_rule as D
import muon_newton_schulz_amd as M


def _sizes():
    r = random.Random(3)
    log = lambda lo, hi: int(math.exp(r.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    for _ in range(300):
        dim = log(64, 7168)
        yield log(16, 4096), log(8192, 163840), dim if r.random() < 0.3 else dim // 64 * 64, \
            r.choice(["bf16", "bf16", "fp32"])


CASES = [(128, 20011, 264, "bf16"), (41, 19863, 1600, "bf16"), (71, 25694, 320, "fp32"),
         (134, 94168, 1284, "bf16"), *_sizes()]


@pytest.mark.parametrize("part", range(4))
def test_no_share_is_empty(part):
    for n, vocab, dim, dtype in CASES[part::4]:
        room = math.ceil(dim / 8) * 8 if D.laid(n, dim, dtype, True) else dim
        piece, _ = D.pieces(n, vocab, dtype)
        s = D.splits(n, room, piece, dtype)
        assert (s - 1) * D.share_of(piece, s) < piece <= s * D.share_of(piece, s)
        forward = M.distill_loss_workspace_size(n, vocab, dim, 5, dtype, backward=False)
        assert M.distill_loss_workspace_size(n, vocab, dim, 5, dtype) == \
            max(forward, D.workspace(n, vocab, dim, 5, dtype)), (n, vocab, dim, dtype)


def test_the_rule_where_shares_were_empty():
    # 39 shares of 576 rows were laid out for 20011 rows, which 35 hold
    assert D.splits(128, 264, 20011, "bf16") == 35
