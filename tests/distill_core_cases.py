"""Distillation cases that run the tile cores which the smaller ones of
test_gpu_distill.py do not choose, or not with sums long enough for their steady
state.  test_distill_core_coverage.py checks on the CPU that both together
reach every core."""

# n, vocab, dim, top, dtype, off (element offset of the operands), fp32 gradients
CORES = [
    (138, 41436, 264, 33, "bf16", 0, 0),    # statistics and g: Half
    (167, 32787, 232, 64, "bf16", 0, 1),
    (5711, 1023, 1464, 5, "bf16", 0, 0),    # dhidden: Half, one share
    (5700, 1021, 1461, 5, "bf16", 1, 1),    # the same from rows laid out
    (17, 42227, 2520, 128, "bf16", 0, 0),   # Half, many shares, the last one ragged
    (11884, 11416, 648, 9, "bf16", 0, 0),   # Half, two pieces of the vocabulary
    (10779, 12893, 408, 3, "bf16", 0, 1),   # and three shares of each
    (66, 12509, 1248, 40, "bf16", 1, 0),    # dhidden: any operands, 128
    (6166, 1078, 480, 17, "bf16", 1, 0),
    (65, 10105, 2880, 30, "fp32", 0, 0),
    (4374, 1023, 928, 12, "fp32", 0, 0),
]
