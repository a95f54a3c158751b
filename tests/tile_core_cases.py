"""Cases that run each tile core of the loss and of the expert products in its
steady state, with ragged ends of the sums and of the tiles.
test_tile_core_coverage.py checks on the CPU that they do."""

# layout, rows, experts, k, n, kind of offsets, dtype, off: element offset of
# the operands (1: off the 16-byte grid).  NN: x w, NT: x w^T, TN: the weights'
# gradient, a sum over an expert's rows.
EXPERTS = [
    ("NN", 130, 1, 1032, 264, "gaps", "bf16", 0),
    ("NN", 2200, 3, 520, 264, "ragged", "bf16", 0),
    ("NN", 900, 20, 520, 4088, "ragged", "bf16", 0),
    ("NN", 3840, 1, 2056, 4088, "gaps", "bf16", 0),
    ("NT", 130, 1, 1032, 264, "gaps", "bf16", 0),
    ("NT", 2200, 3, 520, 264, "ragged", "bf16", 0),
    ("NT", 1500, 8, 520, 4088, "gaps", "bf16", 0),
    ("NT", 3940, 1, 840, 4088, "gaps", "bf16", 0),
    ("TN", 700, 1, 520, 264, "gaps", "bf16", 0),
    ("TN", 3940, 13, 520, 1032, "ragged", "bf16", 0),
    ("TN", 5000, 4, 776, 4088, "gaps", "bf16", 0),
    ("NN", 130, 1, 520, 264, "gaps", "bf16", 1),
    ("NN", 700, 13, 520, 4088, "ragged", "bf16", 1),
    ("NT", 130, 1, 520, 264, "gaps", "bf16", 1),
    ("NT", 700, 13, 520, 4088, "ragged", "bf16", 1),
    ("TN", 300, 1, 520, 264, "gaps", "bf16", 1),
    ("TN", 3940, 13, 520, 520, "ragged", "bf16", 1),
    ("NN", 130, 1, 520, 264, "gaps", "fp32", 0),
    ("NN", 700, 13, 519, 4087, "ragged", "fp32", 0),
    ("NT", 130, 1, 520, 264, "gaps", "fp32", 0),
    ("NT", 700, 13, 519, 4087, "ragged", "fp32", 0),
    ("TN", 300, 1, 520, 264, "gaps", "fp32", 0),
    ("TN", 3940, 13, 520, 519, "ragged", "fp32", 0),
]

# n, vocab, dim, dtype, off
LOSS = [
    (130, 2000, 1032, "bf16", 0),
    (40, 20011, 264, "bf16", 0),
    (130, 33001, 264, "bf16", 0),
    (300, 20011, 392, "bf16", 0),
    (4100, 2000, 2056, "bf16", 0),
    (8200, 2000, 1544, "bf16", 0),
    (600, 20011, 520, "bf16", 0),
    (4000, 4000, 840, "bf16", 0),
    (8200, 20011, 1032, "bf16", 0),   # two pieces, dhidden's sums not split
    (40, 2000, 264, "bf16", 1),
    (130, 8000, 1541, "bf16", 1),
    (2100, 2000, 261, "bf16", 1),
    (40, 2000, 261, "fp32", 0),
    (130, 8000, 1541, "fp32", 0),
    (2100, 2000, 261, "fp32", 0),
]
