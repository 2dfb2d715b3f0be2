"""Products that pairs of thread blocks take: rows, cin, cout, type, activation, rounds of pairs.

Several tiles per pair (the sums of one go back to tensor memory while the MMAs of the next begin), blocks of channels odd
and even in number, more of them than stages; ragged pixels (with and without one for the second block) and outputs; rows
stored in vectors and in pieces; codes that are copied first."""
PAIRS = [
    (2816, 896, 2816, "bf16", "none", 2),    # 7 blocks of channels, whole tiles
    (2816, 896, 2816, "f32", "silu", 2),
    (2916, 1152, 2946, "f16", "gelu", 2),    # 9 blocks; 100 pixels and 130 outputs in the last tiles
    (2700, 1000, 2750, "bf16", "relu6", 2),  # copied codes, rows off 32 bytes
    (2561, 1280, 2817, "f32", "none", 2),    # one pixel, one output; rows off 16 bytes
    (4000, 896, 2816, "f16", "none", 3),     # an odd number of rounds
    (9000, 384, 2048, "bf16", "silu", 4),    # fewer blocks of channels than stages
    (2900, 3584, 2816, "bf16", "gelu", 2),   # 28 blocks
    (4096, 4096, 4096, "bf16", "gelu", 4),   # 32 blocks
    (3136, 1024, 1024, "f32", "none", 1),    # one round, stages used again
    (3000, 1100, 1030, "f16", "relu", 1),
]
