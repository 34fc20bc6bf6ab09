"""Sizes (rows, outputs, inputs) of 4-bit products that reach every kernel once: ("few", rows of a tile, tiles of 16
outputs, waves) or ("many", tiles of outputs of a wave, inputs cut).  test_layers_shapes_host.py holds them against
the rule that chooses."""

LINEAR = {
    ("few", 4, 1, 8): (3, 40, 416),
    ("few", 4, 1, 16): (3, 40, 8224),
    ("few", 16, 1, 8): (9, 40, 416),
    ("few", 16, 1, 16): (9, 40, 8224),
    ("few", 16, 2, 8): (9, 6133, 288),
    ("few", 32, 2, 4): (300, 1027, 160),
    ("few", 32, 2, 8): (40, 3061, 160),
    ("few", 32, 4, 4): (300, 2039, 160),
    ("few", 32, 4, 8): (30, 12277, 160),
    ("few", 64, 4, 4): (90, 12277, 160),
    ("few", 64, 4, 8): (40, 12277, 160),
    ("many", 2, False): (801, 3833, 160),
    ("many", 4, False): (1601, 4073, 160),
    ("many", 4, True): (801, 2033, 8224),
}
GATED = {
    ("few", 4, 1, 8): (3, 40, 416),
    ("few", 4, 1, 16): (3, 40, 8224),
    ("few", 16, 1, 8): (9, 40, 416),
    ("few", 16, 1, 16): (9, 40, 8224),
    ("few", 16, 2, 8): (9, 6133, 288),
    ("few", 32, 2, 4): (20, 12277, 160),
    ("few", 32, 2, 8): (20, 6133, 160),
    ("few", 64, 2, 4): (40, 12277, 160),
    ("few", 64, 2, 8): (40, 6133, 160),
    ("many", 2, False): (801, 2039, 160),
    ("many", 4, False): (1601, 2039, 160),
    ("many", 4, True): (449, 2035, 8224),
}
