"""Sizes (T, E, k, F, K, N) of whole routed layers that the GPU tests run beside
test_layer_gpu.py's; test_layer_plan.py checks that they reach every kernel and choice of
the two launches."""

# rows of every depth (2, 4, 6, 8, 10 chunks of 256), whole (K % 64 == 0) and not, and one shorter than 64
ROWS = [48, 448, 400, 960, 1008, 1472, 1264, 1984, 1840, 2816, 5200]


def _gate():
    for k in ROWS:
        t = 1 if k > 4096 else 2                 # (rows of binary32 fit the blocks' LDS)
        yield (t, 16, 2, 80, k, 20)              # blocks per expert, of 64 weight rows
        yield (t, 16, 16 // t, 2064, k, 20)      # of 128
        yield (t, 64, 4, 608, k, 20)             # blocks per token and rank


GATE = list(_gate())

DOWN = [
    # 32 outputs per block: last blocks of 32, 1 to 16 and 17 to 31 outputs; rows shorter than 64, cut
    # and whole; one wave per row and teams of 2, 3, 4 and 8
    *((16, 12, 3, f, 64, n) for f in (48, 80, 128, 1040, 1088) for n in (1056, 1025, 1040, 1041, 1055)),
    (7, 9, 2, 2576, 80, 2400), (7, 9, 2, 2624, 80, 2410), (13, 20, 4, 4096, 64, 1290), (13, 20, 4, 4112, 64, 1297),
    (9, 6, 1, 8192, 64, 1830), (9, 6, 2, 8208, 64, 1823), (16, 16, 16, 320, 64, 1100), (5, 40, 9, 2064, 144, 3300),
    # both sides of the border
    (16, 8, 2, 144, 64, 1024), (15, 8, 2, 144, 64, 1089), (4, 8, 2, 144, 64, 4096), (4, 8, 2, 144, 64, 4097),
    (1, 8, 2, 144, 64, 16384), (1, 8, 2, 144, 64, 16385), (1, 8, 2, 1088, 64, 16400),
    # 16 outputs per block, teams with cut rows
    (3, 8, 2, 1040, 64, 100), (2, 8, 1, 8208, 64, 50), (1, 8, 3, 2576, 64, 33),
]

# both sides of the limits: LDS of the tokens' rows and of a token's rows of h, tokens, experts per token,
# experts, and raw tokens quantised in the blocks or before
LIMITS = [
    (16, 4, 2, 64, 9472, 32), (16, 4, 2, 64, 9488, 32), (2, 17, 16, 9472, 64, 32),
    (2, 17, 16, 9488, 64, 32), (17, 8, 2, 64, 64, 32), (2, 20, 17, 64, 64, 32), (2, 256, 2, 64, 64, 32),
    (2, 257, 2, 64, 64, 32), (6, 8, 2, 64, 2560, 32), (7, 8, 2, 64, 2560, 32), (3, 8, 2, 64, 2560, 32), (4, 8, 2, 64, 2560, 32),
    (6, 8, 2, 64, 8448, 32), (6, 8, 2, 64, 8704, 32),
]
