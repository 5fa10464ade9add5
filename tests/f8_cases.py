"""Shapes (T, N, K) of the e4m3 products that the GPU tests run; test_f8_plan.py
checks that they reach every kernel that the library can choose."""

SHAPES = [
    # streaming kernel: one token to several tiles of tokens, rows and blocks of K that end anywhere
    (1, 1, 16), (1, 16, 128), (2, 17, 144), (3, 33, 112), (16, 130, 272), (1, 300, 2560), (15, 64, 640),
    (17, 257, 384), (32, 32, 1024), (33, 100, 400), (48, 129, 2576), (64, 96, 6912), (65, 128, 128),
    (66, 1, 16), (127, 255, 144), (129, 130, 2064), (300, 640, 400), (257, 513, 6912), (1000, 72, 512),
    (4, 5000, 28672), (70, 1030, 16384), (31, 4100, 272), (20, 8200, 144), (50, 4099, 400), (64, 4200, 1152),
    # 128 x 128 tiles, two groups of waves: 1, 2, 3 and 5 blocks of K, partial ones
    (70, 9001, 128), (130, 6000, 256), (130, 6001, 272), (257, 4999, 640), (200, 8197, 112), (129, 6400, 1040),
    # 256 x 128 tiles: 1 to 5 blocks of K
    (300, 16500, 128), (300, 16500, 256), (290, 16511, 272), (300, 16640, 512), (257, 17000, 528),
    # 256 x 256 tiles (bfloat16 outputs): 1 to 4 blocks of K
    (1100, 8200, 128), (1030, 8193, 144), (1025, 8448, 256), (1100, 8199, 384), (1280, 8200, 400),
]
