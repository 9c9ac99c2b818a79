"""Products of 4-bit operands that between them run every kernel, dense and in groups, with and without SwiGLU, over whole and
odd numbers of 128-k units; no size is a multiple of its tile.  (kernel, m, n, k, act, groups); act 4 is SwiGLU.  That they
take the kernel is asserted without a GPU, so another choice of kernels shows there which sizes to change here."""
FEW1, FEW2, FEW4, BIG, MID, LOW, THIN = range(7)

PATHS = [
    (FEW1, 5, 72, 640, 0, 0), (FEW1, 13, 40, 1000, 4, 0), (FEW1, 9, 72, 512, 0, 4),
    (FEW2, 29, 2056, 1152, 0, 0), (FEW2, 31, 1032, 1024, 4, 0), (FEW2, 70, 520, 1100, 0, 3),
    (FEW4, 61, 1032, 3328, 0, 0), (FEW4, 187, 264, 2563, 4, 0), (FEW4, 110, 520, 2688, 0, 2),
    (LOW, 1000, 1000, 640, 0, 0), (LOW, 900, 520, 1000, 4, 0), (LOW, 1300, 520, 1152, 0, 40), (LOW, 1400, 264, 300, 4, 33),
    (MID, 2040, 4104, 300, 0, 0), (MID, 2100, 2056, 512, 4, 0), (MID, 5000, 1032, 640, 0, 40), (MID, 4900, 520, 300, 4, 40),
    (BIG, 4090, 4088, 1100, 0, 0), (BIG, 4000, 2040, 1152, 4, 0), (BIG, 8000, 4088, 1100, 0, 4), (BIG, 8000, 2040, 1152, 4, 4),
    (BIG, 7800, 4088, 1100, 0, 0), (BIG, 8000, 2040, 1024, 4, 0),     # more tiles than workgroups
    (THIN, 100, 520, 1152, 0, 64), (THIN, 130, 264, 1100, 4, 64), (THIN, 300, 1032, 500, 0, 70),
]

# (m, n, k) of few rows and many columns of a row so wide that codes of such rows, each at its own place, would lie too far apart
# for a tile, while one row in place of all does not
ONE_ROW_WIDE = (16, 32768, 1 << 26)
