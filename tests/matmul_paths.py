"""Products that between them run every tile of the products' kernel, in each layout of its operands, whole and with k split,
dense and in groups.  (product, m, n, k, act, groups): product 0 is y, 1 dx, 2 dw; act 4 is SwiGLU.  Small for what they
reach; none is a multiple of its tile.  That they reach it is asserted without a GPU, so another choice of tiles
shows there which sizes to change here."""

FORWARD, DX, DW = range(3)

PATHS = [
    # forward, dense: 64 x 128, 128 x 128, 128 x 256, 256 x 256; whole, then k split
    (FORWARD, 39, 64, 64, 0, 0), (FORWARD, 1077, 3848, 64, 0, 0), (FORWARD, 13994, 528, 64, 0, 0), (FORWARD, 4133, 1992, 832, 0, 0),
    (FORWARD, 34, 64, 1064, 0, 0), (FORWARD, 68, 6608, 4480, 0, 0), (FORWARD, 273, 7976, 6992, 0, 0), (FORWARD, 11857, 168, 4992, 0, 0),
    # with SwiGLU
    (FORWARD, 40, 64, 72, 4, 0), (FORWARD, 278, 6576, 72, 4, 0), (FORWARD, 662, 5656, 64, 4, 0), (FORWARD, 10113, 416, 800, 4, 0),
    (FORWARD, 34, 72, 1000, 4, 0), (FORWARD, 66, 2752, 5608, 4, 0), (FORWARD, 264, 6864, 3408, 4, 0), (FORWARD, 150, 5856, 4376, 4, 0),
    # W streamed through registers
    (FORWARD, 1, 64, 64, 0, 0), (FORWARD, 18, 72, 64, 0, 0), (FORWARD, 1, 64, 64, 4, 0), (FORWARD, 20, 64, 64, 4, 0),
    # dx, dense
    (DX, 1, 64, 64, 0, 0), (DX, 11833, 64, 296, 0, 0), (DX, 1333, 64, 5952, 0, 0), (DX, 4178, 784, 1928, 0, 0),
    (DX, 1, 504, 64, 4, 0), (DX, 8853, 3320, 64, 0, 0), (DX, 296, 3000, 7240, 4, 0), (DX, 12103, 2376, 136, 4, 0),
    # dw, dense
    (DW, 1, 64, 64, 0, 0), (DW, 1, 5704, 280, 4, 0), (DW, 1, 3592, 1032, 4, 0), (DW, 844, 7024, 544, 4, 0),
    (DW, 1041, 64, 72, 0, 0), (DW, 4434, 3368, 136, 0, 0), (DW, 5390, 280, 7944, 0, 0), (DW, 4432, 5904, 152, 4, 0),
    # groups, one of them empty and none with a multiple of a step's rows
    (FORWARD, 67, 80, 64, 0, 2), (FORWARD, 15495, 152, 72, 0, 40), (FORWARD, 18, 3608, 80, 0, 40), (FORWARD, 5840, 1080, 832, 0, 40),
    (FORWARD, 73, 64, 64, 4, 2), (FORWARD, 590, 1960, 64, 4, 9), (FORWARD, 8, 4112, 64, 4, 9), (FORWARD, 5497, 592, 808, 4, 40),
    (FORWARD, 1, 64, 64, 0, 3), (FORWARD, 35, 104, 72, 0, 2), (FORWARD, 1, 64, 64, 4, 40), (FORWARD, 40, 72, 64, 4, 2),
    (DX, 1, 64, 64, 0, 3), (DX, 350, 64, 8096, 0, 5), (DX, 18, 64, 3752, 0, 40), (DX, 5978, 824, 1136, 0, 40),
    (DW, 1, 64, 64, 0, 2), (DW, 1, 792, 64, 0, 40), (DW, 1, 816, 136, 0, 40), (DW, 7684, 3816, 136, 0, 9),
    (FORWARD, 1207, 4192, 64, 0, 9), (FORWARD, 695, 4376, 64, 0, 5), (DX, 1273, 64, 3608, 0, 9), (DX, 673, 72, 4440, 0, 5),
    (DW, 939, 64, 7248, 0, 9), (DW, 529, 7312, 64, 0, 5), (DW, 543, 64, 72, 0, 5), (DW, 4101, 4000, 4000, 0, 3),
]


def group_sizes(m, groups):
    """Rows of each group: the second empty, the others uneven (odd where there are rows enough)."""
    left, out = m, []
    for e in range(groups):
        last = e == groups - 1 or (groups == 2 and e == 0)
        rows = 0 if e == 1 else left if last else min(left, (2 * m // groups) * (1 + e % 3) // 3 | 1)
        out.append(rows)
        left -= rows
    return out
