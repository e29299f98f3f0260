"""Products of every form that mx_matmul has on 152 SMs, and their sizes.

A form is (pairs of SMs or not, columns of a tile, way out, CTAs that share a
sum); the pair kernel's cases have more than two tiles for some pair, so that
both buffers of sums and the columns that they share are used again."""
TMA, FROM_BF16, FROM_F32, ADD_BF16, ADD_F32 = range(5)
SMS = 152

#: columns, way out, rows of a, rows of b, K blocks (256 elements of 4 bits, 128 of 8), fp32
PAIRS = [
    (256, TMA, 5700, 2048, 6, False), (256, TMA, 5700, 2048, 6, True),
    # whole lines, and the last tile's rows that are not
    (256, FROM_BF16, 5700, 2048, 4, False), (256, FROM_F32, 5700, 2048, 4, True),
    (256, ADD_BF16, 1800, 4928, 1, False), (256, ADD_F32, 5700, 2048, 4, True),
    # rows that start anywhere
    (256, FROM_BF16, 1800, 4900, 1, False), (256, FROM_BF16, 1800, 4901, 9, False), (256, FROM_F32, 1800, 5001, 1, True),
    (256, ADD_BF16, 1800, 4900, 1, False), (256, ADD_BF16, 1800, 4901, 7, False), (256, ADD_F32, 2400, 5001, 4, True),
    # more K blocks than stages
    (256, FROM_BF16, 5700, 2048, 25, False), (256, ADD_F32, 5700, 2048, 13, True),
    (224, TMA, 1300, 5632, 1, False), (224, TMA, 1300, 5632, 1, True),
    (224, ADD_F32, 1300, 5632, 1, True), (224, ADD_F32, 2600, 3001, 1, True),
    (128, TMA, 19500, 240, 15, False), (128, TMA, 19500, 240, 15, True),
    (128, FROM_BF16, 19648, 232, 3, False), (128, FROM_F32, 19588, 228, 10, True),
    (128, ADD_BF16, 800, 4928, 1, False), (128, ADD_F32, 19812, 228, 32, True),
    (128, FROM_BF16, 800, 4900, 1, False), (128, FROM_F32, 800, 5001, 1, True),
    (128, ADD_BF16, 800, 4900, 1, False), (128, ADD_F32, 19596, 225, 13, True),
]
#: columns, CTAs that share a sum, rows of the one matrix and the other, K blocks
SPLITS = [(16, s, 7, 300, 4 * s if s > 1 else 3) for s in range(1, 9)] \
    + [(32, s, 20, 300, 4 * s if s > 1 else 3) for s in range(1, 9)] \
    + [(64, s, 40, 300, 4 * s + 1) for s in range(2, 9)] + [(64, 1, 150, 2700, 1)]


def elements(four, kblocks):
    return kblocks * (256 if four else 128)
