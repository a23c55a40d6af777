"""Sizes that take the products through each of their kernels, and the plan that each
size is meant to have: a change of the estimates that moves one of them to another
kernel shows in the tests of the plans, which need no GPU."""

FWD, DGRAD, WGRAD = 0, 1, 2
BIG, MID, LOW, ANY = 1, 2, 3, 4  # the public TILES_*: 256 x 256, 128 x 128, 64 x 128, rows of any alignment

# (op, M, N, K), (rows, tiles, split?, rest tiles, rest split?): the sizes are no multiples of a
# tile's or a step's, so that every edge is one
DENSE = [
    ((FWD, 1, 1000, 1288), (1, 0, 0, 0, 0)),
    ((FWD, 2, 1000, 1288), (2, 0, 0, 0, 0)),
    ((FWD, 3, 1000, 1288), (4, 0, 0, 0, 0)),
    ((FWD, 4, 5000, 776), (4, 0, 0, 0, 0)),
    ((FWD, 13, 6008, 136), (16, 0, 0, 0, 0)),
    ((FWD, 1710, 6384, 296), (0, BIG, 0, 0, 0)),
    ((FWD, 7546, 5496, 112), (0, BIG, 0, MID, 0)),
    ((FWD, 2184, 7176, 2264), (0, BIG, 0, MID, 1)),
    ((FWD, 2466, 7992, 216), (0, BIG, 0, LOW, 0)),
    ((FWD, 203, 1584, 1168), (0, MID, 0, 0, 0)),
    ((FWD, 181, 296, 1568), (0, MID, 1, 0, 0)),
    ((FWD, 652, 5400, 168), (0, LOW, 0, 0, 0)),
    ((FWD, 102, 1048, 1128), (0, LOW, 1, 0, 0)),
    ((FWD, 303, 1817, 963), (0, ANY, 0, 0, 0)),
    ((FWD, 3103, 5903, 185), (0, ANY, 0, ANY, 0)),
    ((FWD, 105, 897, 1307), (0, ANY, 1, 0, 0)),
    ((DGRAD, 5665, 392, 1808), (0, BIG, 0, 0, 0)),
    ((DGRAD, 7517, 264, 2456), (0, BIG, 0, MID, 0)),
    ((DGRAD, 7019, 2344, 2320), (0, BIG, 0, MID, 1)),
    ((DGRAD, 577, 7640, 2032), (0, BIG, 1, 0, 0)),
    ((DGRAD, 742, 760, 1040), (0, MID, 0, 0, 0)),
    ((DGRAD, 464, 8168, 104), (0, MID, 1, 0, 0)),
    ((DGRAD, 2449, 600, 1648), (0, LOW, 0, 0, 0)),
    ((DGRAD, 1552, 1336, 152), (0, LOW, 1, 0, 0)),
    ((DGRAD, 254, 1109, 1927), (0, ANY, 0, 0, 0)),
    ((DGRAD, 6922, 175, 2595), (0, ANY, 0, ANY, 0)),
    ((DGRAD, 239, 3625, 453), (0, ANY, 1, 0, 0)),
    ((WGRAD, 262, 5320, 2072), (0, BIG, 0, 0, 0)),
    ((WGRAD, 241, 7496, 2528), (0, BIG, 0, MID, 0)),
    ((WGRAD, 2337, 8016, 2056), (0, BIG, 0, MID, 1)),
    ((WGRAD, 8066, 680, 1720), (0, BIG, 1, 0, 0)),
    ((WGRAD, 163, 1936, 1560), (0, MID, 0, 0, 0)),
    ((WGRAD, 2634, 136, 1392), (0, MID, 1, 0, 0)),
    ((WGRAD, 283, 4664, 808), (0, LOW, 0, 0, 0)),
    ((WGRAD, 4123, 496, 232), (0, LOW, 1, 0, 0)),
    ((WGRAD, 901, 545, 739), (0, ANY, 0, 0, 0)),
    ((WGRAD, 249, 8765, 2067), (0, ANY, 0, ANY, 0)),
    ((WGRAD, 1755, 1073, 249), (0, ANY, 1, 0, 0)),
]

# (op, E, P, N, K), (rows, tiles, split?)
GROUPED = [
    ((FWD, 40, 8, 712, 648), (1, 0, 0)),
    ((FWD, 40, 40, 712, 648), (4, 0, 0)),
    ((FWD, 16, 4628, 2456, 240), (0, BIG, 0)),
    ((FWD, 8, 18, 2160, 2632), (0, BIG, 1)),
    ((FWD, 5, 811, 552, 656), (0, MID, 0)),
    ((FWD, 2, 336, 152, 1224), (0, MID, 1)),
    ((FWD, 33, 2474, 1232, 120), (0, LOW, 0)),
    ((FWD, 33, 215, 176, 2200), (0, LOW, 1)),
    ((FWD, 5, 811, 551, 657), (0, ANY, 0)),
    ((FWD, 2, 336, 151, 1223), (0, ANY, 1)),
    ((DGRAD, 33, 1414, 800, 2336), (0, BIG, 0)),
    ((DGRAD, 8, 9, 2768, 1880), (0, BIG, 1)),
    ((DGRAD, 2, 2392, 176, 648), (0, MID, 0)),
    ((DGRAD, 5, 193, 1480, 216), (0, MID, 1)),
    ((DGRAD, 33, 735, 136, 2552), (0, LOW, 0)),
    ((DGRAD, 16, 172, 1896, 400), (0, LOW, 1)),
    ((DGRAD, 2, 2392, 177, 647), (0, ANY, 0)),
    ((DGRAD, 5, 193, 1481, 215), (0, ANY, 1)),
    ((WGRAD, 16, 452, 2000, 1184), (0, BIG, 0)),
    ((WGRAD, 3, 912, 376, 600), (0, MID, 0)),
    ((WGRAD, 2, 2550, 928, 96), (0, MID, 1)),
    ((WGRAD, 33, 1209, 136, 496), (0, LOW, 0)),
    ((WGRAD, 3, 6668, 168, 1288), (0, LOW, 1)),
    ((WGRAD, 3, 912, 375, 601), (0, ANY, 0)),
    ((WGRAD, 2, 2550, 927, 95), (0, ANY, 1)),
]

# the weights' gradient with sums longer than the 1024 row indexes that it holds at a time:
# rows of the experts, N, K, (tiles, split?)
LONG = [1023, 0, 1024, 1025, 1, 1088, 3333, 2049]
LONG_SUMS = [
    ((LONG, 72, 264), (MID, 1)),
    ((LONG, 504, 776), (MID, 0)),
    ((LONG, 2056, 2056), (BIG, 0)),
    ((LONG, 33, 47), (ANY, 1)),
    ((LONG, 777, 1031), (ANY, 0)),
    # also longer than that in each part of a split sum
    (([9000, 1025, 0, 5000], 264, 264), (MID, 1)),
    (([9000, 0, 7001], 265, 263), (ANY, 1)),
    (([12000, 4668, 0], 168, 1288), (LOW, 1)),
    (([9000], 680, 1720), (BIG, 1)),
]


def names(cases):
    what = ("fwd", "dgrad", "wgrad")
    return [f"{what[c[0]]}_" + "x".join(str(v) for v in c[1:]) for c, _ in cases]


def counts_of(E, P):
    """P rows on E experts: some without rows, some with one, a few and more than a tile, the
    rest with what is left."""
    want = [0, 1, 0, 40, 17, 260, 130, 300, 16, 3]
    counts, left = [], P
    for e in range(E - 1):
        c = min(left, max(want[e % len(want)], (left // (E - e)) * (e % 3 == 2) * 2))
        counts.append(c)
        left -= c
    return counts + [left]
