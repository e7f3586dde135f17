"""The rule by which products in 4 bits take their tiles, restated: which tiling a shape gets on a GPU of 152 SMs, how many
slices of K its tiles have, how many stages the ring of operands, and how many tiles a group of CTAs walks."""
SMS = 152
MAX_SMEM = 232448


def up(n, d):
    return -(-n // d)


def tri(t):
    return t * (t + 1) // 2


def stages(fmt, cg, bn):
    kt = 4 if fmt == "nvfp4" else 2
    stage = 128 * 128 + bn // cg * 128 + kt * 512 * (1 + up(bn, 128))
    return min(8, (MAX_SMEM - 1024 - 4 * 2 * 4096 - 512) // stage)


def tiling(count, m, n, sym):
    """(CTAs of a group, rows of B of a tile)"""
    m1, m2 = up(m, 128), up(m, 256)
    single = up(count * (tri(m1) if sym else m1 * up(n, 128)), SMS)
    pairs = up(count * (tri(m2) if sym else m2 * up(n, 192)), SMS // 2)
    if sym:
        return (2, 256) if 1.75 * pairs < single else (1, 128)
    if 1.2 * pairs < single:
        return 2, 192
    return (1, 64) if 2 * count * m1 * up(n, 128) <= SMS else (1, 128)


def walk(count, m, n, k, sym, fmt):
    """tiling, slices of a tile, stages of the ring, most tiles of a group"""
    cg, bn = tiling(count, m, n, sym)
    rows = up(m, 128 * cg)
    tiles = count * (tri(rows) if sym else rows * up(n, bn))
    return (cg, bn, sym), up(k, 256), stages(fmt, cg, bn), up(tiles, SMS // cg)


# count, m, n, k: for each tiling more slices of K than the ring has stages, in one tile and in several of a group
GEMMS = [(1, 1999, 1283, 2099), (3, 1999, 1283, 2099), (1, 41, 10007, 2085), (1, 300, 8203, 1777), (2, 70, 333, 2501)]
GRAMS = [(1, 2777, 2101), (2, 2777, 1777), (2, 333, 2001), (7, 1025, 1777)]
