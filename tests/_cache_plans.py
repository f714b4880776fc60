"""The sizes at which the GPU tests of the cache's attention run, and that they reach every kernel it chooses from.  The
choice goes by the room in the cache, so that each case of few slots runs with little room and with much."""
import self_attention_gb300 as sa

ROOM = 40000

# B, H, G, T, d, C, lengths
CASES = [
    # B, H, G, T, d, C, lengths
    (1, 1, 1, 1, 64, 1, [0]),
    (1, 1, 1, 1, 128, 130, [129]),
    (2, 3, 4, 1, 128, 200, [63, 64]),
    (3, 2, 1, 1, 64, 1000, [0, 999, 500]),
    (2, 1, 8, 1, 128, 77, [15, 16]),
    (2, 2, 9, 1, 64, 300, [290, 17]),
    (1, 2, 16, 1, 128, 2100, [2050]),
    (5, 1, 17, 1, 64, 90, [1, 2, 3, 88, 31]),
    (2, 2, 1, 5, 128, 140, [120, 0]),
    (2, 3, 2, 13, 64, 270, [255, 128]),
    (1, 1, 4, 33, 128, 700, [600]),
    (2, 2, 4, 64, 128, 330, [266, 1]),
    (1, 2, 8, 64, 64, 400, [200]),
    (2, 1, 3, 50, 128, 200, [127, 128]),
    (1, 1, 1, 64, 64, 64, [0]),
    (40, 2, 2, 1, 64, 70, [i % 69 for i in range(40)]),
]

# runs of blocks over several heads and sequences: B, H, G, T, d, C, raggedness of the lengths
BLOCKS = [
    (8, 4, 2, 10, 128, 1500, 1400), (8, 4, 2, 10, 64, 1500, 1400), (6, 4, 4, 50, 128, 1700, 900), (6, 4, 4, 64, 64, 1700, 1600),
    (3, 5, 8, 60, 128, 2900, 100), (40, 8, 1, 33, 64, 300, 260), (2, 3, 2, 64, 128, 20000, 5000), (33, 7, 4, 64, 128, 270, 200),
    (9, 16, 4, 1, 128, 5000, 4900), (9, 16, 3, 4, 64, 5000, 4900), (300, 1, 1, 20, 64, 200, 130), (1, 1, 4, 64, 128, 30000, 0),
    (9, 16, 4, 1, 128, 9000, 8900), (40, 8, 1, 1, 64, 9000, 8000), (20, 8, 3, 4, 128, 6000, 5000), (33, 8, 3, 4, 64, 6500, 5000),
    (300, 1, 3, 1, 64, 4200, 4100), (11, 7, 2, 33, 128, 1300, 1200), (11, 7, 4, 40, 64, 1300, 1200),
    # parts of the larger tiles, joined by few blocks and by many
    (2, 4, 4, 64, 128, 9000, 3000), (4, 4, 4, 50, 128, 6000, 700), (7, 4, 3, 64, 128, 3700, 900),
    (11, 4, 3, 64, 128, 3700, 900), (2, 1, 2, 40, 64, 20000, 9000), (10, 4, 5, 50, 64, 8000, 600)]

# units by clusters of every size
BLOCKS += [(2, 1, 4, T, d, C, 250) for T in (1, 4) for d in (64, 128) for C in (260, 390, 520, 650, 780, 910)]
BLOCKS += [(8, 5, 4, 1, 128, 390, 300), (8, 5, 3, 3, 128, 386, 300), (6, 9, 3, 3, 64, 650, 500), (20, 8, 2, 1, 128, 210, 200)]

# T, G, d: masks that are no trees, values that are not finite
ODD = [(3, 1, 64), (20, 2, 64), (64, 4, 64), (7, 2, 128), (50, 1, 128), (64, 8, 128)]
POISON = [(4, 1, 64), (7, 2, 128), (30, 4, 128), (64, 2, 64), (64, 4, 128), (64, 8, 64)]


def reached():
    """(kind, rows of a unit, d) of every case."""
    sizes = [(B, H, G, T, c, d) for B, H, G, T, d, C, _ in CASES for c in (C, ROOM)]
    sizes += [(B, H, G, T, C, d) for B, H, G, T, d, C, _ in BLOCKS]
    sizes += [(3, 2, G, T, c, d) for T, G, d in ODD for c in (150, ROOM)]
    sizes += [(2, 2, G, T, c, d) for T, G, d in POISON for c in (300, ROOM)]
    return {sa.attn_debug_cache_plan(*x)[:2] + (x[5],) for x in sizes}


def clusters():
    """(CTAs of a cluster, d) of the cases with few rows."""
    plans = {sa.attn_debug_cache_plan(B, H, G, T, C, d) + (d,) for B, H, G, T, d, C, _ in BLOCKS}
    return {p[2:] for p in plans if p[0] == 1}
