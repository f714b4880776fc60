"""Sizes whose calls reach every kernel that the linear layers' plans choose from.  The plans are fitted
to measurements and change with them, so tests/test_linear_plans.py asserts (on the host) that these sizes still reach
what REQUIRED lists; tests/test_gpu_linear_plans.py compares each with 64 bits.  Rows are odd, widths end
inside tiles."""
import self_attention_gb300 as sa

PAIRS = 76      # pairs of CTAs; more tiles than that and a pair takes several

# M, K, N of attn_linear; per pair kernel one size of several tiles a pair, one of few
FORWARD = [(781, 552, 1096), (1413, 80, 1592), (3571, 1448, 2648), (1113, 1072, 6088), (331, 4104, 9224), (3, 40, 488), (3, 360, 8928),
           (13, 288, 96), (7, 2280, 48), (6129, 184, 8), (3303, 1112, 72), (17, 904, 2920), (407, 7632, 16),
           (187, 4296, 5112), (949, 1400, 264), (731, 2320, 192), (319, 2952, 6104), (5003, 4872, 64),
           (2471, 9296, 32), (1323, 5752, 48)]
# ... of attn_linear_q8
Q8 = [(1449, 112, 3904), (773, 1040, 1304), (1885, 1040, 4104), (6885, 4400, 304), (107, 32, 24), (7, 560, 5072),
      (11, 544, 112), (1, 7344, 152), (8137, 192, 8), (691, 1744, 408), (115, 1056, 704), (169, 2544, 176),
      (169, 8544, 4936), (2789, 5680, 40), (1355, 6032, 64), (321, 5088, 6184), (5213, 6256, 72), (3593, 7072, 40)]
# B, H, N, d_k, N_out of attn_out_proj
HEADS = [(3, 6, 154, 128, 1720), (29, 3, 71, 64, 1304), (76, 4, 178, 128, 672), (61, 3, 7, 64, 64), (5, 6, 3, 64, 1496),
         (7, 2, 4, 128, 176), (15, 17, 7, 64, 8), (53, 2, 21, 128, 264), (24, 9, 137, 128, 32), (5, 14, 334, 128, 8),
         (2, 11, 331, 128, 16), (26, 18, 149, 128, 16), (6, 20, 294, 128, 24), (18, 22, 10, 128, 3616),
         (42, 22, 119, 128, 32)]
# M, K, N of attn_linear_bwd, all gradients
BACKWARD = [(2619, 8, 5368), (15, 520, 192), (565, 1528, 680), (6123, 24, 152), (3317, 216, 7536), (2139, 3032, 40),
            (3039, 376, 4944), (1777, 6368, 632), (3055, 4560, 696), (8805, 496, 376), (4753, 800, 6024),
            (7389, 2976, 176), (7, 5048, 4496), (9, 520, 2080), (795, 696, 6040), (153, 1760, 3112), (347, 176, 4032),
            (45, 5944, 7736), (151, 904, 6896), (529, 3208, 8896), (621, 1624, 6256), (807, 408, 6880),
            (119, 1168, 8784)]
# B, H, N, d_k, N_out of attn_out_proj_bwd; the first is a batch of this framework's ViT-B block
HEADS_BACKWARD = [(32, 12, 576, 64, 768), (6, 2, 266, 64, 3880), (2, 16, 4, 128, 1440), (4, 8, 195, 128, 1160),
                  (6, 4, 154, 64, 416), (15, 16, 9, 128, 40), (120, 8, 188, 128, 8), (21, 6, 251, 64, 4328),
                  (55, 8, 24, 128, 3144), (15, 19, 233, 64, 2448), (32, 4, 362, 64, 1880), (91, 14, 4, 128, 752),
                  (104, 15, 93, 128, 280), (6, 16, 3, 128, 6792), (8, 18, 2, 64, 8928), (9, 4, 5, 128, 2488),
                  (3, 10, 131, 128, 7280), (9, 16, 17, 64, 4600), (3, 2, 162, 128, 2768), (16, 8, 4, 128, 8888),
                  (4, 3, 131, 128, 3664), (73, 7, 13, 128, 9016), (2, 19, 119, 128, 8240), (15, 6, 22, 128, 7352),
                  (22, 4, 24, 64, 6664)]


def _few(*splits_by_rows):
    return {("few", rows, s) for rows, splits in splits_by_rows for s in splits}


REQUIRED = {
    "forward": _few((16, (1, 2, 4, 8)), (32, (1, 2, 4, 8)), (64, (2, 4, 8)), (128, (1, 2, 4, 8)))
    | {("pair", bn, several) for bn in (128, 256) for several in (False, True)},
    "q8": _few((16, (1, 2, 4, 8)), (32, (1, 2, 4, 8)), (64, (2, 4, 8)), (128, (1, 2, 4)))
    | {("pair", bn, several) for bn in (128, 256) for several in (False, True)},
    "heads": _few((16, (1, 2, 4, 8)), (32, (1, 2, 4, 8)), (64, (4, 8)), (128, (1, 2)))
    | {("pair", 128, False), ("pair", 128, True), ("pair", 256, True)},
    "backward": _few((16, (4, 8)), (32, (2, 4, 8)), (64, (4, 8)), (128, (1, 2, 4, 8)))
    | {("products", bn, split, bias) for bn in (128, 256) for split in (False, True) for bias in (0, 1, 2)},
    "heads_backward": _few((16, (2, 4, 8)), (32, (2, 4, 8)), (64, (4, 8)), (128, (1, 2, 4, 8)))
    | {("products", bn, split, bias) for bn in (128, 256) for split in (False, True) for bias in (0, 1, 2)},
}


def forward_plan(kind, size):
    """("few", rows, splits) or ("pair", columns, whether a pair takes several tiles)."""
    B, H, T, d, N = size if len(size) == 5 else (1, 1, *size)
    rows, splits, bn, _, _ = sa.attn_debug_linear_plan(kind, B, H, T, d, N)
    if rows:
        return "few", rows, splits
    blocks = B * -(-T // 32) * 32 if B > 1 and H > 1 and T > 1 else B * T
    return "pair", bn, -(-blocks // 256) * -(-N // bn) > PAIRS


def backward_plans(size, act=0):
    """{("few", rows, splits) of dx where that kernel takes it, ("products", columns, dw split?, way of dbias)
    where one launch takes both}."""
    B, H, T, d, N = size if len(size) == 5 else (1, 1, *size)
    rows, splits, bn, dw, bias = sa.attn_debug_linear_plan(2, B, H, T, d, N, act)
    return {("few", rows, splits)} if rows else {("products", bn, dw > 1, bias)}


def reached():
    return {
        "forward": {forward_plan(0, s) for s in FORWARD},
        "q8": {forward_plan(1, s) for s in Q8},
        "heads": {forward_plan(0, s) for s in HEADS},
        "backward": set().union(*(backward_plans(s) for s in BACKWARD)),
        "heads_backward": set().union(*(backward_plans(s) for s in HEADS_BACKWARD)),
    }
