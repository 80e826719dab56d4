"""Sizes at which the operators of a layer's step take each of their kernels'
variants: run on the GPU by test_gpu_layer_variants.py, and looked over by
test_layer_plans.py, so that a changed rule cannot leave a variant out."""

# vocabulary rows of a 4-bit matrix, and the hidden rows for which each gives a variant of its own
MXFP4_HEAD = [
    (2050, (1, 5, 9, 17, 33, 129)),
    (9001, (5, 9, 17)),
    (16411, (1, 5, 9, 17, 33, 50, 65, 84, 100, 129, 161, 224, 241)),
    (63001, (9, 17, 33, 50, 65, 100)),
    (83003, (9, 17, 33, 50)),
    (120023, (5, 17, 33, 50)),
    (132027, (9, 17, 33, 50)),
    (164003, (9, 17, 33, 50)),
    (200064, (5, 17, 33, 50, 65, 84, 100, 129, 161, 224)),
]

# (T, Hq, Hkv, D, R, interleaved, norm, keys to, tokens of a short call): norm and rotation with two heads a lane, and in
# short calls of the same tokens with one; wave counts of a token that are odd and one, lanes without columns
ROPE = [
    (1501, 30, 5, 64, 32, False, True, "rows", 400),
    (1501, 20, 9, 48, 48, True, True, "bf16", 400),
    (2101, 7, 5, 64, 64, False, False, "e4m3", 700),
    (851, 30, 6, 128, 128, False, True, "rows", 300),
    (1402, 9, 4, 80, 80, True, False, "bf16", 500),
    (1403, 16, 4, 128, 64, False, True, "e4m3", 500),
    (1404, 5, 4, 256, 128, True, True, "rows", 500),
    (1405, 3, 3, 192, 192, False, True, "bf16", 500),
    (4201, 1, 1, 256, 256, True, True, "e4m3", 2000),
]


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, both among them, in no order."""
    return [hi if i == n // 2 else lo + (hi - lo) * (i * 61 % n) // n for i in range(n)]


# Attention with first tokens, by the rows of a tile, the key groups of a work-group over a bf16 and over an 8-bit cache and
# whether the keys are split: tokens already in the cache and new ones of each request, query and key heads, page size,
# window, first tokens, and what else the call takes
ATTENTION_SINKS = [
    ((16, 4, 4, False), _spread(5, 0, 700), [3, 1, 0, 3, 2], 4, 2, 16, 70, 20, dict(causal=False)),
    ((16, 4, 4, True), [2500, 1100, 30], [5, 5, 3], 6, 2, 32, 1100, 70, dict(layout="hnd")),
    ((16, 2, 4, False), _spread(65, 0, 300), [1] * 65, 8, 4, 16, 90, 33, {}),
    ((16, 1, 2, False), _spread(65, 1, 400), [1] * 65, 16, 8, 64, 90, 4, dict(idx=True)),
    ((32, 4, 4, True), [2700, 1300, 5], [8, 7, 8], 6, 2, 16, 1100, 70, dict(idx=True)),
    ((32, 4, 4, False), _spread(33, 100, 1500), [8] * 31 + [0, 5], 16, 4, 64, 1000, 4, {}),
    ((32, 2, 4, False), _spread(65, 0, 300), [8] * 60 + [1, 3, 8, 0, 7], 16, 4, 32, 90, 17, dict(layout="hnd")),
    ((32, 1, 2, False), _spread(65, 0, 200), [7] * 65, 24, 8, 16, 65, 64, {}),
    ((64, 4, 4, True), [3000, 1500], [17, 13], 6, 2, 16, 1500, 130, dict(causal=False)),
    ((64, 4, 4, False), _spread(20, 0, 1600), [9] * 19 + [2], 40, 8, 64, 1000, 5, dict(layout="hnd")),
    ((64, 2, 2, False), _spread(33, 0, 1500), [9] * 30 + [1, 0, 8], 40, 8, 32, 1000, 4, dict(idx=True)),
    ((64, 2, 2, True), _spread(17, 100, 3000), [9] * 17, 40, 8, 128, 2100, 16, {}),
    ((64, 1, 1, False), _spread(128, 0, 150), [9] * 128, 32, 8, 16, 40, 20, {}),
    ((128, 1, 1, False), [300, 900, 20], [601, 37, 1], 64, 8, 16, 500, 70, {}),
    ((128, 1, 1, True), [4500], [513], 32, 8, 64, 4200, 33, {}),
]
