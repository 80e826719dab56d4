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
