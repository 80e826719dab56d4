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
