"""Sizes (m, n, k) that reach every kernel form of the feed-forward operators:
odd token counts, ragged channels, a last piece of K that is not whole, and K
long enough to go round a tile's ring.  The keys are what plan_string says,
with "P" for the number of parts; test_ffn_plan.py holds them to it."""

PRODUCTS = {
    "gemm_i8": {
        "few 16": (9, 200, 4432), "few 32": (17, 200, 4816), "few 64": (37, 200, 4432), "Small": (131, 264, 1040),
        "Mid": (5537, 272, 1008), "Mid / P": (69, 136, 4112), "Shared": (5197, 784, 912), "Big": (5087, 1544, 1248)},
    "gemm_glu": {
        "few 16": (9, 200, 2320), "few 32": (17, 200, 2216), "few 64": (37, 136, 2184), "Small": (131, 136, 520),
        "Mid": (11, 8400, 1752), "Mid / P": (69, 72, 2056), "Shared": (293, 6640, 456), "Big": (1249, 3328, 616)},
    "gemm_glu_i8": {
        "few 16": (9, 200, 4304), "few 32": (17, 200, 4896), "few 64": (37, 136, 4320), "Small": (131, 136, 1040),
        "Mid": (13, 8976, 2288), "Mid / P": (69, 72, 4112), "Shared": (355, 5672, 912), "Big": (2183, 1912, 1200)}}

BACKWARD = {
    "dX + dW: Small": (341, 328, 264), "dX + dW: Mid": (1813, 744, 864), "dX + dW: Shared": (305, 496, 3064),
    "dX + dW: Big": (1009, 488, 6792), "dX: Mid / P, dW: Mid / P": (3759, 528, 16),
    "dX: Mid / P, dW: Big": (263, 3880, 1552), "dX: Mid / P, dW: Shared": (307, 8352, 160),
    "dX: Mid / P, dW: Small": (1, 968, 72), "dX: Mid / P, dW: Mid": (387, 8656, 16), "dX: Mid, dW: Big": (985, 2160, 3728),
    "dX: Shared, dW: Mid / P": (11229, 8, 264), "dX: Small, dW: Mid / P": (2013, 8, 72),
    "dX: Big, dW: Mid / P": (9819, 136, 1376)}

# (m, n, k) of a block whose products have K in parts: the forward ones, the
# down projection from integers and dX, the weight gradients
PARTS = [(100, 272, 9008), (100, 4512, 272), (9000, 144, 272)]
