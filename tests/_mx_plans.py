"""Sizes of products by the kernel that they take: what the tests on the GPU run, and a
test on the host holds to the choice that the library makes."""

FMTS = ("e2m1", "e4m3", "e5m2")
PAIRS = tuple((a, b) for a in FMTS for b in FMTS)
FOUR = (("e2m1", "e2m1"),)
EIGHT = tuple(p for p in PAIRS if p not in FOUR)                  # an operand of 8 bits
BOTH = tuple(p for p in PAIRS if "e2m1" not in p)                 # two
SOME = (("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3"))
BF16, FP32, ANY = ("bf16",), ("fp32",), ("bf16", "fp32")

# rows of a, of b, columns; strips a side of the few-row kernel (0: the many-row kernel), 64-result units a side of
# that one, splits; pairs of formats; types of the result
CASES = [
    # 256 x 256 results a workgroup: one chunk of columns, two, three, five and more; whole and ragged on both sides;
    # 8192^2 and 4096^2 go past the caches
    (8192, 8192, 250, (0, 4, 1), EIGHT, BF16),
    (8100, 8100, 500, (0, 4, 1), PAIRS, BF16),
    (8100, 8100, 700, (0, 4, 1), SOME, BF16),
    (4096, 4096, 1280, (0, 4, 1), PAIRS, BF16),
    (4000, 4000, 1300, (0, 4, 1), PAIRS, BF16),
    (4000, 4090, 2600, (0, 4, 1), SOME, BF16),
    (4096, 4096, 1280, (0, 4, 1), FOUR, FP32),
    (4522, 7059, 523, (0, 4, 1), FOUR, FP32),
    # 128 x 128
    (850, 2729, 1, (0, 2, 1), FOUR, ANY),
    (7548, 296, 31, (0, 2, 1), EIGHT, ANY),
    (2040, 2100, 500, (0, 2, 1), PAIRS, ANY),
    (2048, 2048, 768, (0, 2, 1), SOME, ANY),
    (2000, 2000, 1300, (0, 2, 1), PAIRS, ANY),
    (2048, 2048, 2560, (0, 2, 1), SOME, ANY),
    # 128 x 128, the columns cut: chunks that divide by the splits and that do not, few and many splits
    (100, 130, 20000, (0, 2, 16), EIGHT, ANY),
    (100, 131, 70000, (0, 2, 55), PAIRS, ANY),
    (500, 1000, 16000, (0, 2, 8), EIGHT, FP32),
    (500, 1000, 16000, (0, 2, 8), BOTH, BF16),
    (1, 1, 19265, (0, 2, 19), FOUR, ANY),
    # 2 x 2 strips of the few-row kernel
    (900, 1000, 1300, (2, 0, 1), EIGHT, BF16),
    (34, 8851, 262, (2, 0, 1), BOTH, BF16),
    (202, 3540, 1398, (2, 0, 1), FOUR, BF16),
    (321, 2227, 2842, (2, 0, 1), FOUR, FP32),
    (168, 5431, 4434, (2, 0, 1), EIGHT, FP32),
    # one by one
    (300, 777, 1100, (1, 0, 1), PAIRS, ANY),
    (64, 96, 9000, (1, 0, 1), PAIRS, ANY),
]

CALLS = [(m, n, k, plan, a, b, dtype) for m, n, k, plan, pairs, dtypes in CASES for a, b in pairs for dtype in dtypes]


def name(call):
    m, n, k, plan, a, b, dtype = call
    return f"{m}x{n}x{k}-{a}-{b}-{dtype}"
