"""Sizes at which the products in 32 and 16 bits and their gradients take each
of their kernels: valid rows of the experts, the multiple that segments are
rounded up to, N, K, and the types (0 fp32, 1 bf16, 2 fp16)."""

ALL, HALF = (0, 1, 2), (1, 2)
CASES = [
    ([1], 128, 264, 520, ALL), ([3, 9, 16], 128, 7168, 136, ALL), ([5] * 40, 128, 1032, 264, ALL),
    ([5] * 40, 128, 264, 1032, HALF), ([5] * 40, 128, 1088, 320, ALL), ([5] * 40, 128, 320, 1088, HALF),
    ([2000, 1900], 128, 4096, 136, HALF), ([2000, 1900], 128, 4096, 192, ALL),
    ([1500, 1600], 128, 264, 7176, ALL), ([1500, 1600], 128, 320, 7176, HALF),
    ([300, 0, 290, 301, 17, 255], 128, 2056, 2056, ALL), ([3, 0, 1, 16], 16, 2048, 1032, HALF),
    ([130, 90, 200, 61], 128, 776, 392, ALL), ([130, 90, 200, 61], 128, 768, 384, ALL),
    ([700, 650, 730], 128, 2056, 1032, HALF), ([700, 650, 730], 128, 2048, 1024, ALL),
    ([600, 513, 640, 590, 0, 601, 620, 580], 128, 1152, 1024, HALF),
    ([30, 17, 32, 1], 32, 520, 264, HALF), ([20, 30], 32, 512, 512, HALF),
]


def rows_of(counts, align):
    return sum(-(-n // align) * align for n in counts)
