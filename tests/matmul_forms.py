"""Sizes (rows of the weight, columns, rows of x) of products that together take every kernel that the launchers can dispatch, for one
weight and for two, in one part of x and in three, in both formats; and how a call's kernel is told from its plan."""

ONE_PART = [
    # few rows of x: 2, 4, 8 waves on the long axis; scale bytes four at a time, then one by one
    (12310, 768, 13), (12310, 288, 5), (6161, 512, 7), (6161, 544, 3), (37, 1024, 1), (37, 800, 3), (37, 768, 13), (37, 544, 13),
    # 17 to 32 rows
    (12310, 512, 29), (12310, 800, 17), (37, 2048, 17), (37, 544, 19), (37, 256, 29), (37, 800, 32),
    # many rows: tiles of 32, 64, 128, whole and with the long axis split
    (37, 256, 64), (37, 544, 33), (301, 768, 65), (37, 1056, 33),
    (2051, 256, 1001), (2051, 288, 1001), (515, 256, 2049), (515, 288, 2049), (37, 4096, 2049), (301, 2080, 1500), (37, 2592, 3001),
    (301, 2560, 1001),
    (4099, 256, 1001), (4099, 288, 1001), (16405, 4096, 101), (2051, 4384, 1001), (301, 4384, 3001), (20, 14336, 8192),
]
THREE_PARTS = [
    # few rows of x, converted on the way: 2, 4, 8 waves on the long axis
    (12310, 768, 3), (12310, 288, 13), (6161, 512, 7), (6161, 800, 5), (37, 1024, 1), (37, 544, 2), (37, 256, 5), (37, 288, 7),
    # few rows, prepared
    (37, 1536, 13), (37, 1568, 13), (37, 2560, 7), (37, 2592, 7), (37, 4096, 5), (37, 4128, 5), (37, 4352, 3), (37, 4128, 3),
    (37, 2048, 7), (515, 2080, 7), (12310, 1536, 13),
    # many rows: tiles of 32 whose steps hold all parts, of 128 with a step for each
    (37, 256, 17), (301, 288, 33), (37, 768, 29), (37, 1056, 65), (12310, 256, 512), (6161, 288, 1001), (515, 256, 5000), (515, 288, 5000),
    (515, 2560, 3001), (515, 2592, 3001), (9001, 2560, 101), (9001, 2592, 101),
    (2051, 256, 7001), (2051, 288, 7001), (515, 8192, 3001), (515, 8224, 3001), (301, 8192, 3001), (301, 8224, 3001),
]


def form(call, plan):
    """What decides between the kernels of `call` (weights, mx, rotate, bf16, rows, cols, tokens)."""
    weights, mx, _, _, _, k, _ = call
    together = k // (32 if mx else 16) % 4 == 0  # scale bytes in one load
    if plan.kernel == "few":
        return "few", weights, mx, plan.parts, plan.tokens, plan.prepared, plan.waves_k, together
    return "many", weights, mx, plan.parts, plan.tokens, plan.splits > 1, together
