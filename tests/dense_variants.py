"""Sizes that reach every variant of the dense products' kernels: few rows (one to four groups
of 16, one and two groups of columns a workgroup) and tiles of 64, 128 and 256 rows, each
over several steps with a last one that is not whole, with and without shares of k, in rows
of whole 16-byte chunks and others.  test_dense_launches.py holds them to that on the host,
test_gpu_dense_variants.py runs them."""

# M, N, K
INT8 = [(5, 100, 208), (17, 40, 128), (40, 40, 1040), (5, 100, 207), (17, 40, 129), (40, 40, 1041),
        (9, 16400, 96), (17, 16400, 160), (33, 16400, 96), (9, 16400, 97), (17, 16400, 161), (64, 16384, 95),
        (100, 1000, 528), (100, 300, 4112), (100, 300, 4099), (300, 16400, 272), (300, 16400, 271),
        (500, 8200, 4112), (2100, 4300, 528), (2100, 4300, 1008), (2100, 4300, 1001), (1100, 3400, 16400),
        (2560, 2560, 32784)]
# M, F, K
GATED = [(5, 100, 104), (20, 100, 520), (40, 100, 72), (5, 100, 103), (20, 100, 521), (40, 100, 71),
         (100, 700, 520), (100, 130, 4104), (100, 130, 1001), (300, 8200, 264), (300, 8200, 263), (2100, 2150, 520),
         (2100, 2150, 1001), (1100, 1700, 8200), (2560, 1280, 16392)]
VJP = [(64, 264, 520), (100, 1000, 264), (100, 1000, 263), (8200, 40, 4104), (4100, 96, 2056), (4100, 300, 2055),
       (64, 33000, 8200), (128, 17000, 8200), (128, 17000, 8199), (2100, 2100, 4104), (200, 33000, 4104)]
DTYPES = ["float32", "bfloat16", "float16"]
HALVES = ["bfloat16", "float16"]
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]


def calls():
    """All of them as input lines of the launch recorder."""
    out = []
    for t, dtype in enumerate(DTYPES):
        out += ["int8 %d %d %d %d %d" % (t, *s, s[2] % 16 == 0) for s in INT8]
    for dtype in HALVES:
        t = DTYPES.index(dtype)
        for act in range(len(ACTS)):
            out += ["gated %d %d %d %d %d %d" % (t, *s, s[2] % 8 == 0, act) for s in GATED]
            out += ["vjp %d %d %d %d %d %d" % (t, *s, s[2] % 8 == 0, act) for s in VJP]
    return out
