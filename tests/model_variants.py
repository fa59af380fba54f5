"""Sizes that, with the sizes of the operators' own tests, reach every variant of the model
operators' kernels: the e4m3 product's few rows and its tiles, with and without shares of k,
in rows of whole 16-byte chunks and others; layer norm in every number of threads a row, few
rows and many; distillation in whole rows and in segments.  test_model_launches.py holds them
to that on the host, test_gpu_model_variants.py runs them."""

# M, N, K
FP8 = [(20, 40, 160), (70, 40, 160), (70, 40, 2064), (130, 16400, 160), (20, 8200, 8208), (70, 16400, 160),
       (2100, 40, 8208), (70, 33000, 160), (70, 8200, 8208), (200, 33000, 160), (200, 16400, 8208),
       (20, 40, 41), (70, 40, 41), (70, 40, 4099), (130, 16400, 41), (20, 8200, 4099), (70, 16400, 41),
       (70, 4300, 4099), (70, 33000, 41), (70, 16400, 4099), (200, 33000, 41)]
# rows, columns
NORM = [(800, 4000), (1030, 1024), (769, 8192), (1537, 100), (1540, 520), (1600, 1000), (1536, 2040), (1600, 2000)]
# rows, vocabulary, entries
DISTILL = [(1, 65537, 64), (100, 70001, 9), (127, 131072, 5), (127, 200000, 3), (127, 400001, 33), (130, 70000, 64),
           (128, 65537, 2), (3, 524288, 64)]


def calls(blocks, products, norms, distills):
    """These and the given lists as input lines of the launch recorder, in every type."""
    out = []
    for t in range(3):
        out += ["blocks %d %d %d %d" % (t, *s, r) for s in blocks for r in (1, 128)]
        out += ["fp8 %d %d %d %d %d" % (t, *s, s[2] % 16 == 0) for s in products + FP8]
        for w in {0, t}:
            out += ["norm %d %d %d %d" % (t, w, *s) for s in norms + NORM]
            out += ["norm_vjp %d %d %d %d %d" % (t, w, *s, o) for s in norms + NORM for o in (1, 2, 3)]
        out += ["distill %d %d %d %d %d" % (t, *s, g) for s in distills + DISTILL for g in (0, 1)]
        out += ["distill_vjp %d %d %d %d" % (t, *s) for s in distills + DISTILL]
    return out
