"""One call at least of every compiled kernel of the products and of the activation's gradient:
what tests/test_mm_dispatch_cpu.py holds to be all of them, and tests/test_gpu_mm_variants.py
runs against the oracle."""

FMTS = ("44", "84", "88")

# (rows of the experts, or of the one matrix; n; k; operands; fp32; first byte of E8M0 scales; grouped)
PRODUCTS = []
for fp32 in (False, True):
    for fmt in FMTS:
        # few rows: 16, 32 and 64 columns of a workgroup, and 16 waves for a long contraction
        PRODUCTS += [([13], 300, 640, fmt, fp32, 0, False), ([3, 0, 12, 1], 130, 384, fmt, fp32, 0, True),
                     ([5], 12300, 384, fmt, fp32, 0, False), ([2, 0, 7] + [1] * 60, 270, 256, fmt, fp32, 0, True),
                     ([4], 24600, 256, fmt, fp32, 0, False), ([1, 2, 0] * 60, 270, 256, fmt, fp32, 0, True)]
        PRODUCTS += [([m], 300, k, fmt, fp32, 0, False) for m in (1, 13) for k in (8320, 14336)]
        PRODUCTS += [([2, 0, 9], 130, 8320, fmt, fp32, 0, True)]
        # 17 to 64 rows
        PRODUCTS += [([33], 264, 640, fmt, fp32, 0, False), ([20], 264, 8320, fmt, fp32, 0, False)]
        # tiles of 64, 128 and 256
        sides = [([130], 1100, False), ([700], 4200, False), ([4130], 4100, False), ([130, 0, 33, 257], 264, True),
                 ([300, 5, 0, 700], 4200, True), ([2000, 0, 1030, 257, 900], 4160, True)]
        PRODUCTS += [(c, n, 640, fmt, fp32, 0, g) for c, n, g in sides]
        if fmt == "44":
            PRODUCTS += [([13], 300, 8224, fmt, fp32, 0, False), ([2, 0, 9], 130, 8224, fmt, fp32, 0, True)]
            PRODUCTS += [(c, n, 288, fmt, fp32, 0, g) for c, n, g in sides]
            PRODUCTS += [([200], 264, k, fmt, fp32, 0, False) for k in (8224, 14304)]
        if fmt != "88":
            PRODUCTS += [(c, n, 384, fmt, fp32, 1, g) for c, n, g in sides]
        PRODUCTS += [([200], 264, 14336, fmt, fp32, 0, False)]

# (tokens of the experts, n, k, fp32): tiles of 64, 128 and 256
WGRADS = [(c, n, k, fp32) for fp32 in (False, True)
          for c, n, k in (([130, 33, 0, 257], 130, 328), ([131, 301], 700, 4200), ([256, 128], 700, 4200),
                          ([130, 33, 0, 257], 700, 4200))]

# (rows of the groups, n, activation, fp32, bias gradient, grouped): blocks of 64, 16 and 128 rows
ACT_GRADS = [(c, n, act, fp32, bias, grouped) for fp32 in (False, True) for act in ("gelu", "swiglu")
             for n in (24, 34) for c, bias, grouped in (([40], True, False), ([40], False, False), ([9, 0, 30], True, True),
                                                        ([300], True, False), ([70, 0, 1, 200], True, True))]
ACT_GRADS += [(c, n, act, False, True, grouped) for n, act in ((24, "swiglu"), (26, "gelu"))
              for c, grouped in (([132000], False), ([0, 70000, 129, 1, 0, 128, 61742], True))]
ACT_GRADS += [([0, 40001, 127, 25872], 520, "silu", False, True, True)]
