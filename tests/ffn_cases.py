"""Sizes that reach every kernel of the FFN operators' rules (csrc/ffn_rules.h):
the GPU tests run them, a CPU test asks the rules which kernel each reaches, so
that a change of a rule cannot leave a kernel untested unnoticed."""

# choice, M, N, K
Q8 = ([("kQ8Rows16", 16, 264, 1040), ("kQ8Rows32", 17, 264, 1040), ("kQ8Rows64", 64, 264, 1040)] +
      [("kQ8Rows%dWide" % (16 if m <= 16 else 32 if m <= 32 else 64), m, n, 272)
       for m in (1, 16, 17, 32, 33, 64) for n in (8192, 8200, 8209)] +
      [("kQ8Tile64", 65, 264, 272), ("kQ8Tile64x128Deep", 3300, 264, 272), ("kQ8Tile128Deep", 6000, 264, 272),
       ("kQ8Tile64x128", 700, 6152, 272), ("kQ8Tile128", 6000, 1034, 272), ("kQ8Tile256", 2100, 4104, 272)])

# choice, rows, columns
QUANT = ([("kQuantWave", r, c) for r in (256, 300) for c in (1000, 1792, 2047, 2048)] +
         [("kQuant2048", 255, 2047), ("kQuant2048", 3, 2041), ("kQuant8192", 300, 2049), ("kQuant8192", 2, 8185),
          ("kQuant16384", 2, 8193), ("kQuant16384", 3, 16384), ("kQuantTwice", 2, 16385)])

# choice, rows of each expert, N, K (of NN and NT)
ROWS = [("kRows256", [3300, 1, 2900], 2056, 520), ("kRows128x256", [90, 0, 141, 80] * 10, 1032, 1032),
        ("kRows128", [90, 0, 141, 80] * 10, 1032, 72), ("kRows128Deep", [90, 0, 141, 80] * 10, 520, 72),
        ("kRows64x128", [900, 0, 3, 1100], 264, 72), ("kRowsStream", [40, 0, 1, 90], 136, 264)]

# large tiles, several parts, rows of each expert, N, K (of TN)
MANY = [20, 0, 41, 3, 64, 0, 0, 130]
TN = [(True, False, MANY * 32, 264, 264), (True, False, MANY * 21 + [700, 0, 65], 520, 264),
      (True, False, [900, 0, 3, 1500, 1200, 0, 40, 350], 1288, 1288), (False, False, MANY, 264, 520),
      (False, True, [5000, 0], 136, 264), (False, True, [5000, 70], 136, 264), (False, True, [0, 4100, 1, 900], 72, 200)]
