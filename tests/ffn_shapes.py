"""Shapes of the products and gated blocks whose kernel and tile are part of what a test is for: (rows, columns,
tokens), and what q8_mx_plan.h answers for them in every format, with whether a workgroup has several tiles."""

# One token block and several; tiles of every height; 30 tokens are two tiles of 16, 45 three.
PRODUCTS = [
    ((8353, 1056, 30), "columns 2", False), ((16529, 1056, 45), "columns 4", False), ((33001, 1056, 48), "columns 5", False),
    ((40993, 1056, 61), "columns 4", True), ((65537, 1056, 61), "columns 5", True), ((40993, 544, 30), "columns 4", True),
    ((40, 1056, 20000), "columns 2", True), ((2113, 544, 300), "columns 2", False), ((100, 544, 9000), "columns 4", False),
    ((300, 544, 40), "columns 1", False), ((7001, 1184, 515), "wide 2", False), ((7001, 1184, 1200), "wide 4", False),
]
# fp32 rows alone.
GATED = [
    ((4193, 1056, 20), "columns 2", False), ((8353, 1056, 30), "columns 4", False), ((16529, 544, 61), "columns 5", False),
    ((33001, 544, 33), "columns 5", True), ((20513, 1056, 61), "columns 4", True), ((33001, 544, 30), "columns 5", True),
    ((300, 544, 40), "columns 1", False), ((5153, 544, 200), "wide 2", False), ((4095, 544, 1900), "wide 4", False),
]
# Quantised rows, alone and with fp32 rows.
QUANTISED = [
    ((4096, 544, 20), "columns 2", False), ((8352, 1056, 61), "columns 4", False), ((16512, 1056, 40), "columns 4", True),
    ((17408, 1056, 64), "columns 4", True), ((2112, 544, 200), "columns 4", False), ((17408, 544, 20), "columns 4", True),
    ((8352, 544, 100), "wide 2", False), ((16512, 160, 200), "wide 4", False),
]
