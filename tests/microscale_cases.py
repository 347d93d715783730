"""Shapes (m, n, k) of products of real values. By format and result type they take every kernel that any shape takes, with its sum
whole and in parts (asserted on the CPU in test_microscale_choice.py)."""
REAL = [(1, 2048, 4096), (2, 1001, 1040), (4, 518, 301), (16, 4096, 2048), (17, 124, 327), (30, 4096, 1500), (34, 117, 2456), (36, 101, 307),
        (60, 3000, 700), (300, 1025, 4100), (1403, 134, 5930), (1500, 2600, 1000), (3350, 1180, 400), (4131, 147, 649), (4195, 393, 8450),
        (4374, 411, 4858), (4387, 2516, 308), (4769, 791, 7526), (11114, 133, 12046)]
FORMATS = [(8, 8), (4, 4), (8, 4)]
