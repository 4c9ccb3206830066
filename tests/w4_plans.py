"""The launches of the 4-bit products that the tests force, and the cases they run on; no GPU is needed to read it."""

# column tiles a wave, waves along the columns, waves along K of the streaming kernel
STREAM_SHAPES = [(1, 1, 4), (1, 1, 8), (1, 2, 2), (1, 2, 4), (1, 4, 2), (2, 1, 2), (2, 1, 4), (2, 1, 8), (2, 2, 2),
                 (2, 2, 4), (2, 4, 2)]

# M, K, N, K splits: one to four live row tiles alone and behind full blocks, odd counts of chunks and columns
TILED_CASES = [(1, 128, 16, (1,)), (16, 384, 80, (1, 2)), (17, 640, 272, (1, 4)), (33, 1152, 144, (1, 8)),
               (48, 256, 528, (1, 2)), (49, 896, 64, (1, 7)), (64, 1024, 1040, (1, 2, 4, 8)), (65, 1408, 96, (1, 3)),
               (150, 2176, 208, (1, 5)), (220, 640, 320, (1, 2)), (600, 256, 144, (1,))]

# M, K, N, K split: slices loaded whole, and longer than the loads ahead with one LDS segment and with several,
# for one row tile and for two
STREAM_CASES = [(1, 256, 48, 1), (5, 512, 112, 1), (2, 9088, 48, 1), (16, 4480, 80, 1), (16, 9600, 48, 1), (4, 1024, 64, 2),
                (16, 4992, 80, 3), (11, 9984, 32, 2), (17, 256, 64, 1), (32, 2304, 48, 1), (33, 5120, 80, 1),
                (40, 1024, 48, 4), (20, 9600, 48, 2), (75, 640, 32, 1), (16, 12800, 32, 2), (20, 4352, 48, 2)]

# experts' row counts: every count of live row tiles, several blocks, none
TILED_EXPERT_COUNTS = [0, 1, 16, 17, 33, 48, 64, 65, 0, 150, 5]

# experts' row counts, K, N, topk: one row tile and two, whole slices, one segment and several
STREAM_EXPERTS = [([0, 1, 5, 16, 17, 0, 12], 256, 96, 2), ([3, 0, 16, 9], 4480, 64, 4), ([20, 1, 2, 0], 9600, 32, 3),
                  ([33, 17, 0, 60, 20], 256, 96, 2), ([33, 17, 60], 2304, 64, 1), ([40, 0, 31], 4992, 32, 5)]
