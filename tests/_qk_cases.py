"""Calls of the norms of queries and keys that are taken 16 tokens a workgroup (8 where a row takes 32 lanes), and some whose
backward workgroups take more than 64 steps: B, T, Hq, Hk, d, rot."""
MANY = [(2, 8193, 1, 1, 8, 8), (3, 5467, 3, 2, 32, 24), (2, 8201, 2, 1, 64, 64), (2, 8197, 4, 2, 64, 32), (5, 3301, 2, 2, 104, 40), (2, 8195, 3, 1, 128, 128),
        (2, 8199, 2, 2, 128, 0), (17, 1033, 1, 2, 256, 256), (3, 5471, 2, 1, 200, 64), (1, 16384, 1, 1, 16, 16)]
LONG = [(2, 270001, 1, 1, 8, 8), (1, 40009, 11, 1, 136, 64), (3, 15001, 40, 8, 40, 40), (2, 80003, 12, 1, 64, 64), (2, 90001, 2, 1, 256, 128)]
