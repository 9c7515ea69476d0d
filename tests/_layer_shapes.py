"""Sizes that take the layer operators through each way of laying a call out, with the layout they are here for.
tests/test_layer_plan.py holds the layouts on the host, tests/test_gpu_layer_paths.py runs the sizes."""
from __future__ import annotations

# lens, D, packed, bytes an element, (chunk, workgroups' units, channel tiles): chunk 0 is whole sequences a workgroup
SCANS = [
    ([700] * 8, 1024, False, 2, (0, 8, 32)),
    ([700] * 8, 1024, False, 4, (0, 8, 64)),
    ([768] * 8, 1023, False, 2, (0, 8, 64)),  # one channel a thread
    ([700, 300, 1, 0, 513, 256, 600, 257], 4096, True, 2, (0, 8, 128)),
    ([700, 300, 1, 0, 513, 256, 600, 257], 4096, True, 4, (0, 8, 256)),
    ([5000], 2048, False, 2, (512, 10, 64)),
    ([5000], 2048, False, 4, (1024, 5, 128)),
    ([4000, 0, 900, 1, 2500], 2048, True, 2, (768, 15, 64)),
    ([4000, 0, 900, 1, 2500], 2048, True, 4, (1280, 11, 128)),
]

# M, D, F, bytes, kernels of the forward, of dx and of the weights' gradients
FFNS = [
    (5558, 1864, 2199, 2, "256 256 256"),
    (5395, 1968, 1054, 2, "256 256 256/3"),
    (875, 2320, 5389, 2, "256 256/3 128"),
    (4322, 16, 1358, 2, "128 128/5 128/17"),
    (637, 12, 6369, 4, "128 64/25 128/5"),
    (81, 280, 5670, 4, "64 64/30 128"),
]

# N, D, V, bytes, kernel of the forward, then (width, dl, dW, dx) of each kind of piece
CES = [
    (4119, 1888, 5903, 2, "256 5903 256 256 128"),
    (5486, 1808, 2226, 2, "256 2226 256 256/3 256"),
    (3608, 1080, 5442, 2, "128 5442 128 128 256/3"),
    (2030, 16, 6871, 2, "128 6871 128 128/8 128/27"),
    (5580, 660, 127, 4, "64 127 64 64/30 128"),
    (10, 24, 33001, 2, "rows1x4 33001 rows1x4 128 64/31"),
    (30, 24, 33001, 2, "rows2x4 33001 rows2x4 128 64/31"),
    (60, 24, 33001, 2, "rows4x4 33001 rows4x4 128 64/31"),
    (30, 136, 33001, 4, "rows2x4 33001 rows2x4 64 64/32"),
    (60, 136, 33001, 4, "rows4x4 33001 rows4x4 64 64/32"),
]
