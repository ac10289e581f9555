"""Shapes of the linear layer on 8-bit operands, each with the kernel that the plan
sends it to for 16-bit and for fp32 outputs: tile shape, splits of the summed
index and blocks of 128 of it per split.  The plan is checked on the CPU
(``test_linear_fp8_plan.py``), the results on the GPU
(``test_gpu_linear_fp8_paths.py``)."""

# (N, D, F, 16-bit, fp32)
PATHS = [
    # 256 x 256 tiles: a whole number of them, an even one of blocks of k
    (4096, 512, 4096, "wide:1:4", "paired:1:4"),
    # the last rows, columns and block of k cut short, many blocks of k
    (2050, 2050, 4100, "wide:1:17", "paired:1:17"),
    (3000, 384, 5001, "wide:1:3", "paired:1:3"),
    (20011, 272, 520, "wide:1:3", "paired:1:3"),
    (5001, 528, 3003, "wide:1:5", "paired:1:5"),
    # split
    (4281, 21060, 171, "wide:15:11", "paired:4:42"),
    # 128 x 128 in pairs, unsplit and split
    (4133, 515, 1001, "paired:1:5", "paired:1:5"),
    (2304, 2304, 2304, "paired:1:18", "paired:1:18"),
    (27, 1341, 28, "paired:6:2", "paired:6:2"),
    (4100, 16384, 33, "paired:8:16", "paired:8:16"),
    # four stages, unsplit and split
    (1300, 2300, 1303, "deep:1:18", "deep:1:18"),
    (700, 1300, 2000, "deep:1:11", "deep:1:11"),
    (128, 4096, 4096, "deep:4:8", "deep:4:8"),
]
