"""Shapes of the linear operators, each with the kernel that the plan sends its
forward product and its two gradients to: tile shape, splits of the summed
index and staged tiles of it per split (a * where an operand is laid out anew
first).  The plan is checked on the CPU (``test_linear_plan.py``), the results
on the GPU (``test_gpu_linear_paths.py``)."""

# (N, D, F, values between rows, forward, dX, dW)
PATHS = [
    # 256 x 256 tiles everywhere; the forward's last columns and the input
    # gradient's last k are no whole runs
    (2904, 2904, 2905, 0, "wide:1:46", "wide:1:46", "wide:1:46"),
    # the same on operands laid out anew: the gradients' last columns too
    (2904, 2901, 2905, 0, "wide*:1:46", "wide*:1:46", "wide*:1:46"),
    # an odd number of tiles of k on 256 x 256; 128 x 128 in pairs; four stages, split
    (20011, 264, 520, 0, "wide:1:5", "paired:1:9", "deep:16:20"),
    # pairs through many tiles of k
    (2304, 2304, 2304, 0, "paired:1:36", "paired:1:36", "paired:1:36"),
    # four stages, unsplit
    (1300, 1304, 1303, 0, "deep:1:21", "deep:1:21", "deep:1:21"),
    # a decode batch: four stages, split, for forward and input gradient
    (17, 4096, 4096, 0, "deep:8:8", "deep:8:8", "paired:1:1"),
    (128, 4096, 4096, 0, "deep:4:16", "deep:4:16", "paired:1:2"),
    # unaligned rows through registers: pipelined steps, unsplit and split
    (400, 401, 402, 0, "unaligned:1:7", "unaligned:1:7", "unaligned:1:7"),
    (1300, 515, 1300, 3, "unaligned:1:9", "unaligned:4:6", "unaligned:4:6"),
    (320, 2001, 2000, 0, "unaligned:4:8", "unaligned:4:8", "unaligned:1:5"),
]
