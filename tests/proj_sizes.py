"""Sizes of the 8-bit projection by the kernel that takes them: {(y's type, rows of y of a workgroup): [(M, N, K)]}.

One block of K, whole and cut; a cut last block; more than 16 and more than 32 blocks (the tiles hold the scales of 16 blocks at a
time); M and N whole and cut.  test_proj_kernels.py holds the library's choice to these numbers, so that a kernel that a new choice
leaves without a size is missed there."""

FEW = {16: [(7, 1000, 16), (33, 300, 144), (45, 1000, 1040), (100, 700, 2064), (64, 64, 4368)],
       32: [(130, 900, 16), (24, 5000, 144), (300, 500, 1040), (360, 533, 2064), (130, 900, 4368)],
       64: [(1024, 960, 128), (1000, 1000, 144), (1000, 1000, 272), (1024, 960, 2064), (1000, 1000, 4368)]}
SIZES = {("bf16", k): v for k, v in FEW.items()} | {("f32", k): v for k, v in FEW.items()} | {
    ("bf16", 128): [(15715, 1272, 32), (15715, 1272, 128), (2800, 2740, 144), (3000, 2900, 256), (2190, 2440, 272), (1800, 1810, 2064),
                    (2048, 2048, 2048), (800, 4096, 4096), (1024, 5152, 2048), (1700, 1700, 4368)],
    ("f32", 128): [(2800, 2740, 16), (3200, 2944, 128), (2190, 2440, 144), (2048, 2048, 272), (1800, 1810, 2064), (2048, 2048, 2048),
                   (1700, 1700, 4368)],
    ("bf16", 256): [(3600, 3500, 16), (3584, 3584, 128), (3600, 3500, 272), (3585, 3600, 2064), (3600, 3500, 4368)]}
