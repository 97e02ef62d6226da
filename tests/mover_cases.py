"""Sizes that reach the large-call kernels of routing, row movement and AdamW.
test_mover_cases_cpu.py holds them to the rules of the sources; the GPU tests
run them."""

# T, E, top_k: more than the tokens that a wave chooses for one at a time, with
# every register count of the rows of 16 lanes (64, 128, 256 and 512 experts)
ROUTES = [(1100, 64, 6), (1025, 65, 1), (1500, 100, 10), (1100, 256, 8), (2049, 255, 32), (1200, 300, 17), (1300, 512, 32)]

# T, top_k, columns, elements of padding: sorted rows of 32 MB and more, in whole
# pieces of 64 bytes, in BF16 (and so in FP32)
STREAMED = [(530, 8, 4096, 0), (4500, 4, 1024, 0), (1100, 17, 1056, 32), (16400, 32, 32, 0)]

# element counts of one AdamW call of more than 4 million: odd last blocks, tensors
# below and above one workgroup's four blocks of four waves
ADAMW = [(1 << 22) + 5, 1, 4095, 4096, 4097, 255, 257, 0, 700001]
