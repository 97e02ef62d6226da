"""Sizes that reach what large calls of layer norm, dropout and the recurrence run:
several rounds of rows, several tiles of a span, accesses past the caches.
test_block_cases_cpu.py holds them to the library's plans and the sources' rules;
the GPU tests run them."""

# sequences, rows of each, channels: spans of several tiles, the last one shorter or
# not, and its last tile not whole; one axis, several, and the most spans
SPANS = [(1, 1100, 8192), (1, 600, 16384), (3, 700, 3000), (1, 40000, 72)]

# offsets, rows, channels: the same for packed sequences, with borders inside, at and
# next to the spans' (384 and 768 of the first), empty sequences there, and rows of nobody
PACKED_SPANS = [([0, 100, 384, 384, 500, 767, 769, 1050, 1050], 1100, 8192), ([0, 1100], 1100, 8192),
                ([0, 384, 768, 768, 1100], 1100, 8192), ([0, 5, 20000, 20000, 20256, 39990], 40000, 72)]

# type, sequences, rows of each, channels: elements just below and above those from
# which on accesses go past the caches; whole sequences, spans, and many short ones
STREAMED = [("bf16", 32, 508, 1032), ("bf16", 3, 5419, 1032), ("bf16", 64, 255, 1032), ("bf16", 1024, 16, 1032),
            ("f32", 16, 508, 1032), ("f32", 11, 739, 1032), ("f32", 40, 204, 1032)]
# type, offsets, rows, channels
PACKED_STREAMED = [("bf16", [0, 1, 4000, 4000, 9111, 16250], 16300, 1032), ("f32", [0, 3333, 3333, 8192, 8200], 8200, 1032)]

# type of the output, rows, columns, elements of padding: dropout, likewise; as one
# long row the groups of eight fill no whole number of its pieces of 512
DROPOUT = [("bf16", 4087, 4104, 0), ("bf16", 4099, 4104, 0), ("bf16", 4099, 4104, 32),
           ("f32", 2043, 4104, 0), ("f32", 2051, 4104, 0), ("f32", 2051, 4104, 32)]

# rows, columns: three rounds of rows or more of every cut of the row, the last not whole
NORM = [(131077, 64), (65541, 128), (32773, 256), (16389, 512), (16389, 1024), (4103, 1544), (4103, 2048), (4103, 2056),
        (4103, 4096), (4103, 4104), (4103, 8192), (2051, 8200), (2051, 16384)]
ADD_NORM = [(131077, 64), (65541, 128), (32773, 256), (16389, 512), (16389, 1024), (8197, 2048), (4101, 4096), (4101, 5120),
            (4101, 8192), (4101, 16384)]
NORM_GRADIENT = [(98311, 64), (49159, 128), (24583, 256), (12295, 512), (3847, 1032), (3079, 2048), (1543, 4096),
                 (775, 5120), (775, 8192), (775, 8200), (775, 16384)]


def norm_round(H, many, add):
    """Rows of the forward pass at once: of many rows, of a sum."""
    chunks = (1 if H <= 512 else 2) if not many or H <= 1024 or add else (4 if H <= 2048 else 8)
    waves = -(-H // (512 * chunks))
    sets = max(1, (8 if chunks > 2 and H > 4096 else 4) // waves)
    return sets * (64 // norm_lanes(H)) * (512 if chunks > 2 else 2048)


def norm_gradient_round(H):
    """The same of the gradient."""
    waves = -(-H // (512 if H <= 8192 else 1024))
    return 16 // waves * (64 // norm_lanes(H)) * 256


def norm_lanes(H):
    return 8 if H <= 64 else 16 if H <= 128 else 32 if H <= 256 else 64
