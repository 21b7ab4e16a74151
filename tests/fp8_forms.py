"""Shapes of the FP8 product by the form of the launch that they take on the 148
SMs of a B200 (csa_debug_fp8_form), for the tests that go through every form."""

CLUSTER, TILES, PAIR = 0x1000, 0x2000, 256

# form, n_out, k_in, groups, n_tok: at least 3 tokens, two row blocks and three column blocks
SHAPES = [
    (16, 260, 400, 1, 3),
    (16, 512, 4 * 400, 4, 9),
    (16 | CLUSTER, 300, 4096, 1, 5),
    (16 | TILES, 260, 400, 1, 300),
    (16 | CLUSTER | TILES, 320, 2056, 1, 40),
    (32, 20000, 264, 1, 30),
    (32 | CLUSTER, 2368, 7168, 1, 30),
    (64, 9600, 1160, 1, 60),
    (64 | CLUSTER, 2368, 7168, 1, 52),
    (64 | CLUSTER, 4096, 16 * 4096, 16, 48),
    (128, 9500, 1160, 1, 70),
    (128 | TILES, 2368, 1536, 1, 100),
    (128 | TILES, 8001, 264, 1, 1000),
    (128 | CLUSTER, 2368, 7168, 1, 90),
    (128 | CLUSTER | TILES, 750, 8496, 1, 639),
    (PAIR, 8001, 1032, 1, 450),
    (PAIR, 9456, 1160, 1, 513),
    (PAIR, 6400, 10 * 528, 10, 780),
]

# the kernels there are
FORMS = {16, 16 | CLUSTER, 16 | TILES, 16 | CLUSTER | TILES, 32, 32 | CLUSTER, 64, 64 | CLUSTER, 128, 128 | CLUSTER, 128 | TILES,
         128 | CLUSTER | TILES, PAIR}


def name(shape):
    form, n_out, k_in, groups, n_tok = shape
    kind = "pairs" if form == PAIR else f"{form & 0xFFF}" + ("-cluster" if form & CLUSTER else "") + ("-tiles" if form & TILES else "")
    return f"{kind}-{n_tok}x{n_out}x{k_in}" + (f"-{groups}" if groups > 1 else "")
