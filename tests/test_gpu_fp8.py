"""GPU parity of the FP8 projection product (csa_gemm_fp8) against the fp64
oracle: quantised weights and tokens code by code, products of odd, ragged and
grouped shapes in every form of the launch, several output segments, batch
invariance, blocks that are not finite, the extremes of the scales, streams
and captured graphs."""
import numpy as np
import pytest

from oracle import csa_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return cuda_lib


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def _inputs(n_out, k_in, groups, n_tok, seed, spread=1.0):
    """Tokens with channels of very different size, a real weight, and the
    weight's codes and scales by the oracle."""
    rng = np.random.default_rng(seed)
    loud = np.exp(spread * rng.standard_normal(k_in))
    x = _bf16(rng.standard_normal((n_tok, k_in)) * loud)
    w = _bf16(rng.standard_normal((n_out, k_in // groups)) / np.sqrt(k_in // groups))
    codes, scales = O.fp8_quantize_blocks(w.double().numpy(), rows=128)
    return x, w, codes, scales


def _linear(codes, scales, groups=1):
    from compressed_sparse_long_hca_b200.api import LinearFP8
    return LinearFP8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), groups=groups)


def _check(y, x, codes, scales, groups, bf16=False):
    """|y - ref| <= (blocks * 8 + 32) 2^-23 sum_k |x_k w_k|: every product of
    codes is exact, a step of 32 products and its addition to the running sum
    round at most a few times, and the partial sums are no larger than the sum
    of magnitudes; a BF16 output adds half a step, 2^-8 of the result."""
    xc, xs = O.fp8_quantize_blocks(x.double().numpy(), groups=groups)
    xd, wd = O.fp8_dequantize_blocks(xc, xs, groups=groups), O.fp8_dequantize_blocks(codes, scales, rows=128)
    ref, mag = O.grouped_linear(xd, wd, groups), O.grouped_linear(np.abs(xd), np.abs(wd), groups)
    blocks = -(-(x.shape[1] // groups) // 128)
    bound = (8 * blocks + 32) * 2.0 ** -23 * mag
    if bf16:
        bound = bound * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= bound), f"{int((err > bound).sum())} outside; worst {float((err / (mag + 1e-300)).max()):.3e}"


# n_out, k_in, groups, n_tok
SHAPES = [
    (1, 8, 1, 1),                 # the smallest
    (72, 200, 1, 5),              # ragged everything, one row tile
    (129, 136, 1, 33),            # one row and eight columns beyond a block
    (260, 256, 1, 1),             # the tiny layer's first projection
    (300, 1160, 1, 64),           # K parts that begin inside a scale chunk
    (2368, 7168, 1, 4),           # few row tiles: many K parts
    (2368, 1032, 1, 65),          # 128-token tiles
    (1000, 2056, 1, 200),         # 224-token tiles
    (257, 640, 1, 450),           # three token tiles
    (20000, 264, 1, 231),         # every tile in one item, several items per CTA
    (38000, 8, 1, 3),             # one K block: tiles follow each other at every block
    (2048, 4096, 16, 7),          # grouped
    (512, 4 * 72, 4, 130),        # grouped, the last block of each group short
    (6400, 10 * 264, 10, 520),    # pairs of SMs: grouped, tiles that begin inside a row tile
    (9100, 1160, 1, 513),         # pairs of SMs: two K parts, one token beyond two tiles, a ragged last tile
]


@pytest.mark.parametrize("n_out,k_in,groups,n_tok", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_product_matches_the_oracle(n_out, k_in, groups, n_tok, bf16):
    from compressed_sparse_long_hca_b200.api import LinearFP8
    x, _, codes, scales = _inputs(n_out, k_in, groups, n_tok, n_out + k_in)
    lin = _linear(codes, scales, groups)
    # rows beyond the call's tokens stay as they were
    y = torch.full((n_tok + 2, n_out), 777.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    assert lin(x.cuda(), y[:n_tok]) is not None
    LinearFP8.check_device_error()
    assert bool((y[n_tok:] == y.new_tensor(777.0)).all())
    _check(y[:n_tok], x, codes, scales, groups, bf16)


def test_weight_quantisation_code_by_code():
    from compressed_sparse_long_hca_b200.api import LinearFP8, quantize_fp8_weight
    rng = np.random.default_rng(2)
    w = rng.standard_normal((300, 520)) * np.exp(4 * rng.standard_normal((300, 520)))
    w[:128, :128] = 0                                        # an empty block
    w[130, 130] = 448 * 2.0 ** 5                             # on the border of two scales
    w[131, 300] = 452 * 2.0 ** 60                            # just beyond one, far from 1
    w[256:, 512:] *= 1e-38                                   # subnormal in BF16
    w = _bf16(w)
    codes, scales = quantize_fp8_weight(w.cuda())
    want_c, want_s = O.fp8_quantize_blocks(w.double().numpy(), rows=128)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, want_c)
    x = _bf16(rng.standard_normal((3, 520)))
    y, z = torch.empty((3, 300), device="cuda"), torch.empty((3, 300), device="cuda")
    LinearFP8.quantize(w.float().numpy())(x.cuda(), y)        # from a host array
    _linear(want_c, want_s)(x.cuda(), z)
    assert torch.equal(y, z)
    LinearFP8.quantize(w.view(torch.int16).numpy().view(np.uint16))(x.cuda(), z)      # BF16 bit patterns
    assert torch.equal(y, z)


@pytest.mark.parametrize("n_tok", [1, 40, 300])
def test_token_quantisation_code_by_code(n_tok):
    """With an identity weight the outputs are the dequantised tokens, exact
    in fp32: every code and every scale is seen, at magnitudes from BF16's
    subnormals to near its largest, ties and borders among them."""
    rng = np.random.default_rng(n_tok)
    k = 384
    x = rng.standard_normal((n_tok, k)) * np.exp2(rng.integers(-120, 110, (n_tok, k // 128))).repeat(128, 1)
    x[0, :128] = np.linspace(-448, 448, 128)
    x[-1, 128:256] = 0
    x[0, 256] = 2.0 ** -133
    x[0, 257:] = 0
    x = _bf16(x)
    eye = np.eye(k)
    codes, scales = O.fp8_quantize_blocks(eye, rows=128)
    y = torch.empty((n_tok, k), device="cuda")
    _linear(codes, scales)(x.cuda(), y)
    want = O.fp8_dequantize_blocks(*O.fp8_quantize_blocks(x.double().numpy()))
    keep = np.abs(want) >= 2.0 ** -126                       # the tensor core's sums may drop fp32 subnormals
    assert np.array_equal(y.double().cpu().numpy()[keep], want[keep])
    assert np.all(np.abs(y.double().cpu().numpy()[~keep]) <= 2.0 ** -126)


@pytest.mark.parametrize("n_out,k_in,groups", [(2368, 7168, 1), (9216, 1024, 1), (300, 200, 1), (2048, 4096, 16)])
def test_a_tokens_bits_do_not_depend_on_its_batch(n_out, k_in, groups):
    from compressed_sparse_long_hca_b200.api import LinearFP8
    x, w, _, _ = _inputs(n_out, k_in, groups, 700, 11)
    lin = LinearFP8.quantize(w, groups=groups)
    xd = x.cuda()
    base = torch.empty((700, n_out), device="cuda")
    lin(xd, base)
    rng = np.random.default_rng(1)
    for size in (1, 5, 33, 100, 128, 129, 224, 300):
        pick = torch.from_numpy(rng.choice(700, size=size, replace=False)).cuda()
        y = torch.empty((size, n_out), device="cuda")
        lin(xd[pick].contiguous(), y)
        assert torch.equal(y.view(torch.int32), base[pick].view(torch.int32)), size
    LinearFP8.check_device_error()


def test_segments_of_both_types():
    x, _, codes, scales = _inputs(2368, 1536, 1, 6, 7)
    rows = [512, 512, 128, 128, 64, 1024]
    lin = _linear(codes, scales)
    outs = [torch.empty((6, r), device="cuda") for r in rows[:-1]] + [torch.empty((6, 1024), dtype=torch.bfloat16, device="cuda")]
    lin(x.cuda(), outs)
    y = torch.empty((6, 2368), device="cuda")
    lin(x.cuda(), y)
    for s, (t, part) in enumerate(zip(outs, y.split(rows, dim=1))):
        assert torch.equal(t, part.to(t.dtype)), s
    _check(y, x, codes, scales, 1)


@pytest.mark.parametrize("n_tok,n_out", [(3, 200), (300, 200), (300, 17000)])
def test_values_that_are_not_finite_reach_their_token_alone(n_tok, n_out):
    x, _, codes, scales = _inputs(n_out, 400, 1, n_tok, 9)
    bad = x.clone()
    bad[1, 3], bad[2, 399] = float("inf"), float("nan")
    lin = _linear(codes, scales)
    y, z = torch.empty((n_tok, n_out), device="cuda"), torch.empty((n_tok, n_out), device="cuda")
    lin(x.cuda(), y)
    lin(bad.cuda(), z)
    assert bool(z[1:3].isnan().all())
    z[1:3] = y[1:3]
    assert torch.equal(y, z)
    # a NaN weight block reaches its 128 outputs alone
    nan = scales.copy()
    nan[1, 2] = 255
    _linear(codes, nan)(x.cuda(), z)
    assert bool(z[:, 128:256].isnan().all())
    assert torch.equal(z[:, :128], y[:, :128]) and torch.equal(z[:, 256:], y[:, 256:])


def test_scales_at_both_ends():
    """Codes of a weight scaled by 2^100 and 2^-100 against tokens scaled the
    other way: the same product as unscaled."""
    x, _, codes, scales = _inputs(140, 304, 1, 4, 13)
    for e in (-100, 100):
        y, z = torch.empty((4, 140), device="cuda"), torch.empty((4, 140), device="cuda")
        _linear(codes, scales)(x.cuda(), y)
        xs = (x.float() * 2.0 ** -e).to(torch.bfloat16)
        _linear(codes, (scales.astype(int) + e).clip(0, 254).astype(np.uint8))(xs.cuda(), z)
        assert torch.equal(y, z)


def test_tokens_that_start_off_a_16_byte_boundary():
    x, _, codes, scales = _inputs(140, 264, 1, 9, 17)
    lin = _linear(codes, scales)
    buf = torch.zeros(9 * 264 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(9, 264)
    odd.copy_(x)
    assert odd.data_ptr() % 16
    y, z = torch.empty((9, 140), device="cuda"), torch.empty((9, 140), device="cuda")
    lin(x.cuda(), y)
    lin(odd, z)
    assert torch.equal(y, z)


def test_two_streams_and_two_graphs_do_not_share_scratch():
    """The same weight called on two streams at once, and captured into two
    graphs that are replayed together: every result stays its own."""
    from compressed_sparse_long_hca_b200.api import LinearFP8
    x, w, _, _ = _inputs(2368, 7168, 1, 8, 21)
    lin = LinearFP8.quantize(w)
    xa, xb = x[:4].cuda(), x[4:].cuda()
    want = torch.empty((8, 2368), device="cuda")
    lin(x.cuda(), want)
    ya, yb = torch.zeros((4, 2368), device="cuda"), torch.zeros((4, 2368), device="cuda")
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        lin(xa, ya, stream=sa)                    # a stream that is not the current one
        with torch.cuda.stream(sb):
            lin(xb, yb)
    torch.cuda.synchronize()
    assert torch.equal(ya, want[:4]) and torch.equal(yb, want[4:])
    graphs = []
    for xs, ys in ((xa, ya), (xb, yb)):
        ys.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin(xs, ys)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, (sa, sb)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ya, want[:4]) and torch.equal(yb, want[4:])
    LinearFP8.check_device_error()


def test_an_own_workspace_and_an_empty_batch():
    x, _, codes, scales = _inputs(2368, 1536, 1, 100, 23)
    lin = _linear(codes, scales)
    y, z = torch.empty((100, 2368), device="cuda"), torch.full((100, 2368), 5.0, device="cuda")
    assert lin.workspace_bytes(16) == 0
    lin(x.cuda(), y)
    ws = torch.full((lin.workspace_bytes(100) + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    lin(x.cuda(), z, workspace=ws)
    assert torch.equal(y, z)
    with pytest.raises(RuntimeError, match="workspace smaller"):
        lin(x.cuda(), z, workspace=ws[:1024])
    empty = torch.empty((0, 2368), device="cuda")
    assert lin(x[:0].cuda(), empty) is empty


def test_refusals():
    from compressed_sparse_long_hca_b200.api import LinearFP8, quantize_fp8_weight
    x, _, codes, scales = _inputs(260, 256, 1, 4, 29)
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    lin = LinearFP8(c.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))
    y = torch.empty((4, 260), device="cuda")
    for bad_c, bad_s, groups in ((c.cpu(), s, 1), (c, s.cpu(), 1), (c.float(), s, 1), (c, s.float(), 1), (c.T, s, 1),
                                 (c, s[:2], 1), (c, s, 2), (c[:, :100].contiguous(), s[:, :1].contiguous(), 1), (c[0], s, 1)):
        with pytest.raises(ValueError):
            LinearFP8(bad_c, bad_s, groups=groups)
    for bad_x, bad_y in ((x.float().cuda(), y), (x, y), (x.cuda()[:, :128], y), (x.cuda().T.contiguous().T, y),
                         (x.cuda(), y[:3]), (x.cuda(), y.double()), (x.cuda(), y.cpu()), (x.cuda()[0], y)):
        with pytest.raises(ValueError):
            lin(bad_x, bad_y)
    for outs in ([y[:, :100].contiguous()], [y, y], [], [y[:, :0].contiguous(), y]):
        with pytest.raises(RuntimeError, match="CSA_ERR_ARG"):
            lin(x.cuda(), outs)
    with pytest.raises(ValueError):
        quantize_fp8_weight(torch.zeros(8, device="cuda"))
    with pytest.raises(RuntimeError):
        quantize_fp8_weight(torch.zeros((8, 12), device="cuda"))


# n_out, k_in, groups, n_tok
FORMS = [
    (257, 10320, 1, 130),         # a CTA per part: five token tiles of 32
    (750, 8496, 1, 639),          # a CTA per part: five of 128
    (2051, 8200, 1, 130),         # a CTA per part: more clusters than the SMs hold at once
    (107, 2022 * 8, 1, 1030),     # one row tile, eight parts, 64 tokens a tile
    (2368, 1536, 1, 100),         # whole tiles of at most 128 tokens, four of 32
    (2368, 7168, 1, 30),          # 32 tokens, a CTA per part
    (20000, 264, 1, 30),          # 32 tokens, whole tiles, several per CTA
    (2368, 7168, 1, 52),          # 64 tokens, a CTA per part
    (9600, 1160, 1, 60),          # 64 tokens, whole tiles of two parts
    (90, 264, 1, 1000),           # one launch: 63 tiles of 16 tokens
    (512, 4096, 1, 70),           # one launch: five tiles, a cluster of eight CTAs each
    (2048, 16 * 264, 16, 200),    # one launch: 13 tiles, grouped
    (8001, 264, 1, 1000),         # whole tiles, several per SM
    (8001, 1032, 1, 450),         # pairs, output rows of odd length
    (6400, 10 * 528, 10, 780),    # pairs, grouped: feature tiles that begin inside a row tile
    (9456, 1160, 1, 513),         # pairs: two K parts, a ragged last tile, one token beyond two tiles
    (8002, 1032, 1, 450),         # pairs, output rows on 4 and 8 bytes
]


@pytest.mark.parametrize("n_out,k_in,groups,n_tok", FORMS)
def test_every_form(n_out, k_in, groups, n_tok):
    """Against the oracle, in both types; the first tokens alone, which another
    form computes, have the same bits; rows behind the last stay as they were."""
    x, _, codes, scales = _inputs(n_out, k_in, groups, n_tok, n_tok)
    lin, xd = _linear(codes, scales, groups), x.cuda()
    y = torch.full((n_tok + 1, n_out), 7.0, device="cuda")
    lin(xd, y[:n_tok])
    pick = np.unique(np.r_[0:8, n_tok // 2, n_tok - 20:n_tok])         # the oracle's share of the tokens
    _check(y[pick], x[pick], codes, scales, groups)
    b = torch.full((n_tok + 1, n_out), 7.0, device="cuda", dtype=torch.bfloat16)
    lin(xd, b[:n_tok])
    assert torch.equal(b[:n_tok], y[:n_tok].to(torch.bfloat16))
    assert bool((y[n_tok] == 7).all()) and bool((b[n_tok] == 7).all())
    few = torch.empty((25, n_out), device="cuda")
    lin(xd[:25], few)
    assert torch.equal(few, y[:25])
    need = lin.workspace_bytes(n_tok)                                  # the call stays within its workspace
    ws = torch.full((need + 4096,), 90, dtype=torch.uint8, device="cuda")
    b.zero_()
    lin(xd, b[:n_tok], workspace=ws[:need])
    assert torch.equal(b[:n_tok], y[:n_tok].to(torch.bfloat16)) and bool((ws[need:] == 90).all())
    from compressed_sparse_long_hca_b200.api import LinearFP8
    LinearFP8.check_device_error()


@pytest.mark.parametrize("n_out,k_in,n_tok", [(2368, 1536, 6), (2368, 1536, 50), (2368, 1536, 100), (700, 300 * 8, 300), (20001, 264, 300),
                                              (9100, 1160, 513), (8001, 1032, 450), (8002, 1032, 450), (9456, 1160, 513), (750, 8496, 639)])
def test_segments_that_begin_anywhere(n_out, k_in, n_tok):
    """Segments of odd sizes, in every form of the launch: the outputs are
    those of one segment, and nothing beside them is written."""
    x, _, codes, scales = _inputs(n_out, k_in, 1, n_tok, 31)
    lin = _linear(codes, scales)
    y = torch.empty((n_tok, n_out), device="cuda")
    lin(x.cuda(), y)
    rows = [1, 33, 127, 130, 2, 36, 3]
    rows.append(n_out - sum(rows))
    bufs, outs = [], []
    for s, r in enumerate(rows):
        dt = torch.bfloat16 if s % 2 else torch.float32
        bufs.append(torch.full((n_tok * r + 18,), 5.0, dtype=dt, device="cuda"))
        outs.append(bufs[-1][9: 9 + n_tok * r].view(n_tok, r))       # off 16 bytes
    lin(x.cuda(), outs)
    for b, t, part in zip(bufs, outs, y.split(rows, dim=1)):
        assert torch.equal(t, part.to(t.dtype))
        assert bool((b[:9] == 5).all()) and bool((b[-9:] == 5).all())
    from compressed_sparse_long_hca_b200.api import LinearFP8
    LinearFP8.check_device_error()


FIRST_CALL_CAPTURED = """
import sys, torch
from compressed_sparse_long_hca_b200.api import HeadNorm, LinearFP8
n_tok, n_out, k = (int(v) for v in sys.argv[1:])
g = torch.Generator(device="cuda").manual_seed(1)
lin = LinearFP8.quantize(torch.randn((n_out, k), generator=g, device="cuda"))
x = torch.randn((n_tok, k), generator=g, device="cuda").to(torch.bfloat16)
y, z = torch.zeros((n_tok, n_out), device="cuda"), torch.zeros((n_tok, n_out), device="cuda")
hn = HeadNorm(k, 8)
pos = torch.arange(n_tok, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    lin(x, y)
    hn(pos, x[:, None], None)
graph.replay()
x.copy_(torch.randn((n_tok, k), generator=g, device="cuda"))
xe = x.clone()
graph.replay()
lin(xe, z)
hn(pos, xe[:, None], None)
torch.cuda.synchronize()
assert torch.equal(y, z) and torch.equal(x, xe)
LinearFP8.check_device_error()
print("captured")
"""


@pytest.mark.parametrize("shape", [(4, 2368, 1024), (50, 300, 256), (300, 20000, 256)])
def test_the_first_call_of_a_process_can_be_captured(shape):
    """The launches' set-up (function attributes, module loading) works inside
    a capture, too."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED, *map(str, shape)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_a_long_run_of_k_and_many_tokens():
    """K parts of many scale chunks that begin inside one, and token counts at
    the borders of the launch's forms: one token's bits in all of them."""
    from compressed_sparse_long_hca_b200.api import LinearFP8
    for n_out, k_in in ((520, 8 * 1500), (16512, 1160)):
        x, w, codes, scales = _inputs(n_out, k_in, 1, 1100, 41)
        lin = _linear(codes, scales)
        xd = x.cuda()
        base = torch.empty((1100, n_out), device="cuda")
        lin(xd, base)
        _check(base[:3], x[:3], codes, scales, 1)
        for n in (1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 511, 1025):
            y = torch.empty((n, n_out), device="cuda")
            lin(xd[1100 - n:], y)
            assert torch.equal(y, base[1100 - n:]), (n_out, n)
    LinearFP8.check_device_error()
