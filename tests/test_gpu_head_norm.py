"""GPU parity of the head norms with rotation (csa_head_norm) against the fp64
oracle: dims, types, strides and head counts of both vector widths, values
beyond fp32's squares, rows that are not finite, in-place calls, streams,
captured graphs and refusals; and the attention's rotated queries."""
import numpy as np
import pytest

from compressed_sparse_long_hca_b200 import inputs as I
from oracle import csa_oracle as O
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return cuda_lib


def _check(got, x, weight, eps, pos, R, what):
    """fp32 arithmetic: the sum of squares carries at most 37 roundings (a
    lane adds up to 32 squares, then up to 5 exchanges), half of which reach
    the scale; mean, eps, root, reciprocal, scale and weight add 6 more: below
    32 half steps, 2^-24 each.  A rotation adds the rounding of sine and
    cosine and of two products and moves a pair's errors into each other:
    32 + 8 half steps of |x0| + |x1|.  A BF16 result adds half a step, 2^-8."""
    x = x.double().cpu().numpy()
    w = None if weight is None else weight.double().cpu().numpy()
    flat = O.head_norm(x, w, eps)
    want = flat if pos is None else O.head_norm(x, w, eps, pos.cpu().numpy(), R)
    mag = np.abs(flat)
    if pos is not None and R:
        D = x.shape[-1]
        pair = mag[..., D - R:].reshape(*mag.shape[:-1], R // 2, 2).sum(-1, keepdims=True)
        mag[..., D - R:] = np.broadcast_to(pair, (*pair.shape[:-1], 2)).reshape(*mag.shape[:-1], R)
    bound = 40 * 2.0 ** -24 * mag + 2.0 ** -149
    if got.dtype == BF:
        bound = bound * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8 + 2.0 ** -134
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), f"{what}: {int((~(err <= bound)).sum())} outside, worst {np.nanmax(err / (mag + 1e-300)):.3e}"


def _weights(D, seed):
    g = torch.Generator().manual_seed(seed)
    return 1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)


def _pos(n, seed, far=1 << 20):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, far, n)
    p[0] = 0
    p[-1] = far - 1
    return torch.from_numpy(p).cuda()


# n, H, HK, D, R, q type, k type, rotate_k
SHAPES = [
    (1, 8, 1, 64, 16, F32, F32, False),      # the tiny layer
    (4, 128, 1, 512, 64, BF, F32, False),    # a decode step
    (130, 24, 3, 96, 32, BF, BF, True),      # 12 of 16 lanes a head
    (3, 5, 2, 2, 2, F32, BF, True),          # the smallest dims
    (9, 7, 1, 30, 6, BF, F32, True),         # scalar loads
    (2, 3, 9, 1024, 128, F32, BF, True),     # the largest dims
    (2, 33, 1, 520, 520, BF, BF, False),     # every dim rotated, a lane's last step ragged
    (700, 40, 2, 256, 0, BF, F32, True),     # no rotation; several heads a warp
    (2000, 65, 1, 128, 64, BF, F32, False),  # a token's heads in one block
]


@pytest.mark.parametrize("n,H,HK,D,R,qt,kt,rot", SHAPES)
def test_matches_the_oracle(n, H, HK, D, R, qt, kt, rot):
    from compressed_sparse_long_hca_b200.api import HeadNorm
    g = torch.Generator(device="cuda").manual_seed(D + n)
    q = (2 * torch.randn((n, H, D), generator=g, device="cuda")).to(qt)
    k = (2 * torch.randn((n, HK, D), generator=g, device="cuda")).to(kt)
    qw, kw = _weights(D, 1)
    hn = HeadNorm(D, R, q_weight=qw, k_weight=kw, rotate_k=rot)
    pos = _pos(n, D)
    # rows behind the last token stay as they were
    qo, ko = torch.full((n + 1, H, D), 7.0, dtype=qt, device="cuda"), torch.full((n + 1, HK, D), 7.0, dtype=kt, device="cuda")
    a, b = hn(pos if R else None, q, qo[:n], k, ko[:n])
    assert a.data_ptr() == qo.data_ptr() and b.data_ptr() == ko.data_ptr()
    assert bool((qo[n] == 7).all()) and bool((ko[n] == 7).all())
    _check(qo[:n], q, qw, 1e-6, pos, R, "q")
    _check(ko[:n], k, kw, 1e-6, pos if rot else None, R, "k")


@pytest.mark.parametrize("n,H,HK,D,R,qt,kt,rot", [
    (1501, 4, 7, 384, 86, BF, BF, True), (517, 28, 4, 288, 64, F32, F32, True), (700, 3, 1, 1024, 1024, BF, F32, True),
    (2049, 1, 2, 16, 16, F32, BF, False), (40, 200, 1, 520, 6, BF, BF, True), (5, 1000, 3, 256, 0, BF, F32, False),
    (1300, 5, 3, 128, 64, BF, F32, True), (1300, 0, 3, 100, 10, BF, F32, True), (1300, 2, 0, 70, 70, F32, BF, False),
    (2500, 72, 8, 64, 2, F32, BF, True), (3000, 1, 1, 1024, 2, BF, BF, False), (1200, 90, 2, 128, 64, BF, BF, False)])
def test_many_tokens_of_few_heads(n, H, HK, D, R, qt, kt, rot):
    """A block's run of heads crosses tokens, and goes from queries to keys."""
    test_matches_the_oracle(n, H, HK, D, R, qt, kt, rot)


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_offsets_and_in_place(D, dtype):
    from compressed_sparse_long_hca_b200.api import HeadNorm
    n, H, R = 11, 6, 16
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((n, H, D), generator=g, device="cuda").to(dtype)
    w = _weights(D, 2)[0]
    hn, pos = HeadNorm(D, R, q_weight=w, k_weight=w, rotate_k=True), _pos(n, 3)
    want = torch.empty_like(x)
    hn(pos, x, want)
    _check(want, x, w, 1e-6, pos, R, "contiguous")
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)       # [heads, n, D] in memory
    out = torch.empty((n, 2 * H, D), dtype=dtype, device="cuda")[:, ::2]
    hn(pos, heads_first, out)
    assert torch.equal(out, want)
    buf = torch.zeros(n * H * D + 1, dtype=dtype, device="cuda")        # one element off 16 bytes
    odd = buf[1:].view(n, H, D)
    odd.copy_(x)
    hn(pos, odd, out)
    assert torch.equal(out, want)
    hn(pos, odd)                                                       # in place, off 16 bytes
    assert torch.equal(odd, want) and float(buf[0]) == 0
    both = torch.cat([x, x], 1)                                        # one product's queries and keys, in place
    hn(pos, both[:, :H], None, both[:, H:], None)
    assert torch.equal(both[:, :H], want) and torch.equal(both[:, H:], want)
    hn(pos, x[:, :0], None, x, out)                                    # no query heads, no keys
    assert torch.equal(out, want)
    hn(pos[:0], x[:0], None)
    shared = x[:, :1].expand(n, H, D)                                  # one head for all, read only
    hn(pos, shared, out)
    assert torch.equal(out, want[:, :1].expand(n, H, D))


def test_values_beyond_the_squares_of_fp32():
    from compressed_sparse_long_hca_b200.api import HeadNorm
    D = 256
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((6, 3, D), generator=g, device="cuda")
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, 1] *= 1e25                                                    # one head of a warp
    x[4] *= 1e-18
    for eps in (0.0, 1e-30, 1e-6):
        hn = HeadNorm(D, 0, eps=eps)
        y = torch.empty_like(x)
        hn(None, x, y)
        _check(y, x, None, eps, None, 0, f"eps {eps}")
    z = torch.zeros((1, 2, D), device="cuda")
    HeadNorm(D, 0)(None, z)
    assert bool((z == 0).all())


@pytest.mark.parametrize("D", [64, 512])
def test_heads_that_are_not_finite_stay_alone(D):
    from compressed_sparse_long_hca_b200.api import HeadNorm
    x = torch.randn((3, 8, D), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    hn, pos = HeadNorm(D, 16), _pos(3, 1)
    want = torch.empty_like(x)
    hn(pos, x, want)
    bad = x.clone()
    bad[1, 2, 5] = float("nan")
    bad[2, 3, 7] = float("inf")
    y = torch.empty_like(x)
    hn(pos, bad, y)
    assert bool(y[1, 2].isnan().all())
    assert bool(y[2, 3, 7].isnan()) and bool((y[2, 3, :7] == 0).all())  # inf / inf, and finite / inf
    y[1, 2], y[2, 3] = want[1, 2], want[2, 3]
    assert torch.equal(y, want)


def test_streams_and_graphs():
    from compressed_sparse_long_hca_b200.api import HeadNorm
    D, n = 512, 4
    hn, pos = HeadNorm(D, 64, q_weight=_weights(D, 3)[0]), _pos(n, 9)
    x = torch.randn((n, 128, D), device="cuda").to(BF)
    c = torch.randn((n, 1, D), device="cuda")
    want, cw = torch.empty_like(x), torch.empty_like(c)
    hn(pos, x, want, c, cw)
    y, cy = torch.zeros_like(x), torch.zeros_like(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    hn(pos, x, y, c, cy, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(cy, cw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hn(pos, x, y, c, cy)
    x.mul_(-1)                                                         # the replay reads what is there then
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -want) and torch.equal(cy, cw)


def test_refusals():
    from compressed_sparse_long_hca_b200.api import HeadNorm, LayerProjections
    for kw in (dict(dim=63, rope=0), dict(dim=1026, rope=0), dict(dim=0, rope=0), dict(dim=64, rope=66), dict(dim=64, rope=3),
               dict(dim=64, rope=16, eps=-1.0), dict(dim=64, rope=16, eps=float("nan")), dict(dim=64, rope=16, rope_base=1.0),
               dict(dim=64, rope=16, q_weight=torch.ones(32))):
        with pytest.raises(ValueError):
            HeadNorm(**kw)
    hn = HeadNorm(64, 16)
    x, pos = torch.zeros((3, 2, 64), device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for args in ((None, x), (pos.int(), x), (pos[:2], x), (pos.cpu(), x), (pos, x.cpu()), (pos, x.double()), (pos, x[0]),
                 (pos, x[:, :, :32]), (pos, x, x[:2]), (pos, x, x.to(BF)), (pos, x.transpose(1, 2).contiguous().transpose(1, 2)),
                 (pos, x, None, x[:2], None), (pos, x, None, x.half(), None), (pos, x, None, x, x[:, :1])):
        with pytest.raises(ValueError):
            hn(*args)
    W = np.zeros((64, 32), np.float32)
    for kw in (dict(fmt="fp4"), dict(norm=HeadNorm(32, 16)), dict(norm=HeadNorm(64, 16, rotate_k=True))):
        with pytest.raises(ValueError):
            LayerProjections(csa=False, W_c=W, W_z=W, W_dq=W, W_uq=W, **kw)


@pytest.mark.parametrize("fmt,H,D,R", [("f32", 8, 64, 16), ("mixed", 8, 64, 16), ("mixed", 64, 512, 64)])
@pytest.mark.parametrize("layer", [0, 1])
def test_attention_takes_rotated_queries(fmt, H, D, R, layer):
    """The attention of queries rotated beforehand equals the attention that
    rotates them, in every variant, for decode queries and for a chunk.
    Requests 2 and 3 hold the same tokens as 0 and 1: each pair appends its
    own chunk."""
    from compressed_sparse_long_hca_b200.api import Cache
    rng = np.random.default_rng(11)
    T, n_tok, k, HI, dI = 1100, 5, 40, 4, 32
    cache = Cache(n_csa=1, n_hca=1, H=H, D=D, D_rope=R, H_I=HI, d_I=dI, max_requests=4, max_pages_per_request=3,
                  pool_pages=12, b_pos_csa=np.zeros((1, 8, D)), b_pos_idx=np.zeros((1, 8, dI)),
                  b_pos_hca=np.zeros((1, 128, D)), fmt=fmt)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    some = lambda *shape: dev(rng.standard_normal(shape))
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    for r in range(4):
        cache.request_alloc(r, 1500)
    csa = layer == 0
    twice = lambda t: None if t is None else torch.cat([t, t])
    c, z, ci, zi = some(2, T, D), some(2, T, D), some(2, T, dI) if csa else None, some(2, T, dI) if csa else None
    cache.compress_append(layer, ids, twice(c), twice(z), twice(ci), twice(zi))
    sink = some(H)
    idx = np.stack([np.sort(rng.choice(T // 4, k, replace=False)) for _ in range(2)]).astype(np.int32)
    idx = torch.from_numpy(idx).cuda() if csa else None
    q = I.bf16_grid(rng.standard_normal((2, H, D)).astype(np.float32))
    qd, rd = dev(q).to(cache.qdtype), dev(O.rope(q, T - 1, R)).to(cache.qdtype)
    outs = []
    for variant in ("auto", "high", "low"):
        a, b = torch.empty_like(qd), torch.empty_like(qd)
        cache.decode_attn(layer, ids[:2], qd, idx, sink, a, variant=variant)
        cache.decode_attn(layer, ids[2:], rd, idx, sink, b, variant=variant, q_rotated=True)
        cache.check_device_error()
        for i in range(2):
            Hp.check_attention(b[i].float().cpu().numpy(), a[i].double().cpu().numpy(), f"{variant} {i}", fmt=fmt)
        outs.append(b)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    qc = I.bf16_grid(rng.standard_normal((2, n_tok, H, D)).astype(np.float32))
    rc = O.rope(qc, np.broadcast_to(np.arange(T, T + n_tok)[None, :, None], (2, n_tok, H)), R)
    more = [some(2, n_tok, D), some(2, n_tok, D)] + ([some(2, n_tok, dI), some(2, n_tok, dI)] if csa else [None, None])
    qi, w = (some(2, n_tok, HI, dI), some(2, n_tok, HI)) if csa else (None, None)
    res = []
    for pair, src, flag in ((ids[:2], qc, False), (ids[2:], rc, True)):
        qq = dev(src).to(cache.qdtype)
        out = torch.empty_like(qq)
        cache.prefill_chunk(layer, pair, *more, qq, qi, w, k if csa else 0, sink, out, q_rotated=flag)
        cache.check_device_error()
        res.append(out)
    for i in range(2):
        for j in range(n_tok):
            Hp.check_attention(res[1][i, j].float().cpu().numpy(), res[0][i, j].double().cpu().numpy(), f"chunk {i} {j}",
                               fmt=fmt)
