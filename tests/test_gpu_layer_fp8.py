"""A decode step whose projections are the FP8 products and whose queries and
KV candidates pass the head norms, on the tiny configuration's shapes (hidden
256, 8 heads x 64, RoPE 16, indexer 4 x 32, top-16): hidden states -> FP8
products -> norms with rotation -> append -> index + top-k -> attention of the
rotated queries -> FP8 grouped output projection.  Each stage against the
oracle on the GPU's own inputs to that stage, then the step replayed as one
graph."""
import math

import numpy as np
import pytest

from compressed_sparse_long_hca_b200 import inputs as I
from oracle import csa_oracle as O
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return cuda_lib


def _w(seed, rows, cols, f):
    return I.bf16_grid(I.normal((rows, cols), seed, 98, f) / np.float32(math.sqrt(cols)))


def _fp8(x, W, groups=1):
    """The FP8 product of x and its sum of magnitudes, fp64; W quantised as a whole."""
    codes, scales = O.fp8_quantize_blocks(W, rows=128)
    xc, xs = O.fp8_quantize_blocks(x, groups=groups)
    xd, wd = O.fp8_dequantize_blocks(xc, xs, groups=groups), O.fp8_dequantize_blocks(codes, scales, rows=128)
    return O.grouped_linear(xd, wd, groups), O.grouped_linear(np.abs(xd), np.abs(wd), groups)


def _ok(got, ref, bound, what):
    err = np.abs(np.asarray(got, np.float64).reshape(ref.shape) - ref)
    assert np.all(err <= bound), f"{what}: {int((err > bound).sum())} outside, worst {float((err / (bound + 1e-300)).max()):.3f}"


SUM = 2.0 ** -17          # fp32 sums of at most 4 blocks of products: (4 * 8 + 32) 2^-23 of the magnitudes


@pytest.mark.parametrize("csa", [True, False])
def test_decode_step_stage_by_stage(csa):
    from compressed_sparse_long_hca_b200.api import HeadNorm, LayerProjections, LinearFP8, OutputProjection
    wl = I.C1
    d, D, R, H, H_I, d_I, d_c, k = wl.hidden, wl.D, wl.R, wl.H, wl.H_I, wl.d_I, 64, wl.k
    T, seed, layer = 700, wl.seed + 17, 0 if csa else 1
    pair = Hp.Pair(wl, 1, 1, max_req=1, capacity=T + 64)
    pair.cache.request_alloc(0, T + 64)
    h = I.bf16_grid(I.normal((T + 1, d), seed, 0, 0, 5))
    hd = torch.from_numpy(h).cuda().to(torch.bfloat16)
    names = ["W_c", "W_z"] + (["W_cI", "W_zI", "W_w"] if csa else []) + ["W_dq"]
    rows = [D, D] + ([d_I, d_I, H_I] if csa else []) + [d_c]
    Wd = {n: _w(seed, r, d, i) for i, (n, r) in enumerate(zip(names, rows))}
    Wd["W_uq"] = _w(seed, H * D, d_c, 21)
    if csa:
        Wd["W_uqI"] = _w(seed, H_I * d_I, d_c, 22)
    qw, cw = 1 + 0.1 * I.normal((D,), seed, 1, 1, 1), 1 + 0.1 * I.normal((D,), seed, 1, 1, 2)
    norm = HeadNorm(D, R, q_weight=qw, k_weight=cw)
    P = LayerProjections(csa=csa, fmt="fp8", norm=norm, **Wd)
    plain = LayerProjections(csa=csa, fmt="fp8", **Wd)
    groups, d_model = 2, 384
    W_g, W_o = _w(seed, groups * 128, (H // groups) * D, 31), _w(seed, d_model, groups * 128, 32)
    op = OutputProjection(W_g, W_o, groups, fmt="fp8")
    rid = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.arange(T + 1, dtype=torch.int64, device="cuda")
    # ---- projections, norms and append: ragged chunks of the prefix, then the decode token
    got, raw = [], []
    bounds = [0, 1, 250, T, T + 1]
    for t0, t1 in zip(bounds[:-1], bounds[1:]):
        n = t1 - t0
        o, r = P.new_outputs(n, H), plain.new_outputs(n, H)
        x = hd[t0:t1].contiguous()
        P(x, o, positions=pos[t0:t1])
        plain(x, r)
        v = lambda t: t.view(1, n, -1)
        pair.cache.compress_append(layer, rid, v(o["c"]), v(o["z"]), v(o["ci"]) if csa else None,
                                   v(o["zi"]) if csa else None)
        got.append({key: t.float().cpu().numpy().reshape(n, -1) for key, t in o.items()})
        raw.append({key: t.float().cpu().numpy().reshape(n, -1) for key, t in r.items()})
    torch.cuda.synchronize()
    LinearFP8.check_device_error()
    pair.cache.check_device_error()
    cat, raw = ({key: np.concatenate([g[key] for g in gs]) for key in gs[0]} for gs in (got, raw))
    ref, mag = _fp8(h, np.concatenate([Wd[n] for n in names]))
    keys = ["c", "z"] + (["ci", "zi", "w"] if csa else []) + ["c_q"]
    at = np.cumsum([0] + rows)
    for key, r0, r1 in zip(keys, at[:-1], at[1:]):
        bound = SUM * mag[:, r0:r1] + (np.abs(ref[:, r0:r1]) * 2.0 ** -8 if key == "c_q" else 0)
        _ok(raw[key], ref[:, r0:r1], bound, key)
        if key != "c":
            assert np.array_equal(raw[key], cat[key]), key
    ref, mag = _fp8(raw["c_q"], np.concatenate([Wd["W_uq"]] + ([Wd["W_uqI"]] if csa else [])))
    _ok(raw["q"], ref[:, :H * D], SUM * mag[:, :H * D] * (1 + 2.0 ** -8) + np.abs(ref[:, :H * D]) * 2.0 ** -8, "q")
    if csa:
        _ok(raw["q_idx"], ref[:, H * D:], SUM * mag[:, H * D:], "q_I")
    # the norms of the products as they were stored: fp32 arithmetic (40 half steps of the pair), BF16 queries
    flat = O.head_norm(raw["q"].reshape(-1, H, D), qw, 1e-6)
    want = O.rope(flat, np.arange(T + 1)[:, None].repeat(H, 1), R)
    m = np.abs(flat)
    m[..., D - R:] = np.repeat(m[..., D - R:].reshape(T + 1, H, R // 2, 2).sum(-1), 2, axis=-1)
    _ok(cat["q"], want, 40 * 2.0 ** -24 * m * 1.01 + np.abs(want) * 2.0 ** -8, "normed q")
    want = O.head_norm(raw["c"][:, None], cw, 1e-6)
    _ok(cat["c"], want, 40 * 2.0 ** -24 * np.abs(want), "normed c")
    # ---- the decode token: selection and attention over the stored rows
    p = pair.oracle_params(layer)
    q = torch.from_numpy(cat["q"][T].reshape(1, H, D)).cuda().to(torch.bfloat16)
    sink = pair.params[layer]["sink"]
    out = torch.empty((1, H, D), dtype=torch.bfloat16, device="cuda")
    N = (T + 1) // (4 if csa else 128)
    idx = None
    sel = np.arange(N)
    if csa:
        kv_ref, key_ref = O.csa_entries_all(cat["c"], cat["z"], cat["ci"], cat["zi"], p.b_kv, p.b_idx, R)
        Hp.check_kv_rounding(pair.cache.read_rows(0, 0, 0, 0, N), kv_ref, D, R, "entries")
        idx = torch.empty((1, k), dtype=torch.int32, device="cuda")
        scores, nv = torch.empty((1, N + 9), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        qi, w = (torch.from_numpy(cat[key][T]).cuda().view(*s) for key, s in (("q_idx", (1, H_I, d_I)), ("w", (1, H_I))))
        pair.cache.index_topk(0, rid, qi.contiguous(), w.contiguous(), scores, nv, k, idx)
        sel = idx[0].cpu().numpy()
        assert int(nv[0]) == N and len(set(sel.tolist())) == k
    else:
        Hp.check_kv_rounding(pair.cache.read_rows(1, 0, 0, 0, N), O.hca_entries_all(cat["c"], cat["z"], p.b_kv, R), D, R, "entries")
    sd = torch.from_numpy(sink).cuda()
    pair.cache.decode_attn(layer, rid, q, idx, sd, out, q_rotated=True)
    pair.cache.check_device_error()
    back = O.rope(cat["q"][T].reshape(H, D), -float(T), R)            # the reference rotates it forth
    ref = Hp.attention_over_stored_rows(pair.cache, layer, 0, T, sel, back, sink, D, R)
    Hp.check_attention(out[0].float().cpu().numpy(), ref, "attention")
    # ---- the grouped output projection
    mid, y = torch.empty((1, groups * 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, d_model), device="cuda")
    op(out, mid, y)
    LinearFP8.check_device_error()
    ref, mag = _fp8(out.float().cpu().numpy().reshape(1, -1), W_g, groups)
    _ok(mid.float().cpu().numpy(), ref, SUM * mag * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8, "grouped projection")
    ref, mag = _fp8(mid.float().cpu().numpy(), W_o)
    _ok(y.cpu().numpy(), ref, SUM * mag, "output projection")
    # ---- projections, norms, attention and output projection of the token as one graph
    o, out2, mid2, y2 = P.new_outputs(1, H), torch.zeros_like(out), torch.zeros_like(mid), torch.zeros_like(y)
    x = hd[T:T + 1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P(x, o, positions=pos[T:])
        pair.cache.decode_attn(layer, rid, o["q"], idx, sd, out2, q_rotated=True)
        op(out2, mid2, y2)
    x.zero_()
    g.replay()
    x.copy_(hd[T:T + 1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o["q"], q) and torch.equal(out2, out) and torch.equal(y2, y)
    LinearFP8.check_device_error()
