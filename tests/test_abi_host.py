"""Host-side checks of the C ABI that need no GPU: the library builds and
loads, exports every function include/csa.h declares, and validates
configurations on the host."""
import ctypes
import os
import re

import pytest

from compressed_sparse_long_hca_b200 import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "csa.h")


def declared_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(csa_\w+)\s*\(", src, flags=re.M)))


def test_header_declares_the_path():
    names = declared_functions()
    for f in ("csa_compress_append", "csa_index_scores", "csa_topk", "csa_hca_decode_attn",
              "csa_cache_required_bytes", "csa_cache_init"):
        assert f in names


def test_library_exports_every_declared_symbol(cuda_lib):
    for name in declared_functions():
        assert hasattr(cuda_lib, name), name
        assert name in _lib.SIGNATURES, f"{name} has no Python binding"


def _cfg(**kw):
    base = dict(n_csa_layers=1, n_hca_layers=1, H=128, D=512, D_rope=64, H_I=64, d_I=128, window=128,
                max_requests=4, max_pages_per_request=2048, pool_pages=4 * 2048, rope_base=10000.0)
    base.update(kw)
    return _lib.CsaCfg(**base)


def test_required_bytes_and_validation(cuda_lib):
    c = _cfg()
    nbytes = cuda_lib.csa_cache_required_bytes(ctypes.byref(c))
    # 32768 blocks of (32 CSA rows + 32 index keys + 1 HCA row) at least
    assert nbytes >= 32768 * (32 * 580 + 32 * 68 + 580)
    assert nbytes < 32768 * 24000 + 64 * 2**20
    for bad in (dict(D=500), dict(D_rope=15), dict(window=64), dict(d_I=48), dict(H=0),
                dict(H_I=65), dict(n_csa_layers=0, n_hca_layers=0), dict(pool_pages=0)):
        assert cuda_lib.csa_cache_required_bytes(ctypes.byref(_cfg(**bad))) == 0, bad


def test_init_rejects_bad_arguments_without_launching(cuda_lib):
    c = _cfg()
    h = ctypes.c_void_p()
    # unaligned pointer and too-small arena are refused before any CUDA call
    assert cuda_lib.csa_cache_init(ctypes.byref(c), 0x1001, 1 << 40, None, None, None, ctypes.byref(h)) == -1
    assert cuda_lib.csa_cache_init(ctypes.byref(c), 0x10000, 16, None, None, None, ctypes.byref(h)) == -2
    assert h.value is None
    assert b"256-byte" in cuda_lib.csa_last_error() or True
    # compute calls on a NULL handle fail on the host
    assert cuda_lib.csa_compress_append(None, 0, 1, None, 1, None, None, None, None, None) == -1
    assert cuda_lib.csa_topk(None, 1, None, 1, 1, None, 0, None) == -1


def test_decode_step_packed_input_layout():
    """DecodeStep's packed host buffer: the fields in order (the attention
    query last, copied on its own), each on a 256-byte boundary, sized by
    shape and dtype, none overlapping."""
    import math

    import torch

    from compressed_sparse_long_hca_b200.api import decode_step_fields
    for csa, names in ((True, ["c", "z", "ci", "zi", "q_idx", "w", "q"]), (False, ["c", "z", "q"])):
        fields, total = decode_step_fields(4, 128, 512, 64, 128, csa)
        assert [f[0] for f in fields] == names
        end = 0
        for name, dtype, shape, off, nbytes in fields:
            assert off % 256 == 0 and off >= end, name
            assert nbytes == math.prod(shape) * torch.empty((), dtype=dtype).element_size(), name
            end = off + nbytes
        assert total >= end and total % 256 == 0
    fields, _ = decode_step_fields(4, 128, 512, 64, 128, True)
    f = {x[0]: x for x in fields}
    assert f["q"][4] == 4 * 128 * 512 * 2 and f["q"][1] == torch.bfloat16
    assert f["q_idx"][2] == (4, 64, 128) and f["w"][2] == (4, 64)
    assert f["c"][2] == (4, 1, 512) and f["ci"][2] == (4, 1, 128)


def test_topk_argument_errors_are_returned_before_any_launch(cuda_lib):
    """csa_topk needs no cache: every argument error comes back as
    CSA_ERR_ARG from the host checks (the pointer below is never touched)."""
    P = 0x10000
    cases = [
        ((P, 10, P, -1, 4, P, 0, None), b"n must be"),
        ((P, 10, P, 70000, 4, P, 0, None), b"n must be"),
        ((None, 10, P, 1, 4, P, 0, None), b"NULL"),
        ((P, 10, None, 1, 4, P, 0, None), b"NULL"),
        ((P, 10, P, 1, 4, None, 0, None), b"NULL"),
        ((P, 10, P, 1, 0, P, 0, None), b"k and ld"),
        ((P, 0, P, 1, 4, P, 0, None), b"k and ld"),
        ((P, 10, P, 1, 4, P, 3, None), b"variant"),
    ]
    for args, msg in cases:
        assert cuda_lib.csa_topk(*args) == -1, args
        assert msg in cuda_lib.csa_last_error(), (args, cuda_lib.csa_last_error())
    assert cuda_lib.csa_topk(P, 10, P, 0, 4, P, 0, None) == 0        # an empty batch is a no-op


def test_cache_calls_on_a_null_handle_fail_on_the_host(cuda_lib):
    P = 0x10000
    assert cuda_lib.csa_index_scores(None, 0, 1, P, P, P, P, 8, P, 0, None) == -1
    assert cuda_lib.csa_hca_decode_attn(None, 0, 1, P, P, P, 4, P, 1.0, P, P, 1 << 20, 0, None) == -1
    assert cuda_lib.csa_hca_decode_attn_noalloc(None, 0, 1, P, P, P, 4, P, 1.0, P, None) == -1
    assert cuda_lib.csa_attn_workspace_bytes(None, 0, 1, 4) == 0
    assert cuda_lib.csa_request_alloc(None, 0, 16) == -1
    assert cuda_lib.csa_request_free(None, 0) == -1
    assert cuda_lib.csa_check_device_error(None, None) == -1
    assert cuda_lib.csa_debug_wait_timeout(None, 1000, None) == -1
    assert cuda_lib.csa_decode_step_input_bytes(None, 0, 1) == 0
    assert cuda_lib.csa_decode_step_dev_bytes(None, 0, 1, 16) == 0
    assert cuda_lib.csa_decode_step(None, 0, 1, P, 16, P, 1.0, P, P, P, 1 << 20, None) == -1
    assert cuda_lib.csa_prefill_workspace_bytes(None, 0, 1, 16, 16, 0) == 0
    assert cuda_lib.csa_prefill_chunk(None, 0, 1, P, 16, P, P, P, P, P, P, P, 16, P, 1.0, P, None, P, 1 << 20, 0,
                                      None) == -1


def test_gemm_shapes_and_argument_errors_on_the_host(cuda_lib):
    """The projection GEMM's size function and its argument checks run on the
    host: packed weight bytes are 128-row x 64-column tiles of 16 KB, a bad
    shape gives 0 bytes, and csa_gemm_bf16 returns CSA_ERR_ARG for every bad
    argument before any CUDA call (the pointers below are never touched)."""
    wb = cuda_lib.csa_gemm_weight_bytes
    tile = 128 * 64 * 2
    assert wb(300, 1000, 1) == 3 * 16 * tile                    # ceil(300 / 128) row tiles x ceil(1000 / 64)
    assert wb(16 * 128, 16 * 64, 16) == 16 * 1 * tile           # block diagonal: each row tile reads its group
    for bad in ((0, 64, 1), (256, 0, 1), (256, 64, 0), (256, 63, 1), (300, 64, 2), (256, 96, 3),
                (128 * 70000, 64 * 70000, 70000)):
        assert wb(*bad) == 0, bad
    P = 0x10000
    seg = (_lib.GemmOut * 2)()
    seg[0].rows, seg[0].bf16, seg[0].y = 100, 1, P
    seg[1].rows, seg[1].bf16, seg[1].y = 156, 0, P
    segs = ctypes.cast(seg, ctypes.c_void_p)
    g = cuda_lib.csa_gemm_bf16
    cases = [
        ((P, 256, 63, 1, P, 4, 2, segs, P, 1 << 30, None), b"multiple of 8"),
        ((P, 256, 64, 1, P, 257, 2, segs, P, 1 << 30, None), b"n_tok"),
        ((P, 256, 64, 1, P, 4, 0, segs, P, 1 << 30, None), b"n_seg"),
        ((P, 256, 64, 1, P, 4, 9, segs, P, 1 << 30, None), b"n_seg"),
        ((P, 300, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"add up"),
        ((None, 256, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"NULL"),
        ((P, 256, 64, 1, P, 4, 2, segs, P + 16, 1 << 30, None), b"aligned"),
    ]
    for args, msg in cases:
        assert g(*args) == -1, args
        assert msg in cuda_lib.csa_last_error(), (args, cuda_lib.csa_last_error())
    assert g(P, 256, 64, 1, P, 0, 2, segs, P, 1 << 30, None) == 0     # no tokens: nothing to do
    seg[1].y = None
    assert g(P, 256, 64, 1, P, 4, 2, segs, P, 1 << 30, None) == -1    # a segment without an output


def test_fp8_gemm_shapes_and_argument_errors_on_the_host(cuda_lib):
    """The FP8 product's size function and argument checks run on the host:
    packed bytes are 16 KB tiles of 128 x 128 codes, 512 bytes of scales per
    row tile and four blocks, and 1024 per feature tile (at most 224) and four; every bad argument comes back before any
    launch (the pointers below are never touched)."""
    wb = cuda_lib.csa_gemm_fp8_weight_bytes
    assert wb(300, 1000, 1) == 3 * (8 * 16384 + 2 * 512) + 2 * 2 * 1024
    assert wb(16 * 128, 16 * 64, 16) == 16 * (16384 + 512) + 16 * 1024
    for bad in ((0, 64, 1), (256, 0, 1), (256, 64, 0), (256, 63, 1), (300, 64, 2), (256, 96, 3), (65536 * 128, 64, 1)):
        assert wb(*bad) == 0, bad
    P = 0x10000
    seg = (_lib.GemmOut * 2)()
    seg[0].rows, seg[0].bf16, seg[0].y = 100, 1, P
    seg[1].rows, seg[1].bf16, seg[1].y = 156, 0, P
    segs = ctypes.cast(seg, ctypes.c_void_p)
    g = cuda_lib.csa_gemm_fp8
    cases = [
        ((P, 256, 63, 1, P, 4, 2, segs, P, 1 << 30, None), b"multiple of 8"),
        ((P, 256, 64, 1, P, -1, 2, segs, P, 1 << 30, None), b"n_tok"),
        ((P, 256, 64, 1, P, (1 << 20) + 1, 2, segs, P, 1 << 30, None), b"n_tok"),
        ((P, 256, 64, 1, P, 4, 0, segs, P, 1 << 30, None), b"n_seg"),
        ((P, 256, 64, 1, P, 4, 9, segs, P, 1 << 30, None), b"n_seg"),
        ((P, 300, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"add up"),
        ((P, 100, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"add up"),
        ((None, 256, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"NULL"),
        ((P, 256, 64, 1, None, 4, 2, segs, P, 1 << 30, None), b"NULL"),
        ((P, 256, 64, 1, P + 1, 4, 2, segs, P, 1 << 30, None), b"aligned"),
        ((P, 256, 64, 1, P, 4, 2, segs, P + 16, 1 << 30, None), b"aligned"),
        ((P + 8, 256, 64, 1, P, 4, 2, segs, P, 1 << 30, None), b"aligned"),
    ]
    for args, msg in cases:
        assert g(*args) == -1, args
        assert msg in cuda_lib.csa_last_error(), (args, cuda_lib.csa_last_error())
    assert g(P, 256, 64, 1, P, 0, 2, segs, P, 1 << 30, None) == 0     # no tokens: nothing to do
    seg[1].y = P + 2
    assert g(P, 256, 64, 1, P, 4, 2, segs, P, 1 << 30, None) == -1    # an fp32 segment off its elements
    assert cuda_lib.csa_gemm_fp8_quant_weight(None, 256, 64, 1, P, P, None) == -1
    assert cuda_lib.csa_gemm_fp8_quant_weight(P, 256, 60, 1, P, P, None) == -1
    assert cuda_lib.csa_gemm_fp8_pack_weight(P, P, 256, 64, 1, P + 4, 1 << 30, None) == -1
    assert cuda_lib.csa_gemm_fp8_pack_weight(P, P, 256, 64, 1, P, 100, None) == -2
    assert cuda_lib.csa_gemm_fp8_workspace_bytes(256, 64, 1, 0) == 0
    assert cuda_lib.csa_gemm_fp8_workspace_bytes(256, 64, 1, (1 << 20) + 1) == 0


def test_head_norm_argument_errors_on_the_host(cuda_lib):
    """csa_head_norm refuses bad arguments before any launch (the pointers
    below are never touched)."""
    P = 0x10000
    f = cuda_lib.csa_head_norm

    def part(**kw):
        d = dict(x=P, y=P, weight=P, x_token_stride=512, x_head_stride=64, y_token_stride=512, y_head_stride=64, heads=8,
                 f32=1, rotate=1)
        d.update(kw)
        return ctypes.cast(ctypes.pointer(_lib.HeadNormPart(*[d[n] for n, _ in _lib.HeadNormPart._fields_])), ctypes.c_void_p)

    q = part()
    nan = float("nan")
    cases = [
        ((4, 63, 16, 1e-6, P, P, q, None, None), b"dim"), ((4, 1026, 16, 1e-6, P, P, q, None, None), b"dim"),
        ((4, 64, 66, 1e-6, P, P, q, None, None), b"rope"), ((4, 64, 3, 1e-6, P, P, q, None, None), b"rope"),
        ((4, 64, 16, -1.0, P, P, q, None, None), b"eps"), ((4, 64, 16, nan, P, P, q, None, None), b"eps"),
        ((-1, 64, 16, 1e-6, P, P, q, None, None), b"n_tok"), ((1 << 31, 64, 16, 1e-6, P, P, q, None, None), b"n_tok"),
        ((4, 64, 16, 1e-6, P, P, None, None, None), b"NULL"), ((4, 64, 16, 1e-6, None, P, q, None, None), b"positions"),
        ((4, 64, 16, 1e-6, P, None, q, None, None), b"positions"),
        ((4, 64, 16, 1e-6, P, P, part(x=None), None, None), b"NULL"), ((4, 64, 16, 1e-6, P, P, q, part(y=None), None), b"NULL"),
        ((4, 64, 16, 1e-6, P, P, part(x=P + 2), None, None), b"aligned"),
        ((4, 64, 16, 1e-6, P, P, part(weight=P + 2), None, None), b"aligned"),
        ((4, 64, 16, 1e-6, P, P, part(f32=0, y=P + 1), None, None), b"aligned"),
        ((4, 64, 16, 1e-6, P, P, part(heads=-1), None, None), b"heads"),
        ((4, 64, 16, 1e-6, P, P, q, part(heads=65537), None), b"heads"),
    ]
    for args, msg in cases:
        assert f(*args) == -1, args
        assert msg in cuda_lib.csa_last_error(), (args, cuda_lib.csa_last_error())
    assert f(0, 64, 16, 1e-6, None, None, q, None, None) == 0              # no tokens: nothing to do
    assert f(4, 64, 16, 1e-6, None, None, part(heads=0), None, None) == 0  # no heads


def test_an_fp8_workspace_serves_every_smaller_call(cuda_lib):
    for n_out, k_in, groups in ((33, 64, 1), (750, 8496, 1), (8001, 1032, 1), (2048, 4096, 16)):
        sizes = [cuda_lib.csa_gemm_fp8_workspace_bytes(n_out, k_in, groups, n) for n in range(1, 1400)]
        assert sizes[:16] == [0] * 16
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
        assert all(s >= n * k_in for n, s in enumerate(sizes, 1) if s)


def _head_part(**kw):
    P = 0x10000
    d = dict(x=P, y=P, weight=P, x_token_stride=512, x_head_stride=64, y_token_stride=512, y_head_stride=64, heads=8,
             f32=1, rotate=1)
    d.update(kw)
    return ctypes.cast(ctypes.pointer(_lib.HeadNormPart(*[d[n] for n, _ in _lib.HeadNormPart._fields_])), ctypes.c_void_p)


def test_head_norm_refuses_positions_and_angles_off_their_elements(cuda_lib):
    P = 0x10000
    for pos, theta in ((P + 4, P), (P, P + 4), (P + 1, P)):
        assert cuda_lib.csa_head_norm(4, 64, 16, 1e-6, pos, theta, _head_part(), None, None) == -1, (pos, theta)
        assert b"8-byte aligned" in cuda_lib.csa_last_error()


def test_head_norm_refuses_an_output_whose_heads_overlap(cuda_lib):
    """Against every pair of heads, for strides of either sign and order."""
    import itertools
    P, dim = 0x10000, 4
    for n, heads in ((1, 1), (1, 3), (3, 1), (2, 3), (3, 2), (4, 5)):
        for ts, hs in itertools.product((-14, -8, -3, 0, 1, 4, 6, 8, 9, 12, 20), (-12, -4, 0, 2, 4, 5, 8, 10, 16)):
            at = [t * ts + h * hs for t in range(n) for h in range(heads)]
            overlap = any(abs(a - b) < dim for a, b in itertools.combinations(at, 2))
            part = _head_part(heads=heads, y_token_stride=ts, y_head_stride=hs, rotate=0)
            # (the keys are refused in any case, so that nothing is launched)
            assert cuda_lib.csa_head_norm(n, dim, 0, 1e-6, None, None, part, _head_part(heads=-1), None) == -1
            assert (b"overlap" in cuda_lib.csa_last_error()) == overlap, (n, heads, ts, hs)
    wide = _head_part(heads=65536, y_token_stride=1 << 62, y_head_stride=-(1 << 62), rotate=0)
    assert cuda_lib.csa_head_norm((1 << 31) - 1, 1024, 0, 1e-6, None, None, wide, _head_part(heads=-1), None) == -1
    assert b"overlap" in cuda_lib.csa_last_error()


def test_fp8_gemm_refuses_rows_whose_blocks_cannot_be_counted(cuda_lib):
    P, most = 0x10000, (1 << 31) - 128
    wb = cuda_lib.csa_gemm_fp8_weight_bytes
    assert wb(1, most, 1) == (most // 128) * 16384 + -(-most // 512) * (512 + 1024)
    for k in (most + 8, most + 120):
        assert wb(1, k, 1) == 0
        assert cuda_lib.csa_gemm_fp8_workspace_bytes(1, k, 1, 100) == 0
        assert cuda_lib.csa_gemm_fp8_quant_weight(P, 1, k, 1, P, P, None) == -1
        assert cuda_lib.csa_gemm_fp8_pack_weight(P, P, 1, k, 1, P, 1 << 60, None) == -1


def test_fp8_shapes_by_the_form_of_the_launch(cuda_lib):
    """The forms that the GPU tests are there for, on a B200's 148 SMs: a
    change of the choice makes this fail instead of leaving a form untested."""
    from tests import fp8_forms as F
    form = cuda_lib.csa_debug_fp8_form
    assert {s[0] for s in F.SHAPES} == F.FORMS
    for want, n_out, k_in, groups, n_tok in F.SHAPES:
        assert n_tok >= 3 and n_out > 128 and k_in // groups > 256
        assert form(n_out, k_in, groups, n_tok, 148) == want, (n_out, k_in, groups, n_tok)
    assert form(300, 63, 1, 4, 148) == 0 and form(300, 64, 1, 0, 148) == 0
    # no other form over the range, and the small calls need no workspace
    import random
    rng = random.Random(1)
    for _ in range(4000):
        n_out, k = int(2 ** rng.uniform(0, 17)), 8 * int(2 ** rng.uniform(0, 11))
        n_tok = int(2 ** rng.uniform(0, 13))
        assert form(n_out, k, 1, n_tok, 148) in F.FORMS


def test_fp8_gemm_refuses_an_output_on_its_tokens(cuda_lib):
    X, Y, n, k = 0x10000000, 0x90000000, 100, 4096
    end = X + n * k * 2
    seg = (_lib.GemmOut * 2)()
    segs = ctypes.cast(seg, ctypes.c_void_p)
    seg[0].rows, seg[0].bf16, seg[1].rows, seg[1].bf16 = 1000, 0, 1368, 1
    for y0, y1, overlap in ((X, Y, True), (Y, X, True), (end - 4, Y, True), (X - n * 1000 * 4 + 4, Y, True), (Y, end - 2, True),
                            (Y, X - n * 1368 * 2 + 2, True), (end, X - n * 1368 * 2, False), (X - n * 1000 * 4, end, False)):
        seg[0].y, seg[1].y = y0, y1
        # (without the workspace that it needs nothing is launched in any case)
        assert cuda_lib.csa_gemm_fp8(0x10000, 2368, k, 1, X, n, 2, segs, None, 0, None) != 0
        assert (b"overlaps" in cuda_lib.csa_last_error()) == overlap, (hex(y0), hex(y1))
