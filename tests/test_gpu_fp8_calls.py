"""How the FP8 product is called: on other streams than the current one, and
in the special cases that every form of its launch has to keep."""
import numpy as np
import pytest

from oracle import csa_oracle as O
from tests import fp8_forms as F
from tests import test_gpu_fp8 as T

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return cuda_lib


def test_a_weight_quantised_on_another_stream():
    """While the current stream is busy with what the weight comes from: the
    codes and scales are the oracle's, from a device tensor and a host array,
    and the packed weight gives the product of the same codes."""
    from compressed_sparse_long_hca_b200.api import LinearFP8, quantize_fp8_weight
    rng = np.random.default_rng(3)
    a = rng.standard_normal((700, 1160)).astype(np.float32)
    bf = torch.from_numpy(2 * a).to(torch.bfloat16).double().numpy()          # (doubling is exact)
    want_c, want_s = O.fp8_quantize_blocks(bf, rows=128)
    side = torch.cuda.Stream()
    x = torch.from_numpy(rng.standard_normal((5, 1160)).astype(np.float32)).cuda().to(torch.bfloat16)
    want = torch.empty((5, 700), device="cuda")
    LinearFP8(torch.from_numpy(want_c).cuda(), torch.from_numpy(want_s).cuda())(x, want)
    busy = torch.randn((4096, 4096), device="cuda")
    src = torch.from_numpy(a).cuda()
    torch.cuda.synchronize()
    for host in (False, True):
        for made in ("codes", "linear"):
            for _ in range(10):                                               # some milliseconds of work ahead
                busy = (busy @ busy).clamp(-1, 1)
            w = 2 * a if host else 2 * src
            if made == "codes":
                codes, scales = quantize_fp8_weight(w, stream=side)
                side.synchronize()
                assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want_c)
                assert np.array_equal(scales.cpu().numpy(), want_s)
            else:
                lin = LinearFP8.quantize(w, stream=side)
                del w
                y = torch.empty((5, 700), device="cuda")
                lin(x, y)
                assert torch.equal(y, want)
    LinearFP8.check_device_error()


def test_a_short_workspace_off_its_alignment_is_refused():
    from compressed_sparse_long_hca_b200.api import Linear, LinearFP8
    w = np.zeros((2368, 1536), np.float32)
    x, y = torch.zeros((100, 1536), dtype=torch.bfloat16, device="cuda"), torch.full((100, 2368), 5.0, device="cuda")
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    for lin in (LinearFP8.quantize(w), Linear(w)):
        with pytest.raises(RuntimeError, match="workspace"):
            lin(x, y, workspace=ws[1:101])
    torch.cuda.synchronize()
    assert bool((y == 5).all())
    lin = LinearFP8.quantize(w)
    lin.check_device_error()
    lin.check_device_error(torch.cuda.Stream())


def _form_is(shape):
    from compressed_sparse_long_hca_b200 import _lib
    form, n_out, k_in, groups, n_tok = shape
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the shapes are those of 148 SMs")
    assert _lib.load().csa_debug_fp8_form(n_out, k_in, groups, n_tok, 0) == form


@pytest.mark.parametrize("shape", F.SHAPES, ids=F.name)
def test_values_that_are_not_finite_in_every_form(shape):
    """An infinity and a NaN reach their tokens alone, a NaN weight block its
    outputs alone; everything else keeps its bits."""
    _form_is(shape)
    _, n_out, k_in, groups, n_tok = shape
    x, _, codes, scales = T._inputs(n_out, k_in, groups, n_tok, 9)
    bad = x.clone()
    bad[1, ::k_in // groups], bad[n_tok - 1, k_in // groups - 1::k_in // groups] = float("inf"), float("nan")
    lin = T._linear(codes, scales, groups)
    y, z = torch.empty((n_tok, n_out), device="cuda"), torch.empty((n_tok, n_out), device="cuda")
    lin(x.cuda(), y)
    lin(bad.cuda(), z)
    assert not bool(y.isnan().any())
    assert bool(z[1].isnan().all()) and bool(z[n_tok - 1].isnan().all())
    z[1], z[n_tok - 1] = y[1], y[n_tok - 1]
    assert torch.equal(y, z)
    nan = scales.copy()
    nan[1, 2] = 255
    T._linear(codes, nan, groups)(x.cuda(), z)
    assert bool(z[:, 128:256].isnan().all())
    assert torch.equal(z[:, :128], y[:, :128]) and torch.equal(z[:, 256:], y[:, 256:])
    lin.check_device_error()


@pytest.mark.parametrize("shape", [s for s in F.SHAPES if s[3] == 1 and s[1] > 400], ids=F.name)
def test_segments_that_begin_anywhere_in_every_form(shape):
    _form_is(shape)
    _, n_out, k_in, _, n_tok = shape
    T.test_segments_that_begin_anywhere(n_out, k_in, n_tok)


@pytest.mark.parametrize("shape", [s for s in F.SHAPES if s[3] == 1 and s[1] <= 400], ids=F.name)
def test_segments_of_few_rows_in_every_form(shape):
    """Segments of odd sizes inside one or two row tiles."""
    _form_is(shape)
    _, n_out, k_in, _, n_tok = shape
    x, _, codes, scales = T._inputs(n_out, k_in, 1, n_tok, 33)
    lin = T._linear(codes, scales)
    y = torch.empty((n_tok, n_out), device="cuda")
    lin(x.cuda(), y)
    rows = [1, 33, 127, 2, 36, 3]
    rows.append(n_out - sum(rows))
    outs = [torch.full((n_tok + 1, r), 5.0, dtype=torch.bfloat16 if s % 2 else torch.float32, device="cuda") for s, r in enumerate(rows)]
    lin(x.cuda(), [t[:n_tok] for t in outs])
    for t, part in zip(outs, y.split(rows, dim=1)):
        assert torch.equal(t[:n_tok], part.to(t.dtype)) and bool((t[n_tok] == 5).all())
    lin.check_device_error()


FIRST_CALLS_CAPTURED = """
import torch
from compressed_sparse_long_hca_b200 import _lib
from compressed_sparse_long_hca_b200.api import LinearFP8
from tests import fp8_forms as F
g = torch.Generator(device="cuda").manual_seed(1)
calls = []
for form, n_out, k, groups, n_tok in F.SHAPES:
    assert _lib.load().csa_debug_fp8_form(n_out, k, groups, n_tok, 0) == form
    lin = LinearFP8.quantize(torch.randn((n_out, k // groups), generator=g, device="cuda"), groups=groups)
    x = torch.randn((n_tok, k), generator=g, device="cuda").to(torch.bfloat16)
    calls.append((lin, x, torch.zeros((n_tok, n_out), device="cuda")))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for lin, x, y in calls:
        lin(x, y)
graph.replay()
for _, x, _ in calls:
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
graph.replay()
for lin, x, y in calls:
    z = torch.zeros_like(y)
    lin(x, z)
    assert bool((z != 0).any()) and torch.equal(y, z), tuple(y.shape)
LinearFP8.check_device_error()
print("captured")
"""


def test_the_first_call_of_every_form_can_be_captured():
    """In a process of its own: every kernel's set-up happens inside a capture,
    and calls of all forms follow each other in one graph."""
    import os
    import subprocess
    import sys
    _form_is(F.SHAPES[0])
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n_tok", [3, 40, 300])
def test_in_place_is_refused(n_tok):
    from compressed_sparse_long_hca_b200.api import LinearFP8
    lin = LinearFP8.quantize(np.eye(1024, dtype=np.float32))
    x = torch.ones((n_tok, 1024), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="overlaps x"):
        lin(x, x)
    y = torch.empty_like(x)
    lin(x, y)
    assert torch.equal(x, y)
