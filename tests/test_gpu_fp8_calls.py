"""How the FP8 product is called: on other streams than the current one, and
in the special cases that every form of its launch has to keep."""
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
