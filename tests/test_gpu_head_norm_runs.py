"""GPU parity of the head norms where blocks take runs of tokens, for heads of
520 to 768 values (three steps of a warp, by the kernel of four)."""
import pytest

from tests import test_gpu_head_norm as N

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return cuda_lib


@pytest.mark.parametrize("n,H,HK,D,R,qt,kt,rot", [
    (1200, 9, 0, 576, 64, BF, BF, False), (1001, 5, 3, 768, 64, BF, F32, True), (1300, 2, 1, 520, 520, F32, BF, True),
    (901, 6, 1, 640, 0, F32, F32, True), (1190, 3, 2, 514, 6, BF, BF, True), (2300, 1, 1, 766, 30, BF, BF, False)])
def test_many_tokens_of_few_long_heads(n, H, HK, D, R, qt, kt, rot):
    N.test_matches_the_oracle(n, H, HK, D, R, qt, kt, rot)
