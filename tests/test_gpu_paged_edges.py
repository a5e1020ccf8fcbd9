"""The paged operators at the ends of their arguments' ranges."""
import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

R = pytest.importorskip("recurrent_depth_moe_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    R.load_library()


@pytest.mark.parametrize("hd", [1, 8])
@pytest.mark.parametrize("t_out", [2 ** 31 - 1, 2 ** 31 - 100])
def test_read_into_rows_up_to_the_largest_int(hd, t_out):
    """Outputs of nearly 2^31 rows (2 x 4 GiB at one channel, 2 x 32 GiB at 8): the cached positions,
    and everything behind them as it was."""
    if torch.cuda.mem_get_info()[0] < 2 * t_out * hd * 2 + (2 << 30):
        pytest.skip("needs the memory")
    cache = S.make_cache(R, 1, 1, hd, 48, 16, "bf16", False, 3)
    out = tuple(torch.full((1, 1, t_out, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    R.paged_kv_read(torch.tensor([40], dtype=torch.int32, device="cuda"), cache, out=out)
    for o, x in zip(out, S.cached(cache, 0, 40)):
        assert torch.equal(o[0, 0, :40].cpu().double(), x[0])
        for at in (40, 1 << 20, 1 << 30, t_out - 1000):
            assert (o[0, 0, at:at + 1000] == 7.0).all(), at
    assert cache.read_status() == 0
