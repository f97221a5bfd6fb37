"""Which kernels a call of given bounds takes, told by the workspace it asks for."""
import pytest

from compressed_kv_cache_gva_b200 import gva
from test_gpu_paged import A, BF, Batch
from test_gpu_paged_workspace import required, shape

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(16, 4, 32, 24), (16, 4, 32, 0), (12, 4, 32, 8)])
def test_long_batches_of_narrow_heads_keep_to_one_kernel(heads):
    """Nine to 16 columns of d_h = 32: no tcgen05 row blocks exist, so a long batch of mostly
    single tokens must not be sent to two kernels, the second of them on CUDA cores."""
    most = 4
    sh = shape(heads, 64)
    below = required(sh, 16, 112, most, (96 << 20) // 256 - 1)
    assert required(sh, 16, 112, most, (96 << 20) // 256) == below
    assert required(sh, 16, 112, most, 1 << 22) == below


def test_long_batches_of_wide_heads_take_two_kernels():
    sh = shape(A, 64)
    assert required(sh, 16, 112, 4, (96 << 20) // 512) != required(sh, 16, 112, 4, (96 << 20) // 512 - 1)


def test_a_narrow_batch_above_the_bound_is_right():
    x = Batch((16, 4, 32, 24), 16, [37, 200, 64, 90, 1, 5], [1, 4, 1, 1, 1, 0], seed=6)
    x.check(x.run(BF, total=1 << 19), x.reference(), BF, 2.0 ** -16)
