"""Tree attention with one or two key/value heads for many query heads, up to
more groups of query rows than the chip holds workgroups at once (no range is
cut then)."""
import pytest

from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,Hq,H,D,lens", [(1, 64, 1, 128, [700, 0]), (8, 128, 1, 64, [300, 33]), (5, 96, 2, 256, [131]),
                                           (64, 512, 1, 64, [40])])
def test_many_query_heads(n, Hq, H, D, lens, dtype):
    Case(900 + Hq, dtype, n, Hq, H, D, 64, lens, mask="tree").check()
