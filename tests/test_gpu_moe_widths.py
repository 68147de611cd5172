"""q8_moe at the widths where its tiling has a remainder: stages of 128 columns of either product
(32, 64 or 96 left over), one segment of the down product or several, segments that differ in
length, experts with more than 8 tokens, and tasks that 2, 4 or 8 warps share, with fewer
stages than warps among them."""
import pytest

import test_gpu_moe as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [128, 160, 192, 224, 1056, 2016])
@pytest.mark.parametrize("F", [128, 160, 192, 224])
def test_left_over_columns(H, F):
    moe.run(5, 4, H, F, 2, seed=H + F)


@pytest.mark.parametrize("T,E,k", [(3, 4, 2), (32, 2, 2), (20, 3, 1)])
@pytest.mark.parametrize("F", [480, 512, 544, 1024, 1056, 1504, 1536, 1568, 2048, 2080, 3104])
def test_segments_of_the_down_product(T, E, k, F):
    moe.run(T, E, 96, F, k, seed=F + T)


@pytest.mark.parametrize("H,F", [(32, 32), (128, 32), (256, 64), (288, 160), (1024, 64), (1056, 512), (4096, 32), (8192, 64)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 3, 2), (9, 1, 1), (32, 1, 1)])
def test_tasks_that_warps_share(H, F, T, E, k):
    # few tasks a CTA and from one stage of columns to 64
    moe.run(T, E, H, F, k, seed=H + F + T)
