"""The paged 4-bit cache on the GPU where it can go wrong: ends of the number ranges, calls that are refused on the device,
shares of work without pages.  The reference and the tolerance are those of test_gpu_kv4.py, where nothing else is said."""
import pytest
import torch

from test_gpu_kv4 import BF16, attend, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device(cuda_ok):
    torch.cuda.set_device(0)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1], [64], [256], [300]], ids=str)
def test_canvas_with_fewer_pages_than_its_cluster_has_ctas(lens, causal):
    """A CTA without pages sends a row of weight 0 through the place of its queries: none of their bits may come with it.
    (Such bf16 queries, read as fp16, are infinities and NaN.)"""
    for seed in range(4):
        c = make(2, 128, lens, seed=seed)
        attend(c, 2, 256, BF16, causal=causal, seed=seed, q_scale=2.0 ** 122, scale=2.0 ** -124)
        attend(c, 2, 256, BF16, rows=[130], causal=causal, seed=seed, q_scale=2.0 ** 122, scale=2.0 ** -124)
