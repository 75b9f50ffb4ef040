"""Copies of as many pairs as an int counts."""
import pytest
import torch

from tests import _paged as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 700])
def test_pairs_up_to_the_end_of_int32(cuda_lib, n):
    """The pairs past the first and before the last are passed over.  (The number that a
    CTA goes on to passes 2^31.)"""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, (8 * 16, 512), dtype=torch.uint8, device="cuda", generator=g)
    want = cache.clone()
    src = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    dst = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    for i, (a, b) in zip((0, n // 2, n - 2, n - 1), ((1, 0), (1, 2), (3, 4), (7, 6))):
        src[i], dst[i] = a, b
        want[16 * b:16 * b + 16] = want[16 * a:16 * a + 16]
    smla.smla_cache_copy(cache, P.E4M3, None, src, dst, 16)
    assert torch.equal(cache, want)
    assert smla.smla_get_device_status(clear=True) == 0
    del src, dst
    torch.cuda.empty_cache()
