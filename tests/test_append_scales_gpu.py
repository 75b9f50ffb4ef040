"""smla_cache_append into blocks whose scale another writer left."""
import pytest
import torch

from tests import _paged as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before", [0.0, 2.0 ** -100, 2.0 ** -64])
def test_older_rows_of_a_tiny_scale_keep_their_values(cuda_lib, before):
    """A block whose older rows have the scale 0 (values 0, whatever their codes) or one
    below what the append writes: their values stay what they were, to E4M3's grid."""
    smla = cuda_lib
    torch.manual_seed(1)
    smla.smla_get_device_status(clear=True)
    block, old = 64, 40
    for new in (1.0, 0.0, 2.0 ** -60):                 # the new rows' values
        cache = torch.randint(1, 120, (2 * block, 512), device="cuda").to(torch.uint8)
        scale = torch.full((2,), before, device="cuda")
        was = cache.clone()
        x = (torch.rand((3, 512), device="cuda") + 1).bfloat16() * new
        start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        lens = torch.tensor([old + 3], dtype=torch.int32, device="cuda")
        tab = torch.tensor([[1]], dtype=torch.int32, device="cuda")
        smla.smla_cache_append(x, None, None, start, lens, tab, block, cache, P.BLOCK, scale)
        s = float(scale[1])
        assert s == max(P.block_scale(float(x.float().max())), before)
        val = lambda c: c.view(torch.float8_e4m3fn).double()   # noqa: E731
        want, got = val(was[block:block + old]) * before, val(cache[block:block + old]) * s
        assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s).all())
        if before == 0:
            assert bool((got == 0).all())
        assert torch.equal(cache[:block], was[:block])
        assert torch.equal(cache[block + old + 3:], was[block + old + 3:])
        row = val(cache[block + old:block + old + 3]) * s
        assert bool(((row - x.double()).abs() <= 2.0 ** -4 * x.double() + 2.0 ** -10 * s).all())
    assert smla.smla_get_device_status(clear=True) == 0
