"""Host-side test of the 4-bit cache's handle."""
import pytest

import exact_scaled_dot_gb300 as esd


@pytest.mark.parametrize("name", ["pool", "device", "pages", "Hkv", "d_h", "d_v"])
def test_the_pool_and_its_sizes_are_read_only(name):
    """The library gets the pool's address and sizes as they were given; a tensor assigned later would not be used."""
    with pytest.raises(AttributeError):
        setattr(esd.QuantCache.__new__(esd.QuantCache), name, 1)
