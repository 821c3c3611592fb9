"""What the binding and the training operators' entry points accept and refuse
at the edges: no GPU needed, no call here reaches a launch."""
import enum

import pytest


@pytest.fixture(scope="module")
def z():
    import __graft_entry__
    __graft_entry__.build()
    import zero_optimizer_step_02_gb300 as z
    return z


def test_addresses_may_be_any_kind_of_int(z):
    class Address(int):
        pass

    class Buffers(enum.IntEnum):
        MASTER = 0x7000000

    assert z._capi._addr(Address(0x1234500)) == 0x1234500
    assert z._capi._addr(Buffers.MASTER) == 0x7000000
    assert z._capi._addr(None) is None and z._capi._addr(16) == 16
    arr = z.rank_ptrs([Address(0x1000), Buffers.MASTER, 0x2000])
    assert list(arr) == [0x1000, 0x7000000, 0x2000]
    # through an entry point: refused for its alignment, not for its type
    with pytest.raises(z.ZeroError):
        z.zero_scalars_init(Address(0x1234501), stream=Address(0))
