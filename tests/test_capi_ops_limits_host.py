"""What the binding and the training operators' entry points accept and refuse
at the edges: no GPU needed, no call here reaches a launch."""
import enum
import random

import numpy as np
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


def fits(z, coefs):
    return z.zero_orthogonalize_workspace_bytes(z.matrices(32, 64, coefs=coefs)) > 0


def largest(coefs, points):
    """The largest s^2 and |b s^2 + c s^4| that a dense grid of [0, 1] meets."""
    s, worst = np.linspace(0.0, 1.0, points), 0.0
    with np.errstate(over="ignore", invalid="ignore"):
        for a, b, c in coefs:
            g = s * s
            p = b * g + c * g * g
            worst = max(worst, float(np.nanmax(g)), float(np.nanmax(np.abs(p))))
            s = s * (a + p)
    return worst


# the slopes of the steps multiply: these leave fp16's range between the points
# of any coarse grid (3.6 and 3.4 at most over 513 points)
@pytest.mark.parametrize("step,times", [((2.12717, -4.55896, 1.43027), 9), ((2.13721, -4.81709, 1.67575), 8)])
def test_schedules_that_leave_the_range_between_samples_are_refused(z, step, times):
    assert largest([step] * times, 513) < 5.0 and largest([step] * times, 4_000_001) > 15.0
    assert not fits(z, [step] * times)
    # while the same steps cut off before they leave it are accepted
    n = max(k for k in range(1, times) if largest([step] * k, 4_000_001) < 14.0)
    assert fits(z, [step] * n)


def test_schedules_are_followed_exactly(z):
    rng = random.Random(5)
    taken = 0
    for _ in range(400):
        coefs = [tuple(np.float32(v) for v in (rng.uniform(0.5, 4.5), rng.uniform(-7, 1), rng.uniform(-1, 4)))
                 for _ in range(rng.randint(1, 4))]
        worst = largest([tuple(map(float, c)) for c in coefs], 200_001)
        if worst > 15.001:
            assert not fits(z, coefs)
        elif worst < 14.5:
            # at most four steps of slope under 60: the grid is within 0.5 of the true bound
            assert fits(z, coefs)
            taken += 1
    assert 40 < taken < 360
    for coefs in ([(0.0, 0.0, 0.0)], [(1.0, 0.0, 0.0)] * 32, [(-1.5, 0.5, 0.0)] * 12, [(0.0, 2.5, -1.5)] * 3,
                  [(3.4445, -4.7750, 2.0315)] * 32):
        assert fits(z, coefs)
    for coefs in ([(float("inf"), 0.0, 0.0)], [(0.0, float("nan"), 0.0)], [(1e30, 0.0, 0.0)] * 2, [(3.9, 0.0, 0.0)] * 2):
        assert not fits(z, coefs)


def test_muon_flags_are_checked(z):
    import ctypes
    a, b, c, d, e, f, g = (0x100000000 * k for k in range(1, 8))

    def muon(sc=g, nesterov=1, loss_scaling=0, clipping=0):
        hp, opts = z.muon_hparams(), z._capi.ZeroMuonOpts(loss_scaling, clipping)
        hp.nesterov = nesterov
        ranks = (ctypes.c_void_p * 2)(a, b)
        return z._capi.raw_status("zero_muon_step_ex", ctypes.byref(z.matrices(32, 64)), ctypes.byref(hp), ctypes.byref(opts),
                                  2, ranks, c, d, e, f, sc, None)

    for k in ("nesterov", "loss_scaling", "clipping"):
        assert muon(**{k: 2}) == 1 and muon(**{k: -1}) == 1
    # what they read is the scalars block
    assert muon(sc=None, loss_scaling=1) == 1 and muon(sc=None, clipping=1) == 1
    # the hyper-parameters' layout is what it was
    assert ctypes.sizeof(z._capi.ZeroMuonHparams) == 24


# ------------------------------------------- the forms of the matrix updates
def test_the_tested_shapes_take_the_forms_they_stand_for(z):
    from matrix_forms import FORMS, MUON_FORMS, form_of
    for (rows, cols, batch, products), form in FORMS.items():
        assert form_of(z, rows, cols, batch, products) == (products, form), (rows, cols, batch, products)
    for (rows, cols, batch), form in MUON_FORMS.items():
        assert form_of(z, rows, cols, batch, 0, True) == (3, form), (rows, cols, batch)


def test_no_form_is_left_out(z):
    """Whatever form some shape takes has a shape that the GPU tests run."""
    from matrix_forms import FORMS, form_of
    tested = {(k[3], v) for k, v in FORMS.items()} | {(3, None)}
    rng = random.Random(11)
    reached = {}
    for _ in range(6000):
        rows, cols, batch = (int(2 ** rng.uniform(0, e)) for e in (13, 13, 6))
        if rows * cols * batch > 1 << 26:
            continue
        for products in (1, 3):
            reached.setdefault(form_of(z, rows, cols, batch, products), (rows, cols, batch))
    missing = {f: s for f, s in reached.items() if f not in tested}
    assert not missing
    assert len(reached) >= 12


def test_matrix_plan_arguments_are_checked(z):
    d = z.matrices(300, 400)
    for muon, sms in ((2, 152), (-1, 152), (False, 1)):
        with pytest.raises(z.ZeroError):
            import ctypes
            out = z._capi.ZeroMatrixPlan()
            z._capi._check(z._capi.raw_status("zero_debug_matrix_plan", ctypes.byref(d), muon, sms, ctypes.byref(out)), "plan")
    assert z._capi.raw_status("zero_debug_matrix_plan", None, 0, 152, None) == 1
    for sms in (2, 3, 64, 152, 160, 1000):
        p = z.zero_debug_matrix_plan(d, sms=sms)
        assert p.groups * p.units * (p.tile_rows // 128) <= min(sms, 160)
