"""The Muon step under the step's loss scaling and clipping: what it takes from
the scalars block, and steps that are skipped."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_02_gb300 as z
from test_gpu_muon import BF16, FP16, Job

pytestmark = pytest.mark.gpu

# one SM's form, the general form; a last word of fewer than eight elements
SHAPES = [(2, 96, 160), (3, 33, 17), (2, 300, 520), (1, 257, 301)]


def state(job):
    return [t.clone() for t in (job.momentum, job.master, job.lp)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def step(job, loss_scaling=False, clipping=False, **hp):
    z.zero_muon_step_ex(job.desc, z.muon_hparams(**dict(job.hp, **hp)), job.grads, job.momentum, job.master, job.lp, job.ws,
                        job.sc, loss_scaling, clipping)
    torch.cuda.synchronize()


def set_scalars(job, **kw):
    s = z.read_scalars(job.sc)
    for k, v in kw.items():
        setattr(s, k, v)
    raw = torch.frombuffer(bytearray(bytes(s)), dtype=torch.uint8)
    job.sc[: len(raw)] = raw.cuda()


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), "sum"])
def test_an_overflow_leaves_everything_as_it_was(batch, rows, cols, bad):
    job = Job(rows, cols, batch, 3, FP16)
    z.zero_scalars_init(job.sc, 1024.0)
    job.new_grads(0)
    job.view(job.lp).zero_()
    last = (batch - 1, rows - 1, cols - 1)
    if bad == "sum":       # infinities of both signs: each rank's own, NaN in the sum
        job.view(job.grads[0])[last], job.view(job.grads[2])[last] = float("inf"), float("-inf")
    else:
        job.view(job.grads[1])[last] = bad
    before = state(job)
    step(job, loss_scaling=True)
    sc = z.read_scalars(job.sc)
    assert same(before, state(job))
    assert sc.nonfinite == 1 and sc.status == 0 and sc.loss_scale == 1024.0 and sc.t == 0
    # a later call of the same step skips too, whatever its own gradients
    other = Job(rows, cols, batch, 3, FP16)
    other.new_grads(0)
    other.sc = job.sc
    before = state(other)
    step(other, loss_scaling=True)
    assert same(before, state(other))


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_the_adam_step_of_a_flagged_step_is_skipped_and_the_next_one_counts(batch, rows, cols):
    hp = z.hparams(loss_scaling=True)
    vec = z.StepBuffers(z.Plan(1000, 2, stage=2, grad_dtype=FP16), hp)
    vec.init_scalars(512.0)
    vec.master.normal_()
    vec.grads.normal_()
    job = Job(rows, cols, batch, 2, FP16)
    job.sc = vec.scalars
    for k, bad in enumerate((False, True, False)):
        job.new_grads(k)
        if bad:
            job.view(job.grads[0])[0, 0, 0] = float("inf")
        muon, adam = state(job), [vec.master.clone(), vec.m.clone()]
        step(job, loss_scaling=True)
        vec.step(hp)
        sc = vec.scalars_host()
        assert same(muon, state(job)) == bad and torch.equal(adam[0], vec.master) == bad
        assert sc.nonfinite == 0 and sc.overflow == int(bad)
        assert (sc.t, sc.loss_scale) == ((1, 512.0), (1, 256.0), (2, 256.0))[k]
        assert bool(torch.isfinite(job.view(job.master)).all())


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_the_scale_is_the_scalars_block_s(batch, rows, cols):
    # the same bits as with the same scale by value
    a, b = (Job(rows, cols, batch, 3, FP16, loss_scale=256.0) for _ in range(2))
    z.zero_scalars_init(a.sc, 256.0)
    for job in (a, b):
        job.new_grads(0)
    step(a, loss_scaling=True, loss_scale=3.0)
    step(b)
    assert same(state(a), state(b))
    assert z.read_scalars(a.sc).nonfinite == 0


def test_a_flag_of_the_reduce_pass_skips():
    hp = z.hparams(loss_scaling=True)
    plan = z.Plan(64, 2, stage=2, grad_dtype=FP16)
    vec = z.StepBuffers(plan, hp)
    vec.init_scalars(1.0)
    vec.grads.zero_()
    vec.grads[1, 63] = float("inf")
    z.zero_reduce_scatter(plan.handle, vec.rank_list(), hp, vec.scalars, torch.empty(plan.padded, device="cuda"), vec.ws)
    job = Job(130, 140, 1, 2, FP16)
    job.sc = vec.scalars
    job.new_grads(0)
    before = state(job)
    step(job, loss_scaling=True)
    assert same(before, state(job))
    step(job)                      # not a call under loss scaling: the flag is not its own
    assert not same(before, state(job))


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_the_clip_coefficient_multiplies_the_mean(batch, rows, cols):
    job = Job(rows, cols, batch, 3, BF16, nesterov=False)
    job.new_grads(0)
    set_scalars(job, clip_coef=0.37)
    # in numpy: IEEE operations one by one (torch divides by a number on the GPU through its reciprocal)
    f32 = lambda t: job.view(t).float().cpu().numpy()  # noqa: E731
    acc = np.zeros((batch, rows, cols), np.float32)
    for t in job.grads:
        acc = acc + f32(t)
    want = np.float32(0.95) * f32(job.momentum) + (acc / np.float32(3.0)) * np.float32(0.37)
    step(job, clipping=True)
    assert np.array_equal(f32(job.momentum), want)
    assert abs(z.read_scalars(job.sc).clip_coef - 0.37) < 1e-7


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_without_the_two_nothing_of_the_block_is_read(batch, rows, cols):
    a, b = (Job(rows, cols, batch, 3, BF16) for _ in range(2))
    for job in (a, b):
        job.new_grads(0)
    set_scalars(a, clip_coef=0.37, loss_scale=1024.0, nonfinite=1)
    before = z.read_scalars(a.sc)
    step(a)
    z.zero_muon_step(b.desc, z.muon_hparams(**b.hp), b.grads, b.momentum, b.master, b.lp, b.ws)
    torch.cuda.synchronize()
    assert same(state(a), state(b))
    assert bytes(before) == bytes(z.read_scalars(a.sc))


def test_skipped_and_taken_steps_in_one_graph():
    # the decision is the device's: one captured step, replayed with and without an overflow
    job = Job(96, 160, 2, 2, FP16)
    z.zero_scalars_init(job.sc, 1.0)
    job.new_grads(0)
    good = [t.clone() for t in job.grads]
    hp = z.muon_hparams(**job.hp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_muon_step_ex(job.desc, hp, job.grads, job.momentum, job.master, job.lp, job.ws, job.sc, loss_scaling=True)
    before = state(job)
    job.view(job.grads[1])[1, 5, 5] = float("inf")
    graph.replay()
    torch.cuda.synchronize()
    assert same(before, state(job))
    set_scalars(job, nonfinite=0)
    for t, g in zip(job.grads, good):
        t.copy_(g)
    graph.replay()
    torch.cuda.synchronize()
    assert not same(before, state(job)) and bool(torch.isfinite(job.view(job.master)).all())
