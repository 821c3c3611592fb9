"""Every form that the orthogonalised update and the Muon step take, at the
smallest sizes that reach it, against 64 bits.

Tolerances.  Three products: as in test_gpu_muon.  One product: each operand
rounded to fp16 is off by 2e-4 root mean square, the five of a step are
independent of one another over 256 terms and more (sqrt(5) * 2e-4 = 4.5e-4),
and the steps add up in full at worst: 2.3e-3 of the 2-norm.  The errors of
single elements are spread like the elements: eight times that of the root mean
square, plus the element's own rounding."""
import pytest
import torch

import zero_optimizer_step_02_gb300 as z
from matrix_forms import FORMS, MUON_FORMS, form_of
from test_gpu_muon import BF16, FP32, UNIT, Job, gradients, orthogonalize, plain, tolerance

pytestmark = pytest.mark.gpu


def allowed(rows, cols, products, out_dt):
    return 2.3e-3 + UNIT[out_dt] if products == 1 else tolerance(rows, cols, 3, out_dt)


def check(got, want, tol, unit):
    for a, b in zip(got.double(), want):
        d, rms = a - b, float(b.norm()) / b.numel() ** 0.5
        assert float(d.norm()) <= tol * float(b.norm())
        assert bool((d.abs() <= 8 * tol * rms + unit * b.abs()).all())


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("rows,cols,batch,products", list(FORMS))
def test_form(rows, cols, batch, products):
    assert form_of(z, rows, cols, batch, products, sms=sms()) == (products, FORMS[rows, cols, batch, products])
    g = gradients(batch, rows, cols)
    x, o = orthogonalize(g, FP32, FP32, products)
    check(o, plain(x), allowed(rows, cols, products, FP32), UNIT[FP32])
    again = orthogonalize(g, FP32, FP32, products)[1]
    assert torch.equal(o, again)


# each matrix in one SM
@pytest.mark.parametrize("rows,cols,batch", [(96, 160, 2), (128, 256, 1), (256, 128, 1), (15, 17, 1), (113, 65, 2),
                                             (64, 64, 200), (100, 193, 3)])
def test_one_sm_form(rows, cols, batch):
    assert form_of(z, rows, cols, batch, 3, sms=sms()) == (3, None)
    x, o = orthogonalize(gradients(batch, rows, cols), FP32, FP32, 3)
    check(o, plain(x), allowed(rows, cols, 3, FP32), UNIT[FP32])


# results of two bytes, rows that do not lie on whole words, by the default choice of products
@pytest.mark.parametrize("rows,cols,batch", [(768, 768, 12), (1004, 4541, 3), (4046, 1032, 1), (2304, 2304, 1)])
def test_bf16_results_by_default(rows, cols, batch):
    assert form_of(z, rows, cols, batch, 1, sms=sms())[0] == 1
    x, o = orthogonalize(gradients(batch, rows, cols), BF16, BF16, 0, out_ld=cols + 3, gap=5)
    check(o, plain(x), allowed(rows, cols, 1, BF16), UNIT[BF16])


@pytest.mark.parametrize("rows,cols,batch", list(MUON_FORMS))
def test_muon_form(rows, cols, batch):
    assert form_of(z, rows, cols, batch, 0, True, sms=sms()) == (3, MUON_FORMS[rows, cols, batch])
    job = Job(rows, cols, batch, 2, BF16, gap=8)
    job.new_grads(0)
    m0, w0 = job.view(job.momentum).double(), job.view(job.master).double()
    mean = sum(job.view(t).double() for t in job.grads) / 2
    job.step_and_check()
    # element by element, as above: the update is step * o
    step = 0.02 * 0.2 * max(rows, cols) ** 0.5
    o = plain(mean + 0.95 * (0.95 * m0 + mean))
    err = (job.view(job.master).double() - (w0 * (1 - 0.02 * 0.1) - step * o)).abs()
    tol = allowed(rows, cols, 3, FP32) + 1e-6
    for i in range(batch):
        rms = float(o[i].norm()) / o[i].numel() ** 0.5
        assert bool((err[i] <= step * (8 * tol * rms + UNIT[FP32] * o[i].abs()) + 4 * UNIT[FP32] * (w0[i].abs() + step * o[i].abs())).all())
