"""Layer norm where it can go wrong beside its shapes: calls from two host
threads, rows of huge values, widths above 8192 with many rows."""
import ctypes
import threading

import pytest
import torch

import zero_optimizer_step_02_gb300 as z

pytestmark = pytest.mark.gpu


def test_two_host_threads_each_with_its_own_stream():
    # two widths of one kernel that ask for different amounts of shared memory;
    # the threads share no workspace, so no order between their calls is asked
    # for and each call has to succeed
    calls, errors = 3000, []
    start = threading.Barrier(2)

    def work(cols):
        x = torch.randn(2048, cols, device="cuda").bfloat16()
        dy = torch.randn(2048, cols, device="cuda").bfloat16()
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(2048, device="cuda"), torch.empty(2048, device="cuda")
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        d = z.layernorm(2048, cols)
        ws = torch.empty(z.zero_layernorm_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        ptr = [ctypes.c_void_p(t.data_ptr()) for t in (x, y, mean, rstd, dy, dx, dg, db, ws)]
        stream = ctypes.c_void_p(s.cuda_stream)
        start.wait()
        for _ in range(calls):
            a = z._capi.raw_status("zero_layernorm_forward", ctypes.byref(d), ptr[0], None, None, ptr[1], ptr[2], ptr[3],
                                   stream)
            b = z._capi.raw_status("zero_layernorm_backward", ctypes.byref(d), ptr[4], ptr[0], None, ptr[2], ptr[3],
                                   ptr[5], ptr[6], ptr[7], ptr[8], stream)
            if a != 0 or b != 0:
                errors.append((cols, a, b))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in (4096, 1536)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []
