"""GPU: calls of several host threads at once.  What a call sets for its own launch must not reach another's."""
import ctypes as C
import threading

import pytest
import torch

from long_context_kv_obs_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = 4000


def together(jobs):
    """Every job(stream) CALLS times in a thread of its own, on a stream of its own: the statuses they returned.
    (Prebuilt arguments: the calls run without Python's lock and take most of a thread's time.)"""
    status, start = set(), threading.Barrier(len(jobs))
    streams = [torch.cuda.Stream() for _ in jobs]

    def work(job, stream):
        start.wait()
        status.update([job(stream) for _ in range(CALLS)])

    threads = [threading.Thread(target=work, args=(j, C.c_void_p(s.cuda_stream))) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return status


def test_samples_of_different_vocabularies():
    lib, jobs, want, got, keep = B.lib(), [], [], [], []
    for n, V in ((1, 500), (1, 262144), (80, 40000), (2, 16000)):
        z = torch.randn(n, V, device=DEV).to(torch.bfloat16)
        u, p, token = torch.rand(n, device=DEV), torch.full((n,), 0.9, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
        B.kvc_sample(logits=z, u=u, token=token, top_p=p)
        want.append(token.clone())
        got.append(token)
        a = B.SampleArgs()
        a.n, a.V, a.logits, a.dtype, a.row_stride = n, V, z.data_ptr(), B.KVC_BF16, V
        a.u, a.top_p, a.token = u.data_ptr(), p.data_ptr(), token.data_ptr()
        keep.append((z, u, p, a))
        jobs.append(lambda s, a=a: lib.kvc_sample(C.byref(a), s))
    assert together(jobs) == {0}
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert B.kvc_check_status() == 0
