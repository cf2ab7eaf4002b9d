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


def test_attention_of_different_groups_in_new_threads():
    """Calls of threads that made no CUDA call before: their tensor maps want a context."""
    lib, jobs, want, got, keep = B.lib(), [], [], [], []
    for G in (1, 8, 4):
        Bn, L, H, d, n, P = 3, 1, 2, 128, 100, 200
        m = B.model(L, H * G, H, d)
        q, K, V, Kp, Vp = [torch.randn(*s, device=DEV).to(torch.bfloat16)
                           for s in ((Bn, L, H * G, d), (Bn, L, H, n, d), (Bn, L, H, n, d), (L, H, P, d), (L, H, P, d))]
        o = torch.empty(Bn, L, H * G, d, device=DEV)
        kw = dict(q=q, o=o, K=K, V=V, lens=torch.full((Bn, L), n, dtype=torch.int32, device=DEV), max_len=n)
        if G > 1:
            kw.update(K_prefix=Kp, V_prefix=Vp, lens_prefix=torch.full((L,), P, dtype=torch.int32, device=DEV), max_len_prefix=P)
        ws = B.kvc_prefix_decode_attn(m, **kw)
        want.append(o.clone())
        got.append(o)
        a = B.prefix_decode_args(m, **kw)
        keep.append((m, a, kw, ws))
        jobs.append(lambda s, m=m, a=a, ws=ws: lib.kvc_prefix_decode_attn(C.byref(m), C.byref(a), ws.data_ptr(), ws.numel(), s))
    assert together(jobs) == {0}
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert B.kvc_check_status() == 0


def test_decode_in_a_new_thread():
    Bn, L, Hq, H, d, n = 2, 2, 8, 2, 128, 300
    m = B.model(L, Hq, H, d)
    q, K, V = [torch.randn(*s, device=DEV).to(torch.bfloat16) for s in ((Bn, L, Hq, d), (Bn, L, H, n, d), (Bn, L, H, n, d))]
    first, o = torch.empty(Bn, L, Hq, d, device=DEV), torch.empty(Bn, L, Hq, d, device=DEV)
    kw = dict(q=q, K=K, V=V, lens=torch.full((Bn, L), n, dtype=torch.int32, device=DEV), max_len=n)
    before = B.kvc_launch_count()
    ws = B.kvc_decode_attn(m, o=first, **kw)
    launches = B.kvc_launch_count() - before
    raised, stream = [], torch.cuda.current_stream()

    def work():
        try:
            B.kvc_decode_attn(m, o=o, workspace=ws, stream=stream, **kw)
        except Exception as e:                                       # noqa: BLE001
            raised.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert raised == [] and torch.equal(o, first)
    assert B.kvc_launch_count() - before == 2 * launches            # by the same kernels
    assert B.kvc_check_status() == 0
