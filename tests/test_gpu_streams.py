"""GPU: calls on a stream other than the current one: what they allocate and copy belongs to that stream."""
import pytest
import torch

from long_context_kv_obs_b200 import binding as B
from long_context_kv_obs_b200.pipeline import SharedPromptBatch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def i32(x, *shape):
    return torch.full(shape, x, dtype=torch.int32, device=DEV)


def ready(**kw):
    """Arguments whose contents are there, whatever stream reads them."""
    torch.cuda.synchronize()
    return kw


def attention():
    Bn, L, Hq, H, d, n, P = 2, 2, 8, 2, 128, 300, 500
    q, K, V, Kp, Vp = [torch.randn(*s, device=DEV).to(BF) for s in
                       ((Bn, L, Hq, d), (Bn, L, H, n, d), (Bn, L, H, n, d), (L, H, P, d), (L, H, P, d))]
    kw = ready(q=q, o=torch.empty(Bn, L, Hq, d, device=DEV), K=K, V=V, lens=i32(n, Bn, L), max_len=n, K_prefix=Kp,
               V_prefix=Vp, lens_prefix=i32(P, L), max_len_prefix=P)
    return lambda s: B.kvc_prefix_decode_attn(B.model(L, Hq, H, d), stream=s, **kw)


def decode():
    Bn, L, Hq, H, d, n = 2, 2, 8, 2, 128, 4000
    q, K, V = [torch.randn(*s, device=DEV).to(BF) for s in ((Bn, L, Hq, d), (Bn, L, H, n, d), (Bn, L, H, n, d))]
    kw = ready(q=q, K=K, V=V, lens=i32(n, Bn, L), max_len=n, o=torch.empty(Bn, L, Hq, d, device=DEV))
    return lambda s: B.kvc_decode_attn(B.model(L, Hq, H, d), stream=s, **kw)


def tables():
    lens = i32(0, 5)
    kw = ready(lens=lens, lens_new=i32(20, 5), lens_out=lens, table=i32(-1, 5, 2),
               state=torch.tensor([0, 40], dtype=torch.int32, device=DEV), ring=torch.arange(40, dtype=torch.int32, device=DEV))
    return lambda s: B.kvc_page_tables(page=16, stream=s, **kw)


def select():
    kw = ready(S=torch.rand(2, 2, 1000, device=DEV), k_out=i32(0, 2), idx=i32(0, 2, 2, 400))
    return lambda s: B.kvc_select(B.model(2, 8, 2, 128), n=1000, w=16, rho=0.25, stream=s, **kw)


@pytest.mark.parametrize("make", [attention, decode, tables, select])
def test_a_workspace_made_by_a_call_is_its_streams_own(make):
    """Given back, its memory is not handed out on the current stream, where earlier work may still be under way."""
    call, s = make(), torch.cuda.Stream()
    call(s)                                                          # what a first call sets up
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ws = call(s)
    torch.cuda.synchronize()
    at, n = ws.data_ptr(), ws.numel()
    del ws
    here = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(200)]
    assert all(x.data_ptr() != at for x in here)
    with torch.cuda.stream(s):
        there = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(200)]
    assert any(x.data_ptr() == at for x in there)
    assert B.kvc_check_status() == 0


def test_a_step_copies_strided_rows_on_its_own_stream():
    """k and v as [L][B][H][d] memory cannot be viewed as rows: their copies are made, and kept, on the step's stream."""
    Bn, L, Hq, H, d = 3, 4, 8, 2, 128
    m = B.model(L, Hq, H, d)
    Kp, Vp = [torch.randn(L, H, 100, d, device=DEV).to(BF) for _ in range(2)]
    sb = SharedPromptBatch(m, Kp, Vp, i32(100, L), batch=Bn, n_pages=Bn * L, max_len=16)
    k, v = [torch.randn(L, Bn, H, d, device=DEV).to(BF).transpose(0, 1) for _ in range(2)]
    q = torch.randn(Bn, L, Hq, d, device=DEV).to(BF)
    s, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    sb.step(q, v, k, stream=s)                                       # what a first step sets up
    torch.cuda.synchronize()
    torch.cuda._sleep(2 ** 30)                                       # half a second: the current stream is busy
    done.record()
    sb.step(q, k, v, stream=s)
    s.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    at = sb.slots.view(Bn, L).tolist()
    for b in range(Bn):
        for l in range(L):
            page, i = divmod(at[b][l], 16)
            assert i == 1 and torch.equal(sb.K[page, :, 1], k[b, l]) and torch.equal(sb.V[page, :, 1], v[b, l])
    assert B.kvc_check_status() == 0
