"""GPU: a batch that answers from one compressed prompt, step by step as a user runs it - score, select,
compact and merge once, then page tables, append, shared-prompt attention and sampling - against
the fp64 oracle on the GPU's own compressed cache."""
import numpy as np
import pytest
import torch

from long_context_kv_obs_b200 import binding as B
from long_context_kv_obs_b200 import synth
from long_context_kv_obs_b200.pipeline import PrefillCompressor, SharedPromptBatch
from oracle import serving
from tests.helpers import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
# fp32 logits of d = 128 products of N(0, 1) entries (|q k| below 60 after the scale) are off by less than
# gamma_256 * 60 = 1.9e-3 of 2^-10, weights by 2^-16, outputs are means of values below 6: far inside 1e-3
ATOL = 1e-3


def compressed(seed=3, merge=True):
    wl = synth.WORKLOADS[3 if merge else 2].scaled(n_layers=2, n=1500, vocab=2000, hidden=256, bucket=256)
    inp = synth.gen_prefill(wl, seed=seed, device=DEV, with_logits=not merge, with_hidden=not merge)
    pc = PrefillCompressor(wl, inp, keep_A=True, merge=merge)
    pc.run()
    return wl, pc


def check_step(wl, pc, sb, o, q, own):
    k, G = pc.k.cpu().numpy(), wl.group
    on, qn = np64(o), np64(q)
    for b in range(len(own)):
        for l in range(wl.n_layers):
            for g in range(wl.n_kv_heads):
                n = int(k[l])
                kk = np.array([x[0][l, g] for x in own[b]]).reshape(-1, wl.head_dim)
                vv = np.array([x[1][l, g] for x in own[b]]).reshape(-1, wl.head_dim)
                want, lse, _ = serving.prefix_attention(qn[b, l, g * G:(g + 1) * G], np64(pc.Kc[l, g, :n]), np64(pc.Vc[l, g, :n]),
                                                        kk, vv, np64(pc.R[l, g, :n]) if pc.merge else None)
                assert np.abs(on[b, l, g * G:(g + 1) * G] - want).max() < ATOL
                assert np.abs(np64(sb.lse)[b, l, g * G:(g + 1) * G] - lse).max() < ATOL


@pytest.mark.parametrize("merge", [True, False])
def test_steps_releases_and_sampling_follow_the_oracle(merge):
    wl, pc = compressed(merge=merge)
    Bn, L, H, d = 5, wl.n_layers, wl.n_kv_heads, wl.head_dim
    sb = SharedPromptBatch(pc.m, pc.Kc, pc.Vc, pc.k, batch=Bn, n_pages=Bn * L * 3, max_len=40, R=pc.R if merge else None)
    g = torch.Generator(device=DEV).manual_seed(1)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)
    own = [[] for _ in range(Bn)]
    free = sb.ring.numel()
    for t in range(36):
        if t in (17, 20):                       # sequences end, their pages go back, others take their place
            keep = torch.ones(Bn, 1, dtype=torch.int32, device=DEV)
            gone = [1, 4] if t == 17 else [0]
            keep[gone] = 0
            sb.resize((sb.lens * keep).contiguous())
            for b in gone:
                own[b] = []
        q, k, v = draw(Bn, L, wl.n_q_heads, d), draw(Bn, L, H, d), draw(Bn, L, H, d)
        o = sb.step(q, k, v)
        for b in range(Bn):
            own[b].append((np64(k[b]), np64(v[b])))
        if t in (0, 15, 16, 17, 20, 35):
            check_step(wl, pc, sb, o, q, own)
        assert sb.lens.tolist() == [[len(x)] * L for x in own]
        held = sum(-(-len(x) // 16) * L for x in own)
        assert int(sb.state[1]) == free - held
    # no page is held twice
    used = [int(p) for b in range(Bn) for l in range(L) for p in sb.table[b, l, :-(-len(own[b]) // 16)]]
    ring, (head, count) = sb.ring.tolist(), sb.state.tolist()
    spare = [ring[(head + i) % free] for i in range(count)]
    assert sorted(used + spare) == list(range(free))
    z = synth.gen_logits(Bn, 3001, torch.bfloat16, seed=9, device=DEV, dominant=True)
    u = torch.rand(Bn, device=DEV, generator=g)
    p = torch.full((Bn,), 0.9, device=DEV)
    token = sb.sample(z, u, top_p=p, temperature=p)
    assert token.tolist() == [serving.sample(np64(z[b]), float(u[b]), temperature=float(p[b]), top_p=float(p[b]))[0]
                              for b in range(Bn)]
    assert B.kvc_check_status() == 0


def test_a_captured_step_replays_on_growing_rows():
    wl, pc = compressed(seed=4)
    Bn, L, H, d = 33, wl.n_layers, wl.n_kv_heads, wl.head_dim
    sb = SharedPromptBatch(pc.m, pc.Kc, pc.Vc, pc.k, batch=Bn, n_pages=Bn * L * 3, max_len=40, R=pc.R)
    g = torch.Generator(device=DEV).manual_seed(2)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)
    q, k, v = draw(Bn, L, wl.n_q_heads, d), draw(Bn, L, H, d), draw(Bn, L, H, d)
    z, u = synth.gen_logits(Bn, 5000, torch.bfloat16, seed=5, device=DEV, dominant=False), torch.rand(Bn, device=DEV)
    p = torch.full((Bn,), 0.95, device=DEV)
    own = [[] for _ in range(Bn)]

    def note():
        for b in range(Bn):
            own[b].append((np64(k[b]), np64(v[b])))

    sb.step(q, k, v)
    sb.sample(z, u, top_p=p)
    note()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = sb.step(q, k, v)
        token = sb.sample(z, u, top_p=p)
    for t in range(18):                         # the capture itself ran nothing
        for x in (q, k, v):
            x.copy_(draw(*x.shape))
        graph.replay()
        note()
    torch.cuda.synchronize()
    check_step(wl, pc, sb, o, q, own[:3])
    assert sb.lens.tolist() == [[19] * L] * Bn
    assert token.tolist() == [serving.sample(np64(z[b]), float(u[b]), top_p=float(p[b]))[0] for b in range(Bn)]
    assert B.kvc_check_status() == 0


def test_the_decode_call_and_the_shared_prompt_call_agree():
    """kvc_decode_attn over one cache that holds prompt and own rows, and the shared form: the same
    attention, each within its arithmetic of the other."""
    L, Hq, H, d, Bn, P, n = 2, 8, 2, 128, 6, 700, 50
    m = B.model(L, Hq, H, d)
    g = torch.Generator(device=DEV).manual_seed(3)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)
    Kp, Vp, Ko, Vo, q = draw(L, H, P, d), draw(L, H, P, d), draw(Bn, L, H, n, d), draw(Bn, L, H, n, d), draw(Bn, L, Hq, d)
    full = lambda a, b: torch.cat([a[None].expand(Bn, -1, -1, -1, -1), b], 3).contiguous()
    o1, o2 = torch.empty(Bn, L, Hq, d, device=DEV), torch.empty(Bn, L, Hq, d, device=DEV)
    i32 = lambda x, *s: torch.full(s, x, dtype=torch.int32, device=DEV)
    B.kvc_decode_attn(m, q=q, K=full(Kp, Ko), V=full(Vp, Vo), lens=i32(P + n, Bn, L), max_len=P + n, o=o1)
    B.kvc_prefix_decode_attn(m, q=q, K_prefix=Kp, V_prefix=Vp, lens_prefix=i32(P, L), max_len_prefix=P, K=Ko, V=Vo,
                             lens=i32(n, Bn, L), max_len=n, o=o2)
    assert float((o1 - o2).abs().max()) < 2e-5


def small_batch(Bn, L, max_len, n_pages, page=16, seed=6):
    """A batch on a prompt of 90 and 100 rows, fp32, and a function that runs a step and checks it."""
    Hq, H, d, P = 4, 2, 64, 100
    g = torch.Generator(device=DEV).manual_seed(seed)
    draw = lambda *s: torch.randn(*s, device=DEV, generator=g)
    m = B.model(L, Hq, H, d)
    Kp, Vp, R = draw(L, H, P, d), draw(L, H, P, d), 1 + 3 * torch.rand(L, H, P, device=DEV, generator=g)
    k = torch.tensor(([90, 100] * L)[:L], dtype=torch.int32, device=DEV)
    sb = SharedPromptBatch(m, Kp, Vp, k, batch=Bn, n_pages=n_pages, max_len=max_len, page=page, R=R)
    own = [[] for _ in range(Bn)]

    def step(live=None, stored=True, **kw):
        """One step; the rows that the sequences then hold, and how far its results are from the oracle's."""
        q, kk, vv = draw(Bn, L, Hq, d), draw(Bn, L, H, d), draw(Bn, L, H, d)
        o = np64(sb.step(q, kk, vv, **({} if live is None else dict(live=live)), **kw))
        for b in range(Bn):
            if stored and (live is None or bool(live[b])):
                own[b].append((np64(kk[b]), np64(vv[b])))
        worst = 0.0
        for b in range(Bn):
            for l in range(L):
                for h in range(H):
                    n, G = int(k[l]), Hq // H
                    ko, vo = [np.array([x[i][l, h] for x in own[b]]).reshape(-1, d) for i in (0, 1)]
                    want, lse, _ = serving.prefix_attention(np64(q[b, l, h * G:(h + 1) * G]), np64(Kp[l, h, :n]), np64(Vp[l, h, :n]),
                                                            ko, vo, np64(R[l, h, :n]))
                    worst = max(worst, np.abs(o[b, l, h * G:(h + 1) * G] - want).max(),
                                np.abs(np64(sb.lse)[b, l, h * G:(h + 1) * G] - lse).max())
        return worst

    return sb, own, step


# fp32, d = 64: a logit is off by at most gamma_64 (of 2^-23) of sum |q k| / 8 < 10, 7.6e-5; an output by twice that
# times the values' spread of about 1, and 150 sums and weights of 2^-23.  A key left out moves a row by some 1e-2.
STEP_ATOL = 2e-4


def test_every_token_that_is_stored_is_attended_and_a_full_row_refuses_the_step_as_a_whole():
    sb, own, step = small_batch(3, 2, max_len=40, n_pages=3 * 2 * 3)
    for t in range(48):                                              # 40 tokens want three pages, which hold 48
        assert step() < STEP_ATOL, t
        assert B.kvc_check_status() == 0
    assert sb.max_len == 48 and sb.lens.tolist() == [[48, 48]] * 3
    K, table = sb.K.clone(), sb.table.clone()
    assert step(stored=False) < STEP_ATOL                            # over what is there
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    assert sb.lens.tolist() == [[48, 48]] * 3 and torch.equal(sb.K, K) and torch.equal(sb.table, table)
    sb.resize(sb.lens * torch.tensor([[0], [1], [1]], dtype=torch.int32, device=DEV))   # one ends; the others are full
    own[0].clear()
    assert step(stored=False) < STEP_ATOL
    with pytest.raises(B.KvcError):
        B.kvc_check_status()


def test_a_pool_one_page_short_refuses_the_step_as_a_whole():
    sb, own, step = small_batch(3, 2, max_len=40, n_pages=3 * 2 + 5)
    for t in range(16):
        assert step() < STEP_ATOL
    assert B.kvc_check_status() == 0
    assert step(stored=False) < STEP_ATOL                            # six rows want a page, five are free
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    assert sb.lens.tolist() == [[16, 16]] * 3 and int(sb.state[1]) == 5
    sb.resize(sb.lens * torch.tensor([[1], [0], [1]], dtype=torch.int32, device=DEV))
    own[1].clear()
    assert step() < STEP_ATOL
    assert B.kvc_check_status() == 0 and sb.lens.tolist() == [[17, 17], [1, 1], [17, 17]]


def test_sequences_rest_end_and_start_again():
    L, Bn, n_pages = 2, 5, 5 * 2 * 2
    sb, own, step = small_batch(Bn, L, max_len=32, n_pages=n_pages)
    rng = np.random.default_rng(8)
    mask = lambda m: torch.tensor(m, dtype=torch.bool, device=DEV)
    for t in range(40):
        if t % 7 == 6:                                               # one ends: its pages go back, and stay there while it rests
            b = int(rng.integers(0, Bn))
            keep = torch.ones(Bn, 1, dtype=torch.int32, device=DEV)
            keep[b] = 0
            sb.resize(sb.lens * keep)
            own[b].clear()
        live = [bool(x) and len(own[b]) < 32 for b, x in enumerate(rng.random(Bn) < (0.0 if t == 20 else 1.0 if t == 5 else 0.6))]
        assert step(live=mask(live)) < STEP_ATOL, (t, live)
        assert sb.lens.tolist() == [[len(x)] * L for x in own]
        assert int(sb.state[1]) == n_pages - sum(-(-len(x) // 16) * L for x in own)
    # full ones rest, the others go on
    while min(map(len, own)) < 32:
        assert step(live=(sb.lens[:, 0] < 32)) < STEP_ATOL
    assert B.kvc_check_status() == 0
    assert step(live=mask([False] * Bn)) < STEP_ATOL
    assert B.kvc_check_status() == 0
    assert step(live=mask([True] + [False] * (Bn - 1)), stored=False) < STEP_ATOL      # refused: the row is full
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    for bad in (torch.ones(Bn, dtype=torch.int32, device=DEV), mask([True] * (Bn + 1)), torch.ones(Bn, dtype=torch.bool)):
        with pytest.raises(ValueError):
            step(live=bad)


def test_a_captured_step_with_resting_sequences_replays():
    L, Bn = 2, 6
    sb, own, step = small_batch(Bn, L, max_len=32, n_pages=Bn * L * 2)
    live = torch.ones(Bn, dtype=torch.bool, device=DEV)
    assert step(live=live) < STEP_ATOL
    q, k, v = torch.randn(Bn, L, 4, 64, device=DEV), torch.randn(Bn, L, 2, 64, device=DEV), torch.randn(Bn, L, 2, 64, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sb.step(q, k, v, live=live)
    rng = np.random.default_rng(9)
    for _ in range(20):
        m = rng.random(Bn) < 0.6
        live.copy_(torch.as_tensor(m))
        for x in (k, v):
            x.normal_()
        graph.replay()
        for b in np.flatnonzero(m):
            own[b].append((np64(k[b]), np64(v[b])))
    assert sb.lens.tolist() == [[len(x)] * L for x in own]
    assert step(live=~live) < STEP_ATOL                              # an eager step on the same rows sees them all
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    some, before = torch.arange(Bn, device=DEV) % 2 == 0, sb.lens.clone()
    torch.cuda.synchronize()
    sb.append(k, v, stream=s, live=some)
    s.synchronize()
    assert torch.equal(sb.lens, before + some[:, None].int())
    assert B.kvc_check_status() == 0
