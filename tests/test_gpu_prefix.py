"""GPU: decode attention over a shared prompt and each sequence's own rows against the fp64 oracle.

Tolerance, per output element, from the arithmetic (u = 2^-24):
* a logit is an fp32 dot product of d exact products, possibly truncated while it is accumulated:
  |dz| <= gamma_d scale sum |q k| with the unit roundoff doubled, plus 3 u |z| for the scale's
  product and the difference to the maximum, plus 2^-20 alpha_c for the fp32 log2 of R;
* exp2 adds 2^-22; the running rescales one rounding each (2^-22 together, at most one in 2^8);
* a weight kept as a bf16 pair carries 2^-8 of 2^-8 = 2^-16;
* sums over n keys in fp32: gamma_n with the roundoff doubled.
With w the exact weights, |do| <= E sum w |v - o| + gamma_n sum w |v| for a relative weight error of E
(first order; E is below 2^-12 here, its square is covered by doubling), and |dlse| <= max |dz| + 2^-20 + gamma_n.
"""
import numpy as np
import pytest
import torch

from long_context_kv_obs_b200 import binding as B
from oracle import serving
from tests.helpers import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def gamma(n, u=2 * U):
    return n * u / (1 - n * u)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Case:
    """Inputs of one call; rows behind every length hold NaN, unused table entries are negative."""

    def __init__(self, B_, L, Hkv, G, d, P, own, page=16, dt=torch.bfloat16, qdt=None, merged=False, layout="head", seed=0,
                 lens_p=None, lens=None, qs=1.0, prompt=True, has_own=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.m = B.model(L, Hkv * G, Hkv, d)
        self.dims = (B_, L, Hkv, G, d)
        self.P, self.page = P, page
        self.q = (qs * torch.randn(B_, L, Hkv * G, d, device=DEV, generator=g)).to(qdt or dt)
        self.prompt, self.has_own = prompt, has_own
        self.lens_p = lens_p if lens_p is not None else [P] + [int(x) for x in rng.integers(max(0, P // 2), P + 1, L - 1)]
        self.lens = np.asarray(lens if lens is not None else rng.integers(0, own + 1, (B_, L)))
        self.max_len = max(1, own)
        self.R = None
        if prompt:
            buf = torch.randn(2, L, Hkv, P + 3, d, device=DEV, generator=g).to(dt)
            self.Kp, self.Vp = buf[0, :, :, :P], buf[1, :, :, :P]
            self.Kp[:, :, 0] *= 3
            for l in range(L):
                self.Kp[l, :, self.lens_p[l]:] = float("nan")
                self.Vp[l, :, self.lens_p[l]:] = float("nan")
            if merged:
                self.R = 1 + 3 * torch.rand(L, Hkv, P, device=DEV, generator=g)
        if has_own:
            if page:
                pg = -(-self.lens // page)
                held = int(pg.sum())
                n_pages = held + 2
                ids = rng.permutation(n_pages)
                width = -(-self.max_len // page) + 1
                table = rng.integers(-5, 0, (B_, L, width))
                k = 0
                for b in range(B_):
                    for l in range(L):
                        table[b, l, :pg[b, l]] = ids[k:k + pg[b, l]]
                        k += pg[b, l]
                self.table = i32(table)
                shape = (n_pages, Hkv, page, d) if layout == "head" else (n_pages, page, Hkv, d)
                K, V = [torch.randn(*shape, device=DEV, generator=g).to(dt) for _ in range(2)]
                self.K, self.V = (K, V) if layout == "head" else (K.transpose(1, 2), V.transpose(1, 2))
                spare = [int(x) for x in ids[held:]]
                self.K[spare], self.V[spare] = float("nan"), float("nan")
                for b in range(B_):
                    for l in range(L):
                        n = int(self.lens[b, l])
                        if n % page:
                            last = int(table[b, l, n // page])
                            self.K[last, :, n % page:], self.V[last, :, n % page:] = float("nan"), float("nan")
            else:
                self.table = None
                self.K, self.V = [torch.randn(B_, L, Hkv, self.max_len + 2, d, device=DEV, generator=g).to(dt)
                                  for _ in range(2)]
                for b in range(B_):
                    for l in range(L):
                        n = int(self.lens[b, l])
                        self.K[b, l, :, n:], self.V[b, l, :, n:] = float("nan"), float("nan")
        self.o = torch.full((B_, L, Hkv * G, d), float("nan"), device=DEV)
        self.lse = torch.full((B_, L, Hkv * G), float("nan"), device=DEV)

    def kw(self):
        kw = dict(q=self.q, o=self.o, lse=self.lse)
        if self.prompt:
            kw.update(K_prefix=self.Kp, V_prefix=self.Vp, lens_prefix=i32(self.lens_p), max_len_prefix=self.P, R=self.R)
        if self.has_own:
            kw.update(K=self.K, V=self.V, table=self.table, lens=i32(self.lens), max_len=self.max_len)
        return kw

    def run(self, **more):
        return B.kvc_prefix_decode_attn(self.m, **{**self.kw(), **more})

    def own_rows(self, b, l, g):
        if not self.has_own:
            return np.zeros((0, self.dims[4])), np.zeros((0, self.dims[4]))
        n = int(self.lens[b, l])
        if self.table is None:
            return np64(self.K[b, l, g, :n]), np64(self.V[b, l, g, :n])
        t = self.table[b, l, :-(-n // self.page)].long()
        return [np64(x[t][:, g].reshape(-1, self.dims[4])[:n]) for x in (self.K, self.V)]

    def check(self, alpha_c=1.0, scale=None, pair=True):
        B_, L, Hkv, G, d = self.dims
        o, lse, q = np64(self.o), np64(self.lse), np64(self.q)
        assert np.isfinite(o).all()
        sc = d ** -0.5 if scale is None else scale
        for l in range(L):
            P = self.lens_p[l] if self.prompt else 0
            for g in range(Hkv):
                kp = np64(self.Kp[l, g, :P]) if P else np.zeros((0, d))
                vp = np64(self.Vp[l, g, :P]) if P else np.zeros((0, d))
                R = np64(self.R[l, g, :P]) if self.R is not None else None
                for b in range(B_):
                    ko, vo = self.own_rows(b, l, g)
                    qq = q[b, l, g * G:(g + 1) * G]
                    ro, rl, w = serving.prefix_attention(qq, kp, vp, ko, vo, R, alpha_c, sc)
                    n = w.shape[1]
                    go, gl = o[b, l, g * G:(g + 1) * G], lse[b, l, g * G:(g + 1) * G]
                    if n == 0:
                        assert (go == 0).all() and (gl == -np.inf).all()
                        continue
                    kk, vv = np.concatenate([kp, ko]), np.concatenate([vp, vo])
                    dz = (gamma(d) * sc * (np.abs(qq) @ np.abs(kk).T) + 3 * U * sc * np.abs(qq @ kk.T)).max(axis=1)
                    dz = dz + 3 * U * 40 + (2.0 ** -20 * abs(alpha_c) if R is not None else 0)
                    E = 2 * dz + 2.0 ** -21 + (2.0 ** -16 if pair else 0)
                    spread = np.stack([(w[h][:, None] * np.abs(vv - ro[h])).sum(0) for h in range(G)])
                    lim = 2 * E[:, None] * spread + gamma(n + 64) * (w @ np.abs(vv)) + 1e-30
                    err = np.abs(go - ro)
                    assert (err <= lim).all(), (b, l, g, float((err / lim).max()))
                    assert (np.abs(gl - rl) <= dz + 2.0 ** -20 + gamma(n + 64) + 2 * U * np.abs(rl)).all(), (b, l, g)


BF, FP = torch.bfloat16, torch.float32
SHAPES = [
    # B, L, Hkv, G, d, P, own, page
    (1, 1, 1, 1, 128, 1, 1, 16),
    (2, 2, 2, 4, 128, 129, 33, 16),
    (3, 3, 2, 7, 128, 500, 70, 32),
    (8, 2, 4, 7, 128, 777, 130, 64),
    (16, 1, 8, 4, 128, 1100, 65, 128),
    (33, 2, 2, 4, 128, 300, 64, 256),       # 132 rows: one query row block and four rows
    (64, 1, 1, 4, 128, 1000, 200, 16),      # 256 rows
    (40, 1, 2, 8, 64, 385, 20, 16),         # 320 rows: two row blocks
    (5, 3, 3, 5, 64, 640, 100, 32),
    (150, 1, 1, 2, 128, 257, 17, 16),
]


@pytest.mark.parametrize("merged", [False, True])
@pytest.mark.parametrize("B_,L,Hkv,G,d,P,own,page", SHAPES)
def test_bf16_matches_the_oracle(B_, L, Hkv, G, d, P, own, page, merged):
    c = Case(B_, L, Hkv, G, d, P, own, page, merged=merged, seed=P + own)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()


@pytest.mark.parametrize("dt,qdt", [(FP, FP), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("B_,L,Hkv,G,d,P,own,page", [SHAPES[i] for i in (0, 1, 2, 4, 7, 8)])
def test_fp32_caches_or_queries_match_the_oracle(B_, L, Hkv, G, d, P, own, page, dt, qdt):
    c = Case(B_, L, Hkv, G, d, P, own, page, dt=dt, qdt=qdt, merged=True, seed=P + own + 1)
    c.run()
    assert B.kvc_check_status() == 0
    c.check(pair=False)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("B_,L,Hkv,G,d,P,own,page", [SHAPES[i] for i in (1, 3, 8)])
def test_contiguous_own_rows(B_, L, Hkv, G, d, P, own, page, dt):
    c = Case(B_, L, Hkv, G, d, P, own, 0, dt=dt, seed=3)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()


@pytest.mark.parametrize("dt", [BF, FP])
def test_tokens_first_in_a_page_and_only_one_side(dt):
    c = Case(4, 2, 3, 4, 128, 200, 90, 32, dt=dt, layout="token", seed=4)
    c.run()
    c.check()
    c = Case(4, 2, 3, 4, 128, 200, 90, 32, dt=dt, seed=5, prompt=False)
    c.run()
    c.check()
    c = Case(4, 2, 3, 4, 128, 200, 90, 32, dt=dt, seed=6, has_own=False)
    c.run()
    c.check()
    assert B.kvc_check_status() == 0


@pytest.mark.parametrize("dt", [BF, FP])
def test_empty_rows_and_edges(dt):
    """No prompt in a layer, no own rows in a sequence, neither, one key, lengths at tile borders."""
    lens = [[0, 0, 0, 0, 0], [1, 1, 1, 1, 1], [64, 63, 65, 128, 0], [16, 15, 17, 0, 200]]
    c = Case(4, 5, 2, 4, 128, 256, 200, 16, dt=dt, seed=7, lens_p=[0, 1, 128, 127, 256], lens=lens, merged=True)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()
    c = Case(4, 5, 2, 4, 128, 256, 200, 16, dt=dt, seed=8, lens_p=[0] * 5, lens=lens)
    c.run()
    c.check()
    c = Case(2, 2, 1, 4, 64, 100, 50, 16, dt=dt, seed=9, lens_p=[0, 0], lens=[[0, 0], [0, 0]])
    c.run()
    c.check()


@pytest.mark.parametrize("dt", [BF, FP])
def test_large_logits_rescale_and_scale_argument(dt):
    """Logits in the hundreds: the running maximum moves often; a scale and an alpha_c of one's own."""
    c = Case(9, 1, 2, 4, 128, 900, 100, 16, dt=dt, seed=10, qs=12.0, merged=True)
    c.run()
    c.check()
    c.run(scale=0.25, alpha_c=-0.5)
    c.check(scale=0.25, alpha_c=-0.5)
    # keys that grow along the sequence: every tile moves the maximum
    c.Kp.mul_(torch.linspace(0.01, 2, 900, device=DEV)[:, None].to(dt))
    c.run()
    c.check()


def test_lengths_and_pages_out_of_bounds_are_clamped_and_recorded():
    c = Case(3, 2, 2, 4, 128, 200, 60, 16, seed=11, lens_p=[200, 200], lens=np.full((3, 2), 60))
    kw = c.kw()
    c.check_ = None
    B.kvc_prefix_decode_attn(c.m, **{**kw, "lens_prefix": i32([4000, 200])})
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    c.check()
    B.kvc_prefix_decode_attn(c.m, **{**kw, "lens": i32([[60, 60], [60, 9000], [60, 60]])})
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    c.check()
    # a page id outside the pool reads as rows of zeros
    t = c.table.clone()
    t[1, 0, 1] = c.K.shape[0] + 3
    t[2, 1, 0] = -4
    B.kvc_prefix_decode_attn(c.m, **{**kw, "table": t})
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    K = torch.cat([c.K, torch.zeros_like(c.K[:1])])
    V = torch.cat([c.V, torch.zeros_like(c.V[:1])])
    t[1, 0, 1] = t[2, 1, 0] = c.K.shape[0]
    c.K, c.V, c.table = K, V, t
    c.check()


def test_equal_calls_are_bit_identical_and_graphs_replay():
    c = Case(20, 3, 2, 4, 128, 2000, 150, 16, seed=12, merged=True)
    ws = c.run()
    first = (c.o.clone(), c.lse.clone())
    for _ in range(3):
        c.o.fill_(float("nan"))
        ws.fill_(0xff)
        c.run(workspace=ws)
        assert torch.equal(c.o, first[0]) and torch.equal(c.lse, first[1])
    # two graphs with workspaces of their own, replayed on two streams at once
    other = Case(20, 3, 2, 4, 128, 2000, 150, 16, seed=13)
    graphs = []
    for x, w in ((c, ws), (other, torch.empty_like(ws))):
        x.run(workspace=w)
        kw = x.kw()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.kvc_prefix_decode_attn(x.m, workspace=w, **kw)
        graphs.append((g, kw, w))
    want = other.o.clone()
    c.o.zero_()
    other.o.zero_()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, first[0]) and torch.equal(other.o, want)
    assert B.kvc_check_status() == 0


def test_lse_ring_slot_and_another_stream():
    c = Case(6, 2, 2, 4, 128, 300, 40, 16, seed=14)
    ring = torch.zeros(6, 2, 8, 5, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(lse=ring[..., 3], stream=s)
    s.synchronize()
    c.lse = ring[..., 3].contiguous()
    c.check()
    ring[..., 3] = 0
    assert int(torch.count_nonzero(ring)) == 0


def test_refusals_launch_nothing():
    c = Case(2, 1, 2, 4, 128, 64, 40, 16, seed=15)
    kw = c.kw()
    ws = c.run()
    before = B.kvc_launch_count()
    bad = [dict(workspace=ws[:64]), dict(K=None, V=None, table=None, K_prefix=None, V_prefix=None, R=None), dict(scale=-1.0),
           dict(scale=float("nan")), dict(lens=i32([[1]])), dict(max_len_prefix=65), dict(max_len=400), dict(o=c.o[:1]),
           dict(q=c.q.cpu()), dict(table=c.table[:1]), dict(K=c.K.float()), dict(V_prefix=c.Vp.float()),
           dict(K_prefix=c.Kp[:, :1]), dict(table=c.table.long())]
    for change in bad:
        with pytest.raises((ValueError, TypeError, B.KvcError)):
            B.kvc_prefix_decode_attn(c.m, **{**kw, **change})
    with pytest.raises(B.KvcError):
        B.kvc_prefix_decode_attn(B.model(1, 18, 2, 128), q=torch.zeros(2, 1, 18, 128, device=DEV, dtype=BF),
                                 o=torch.zeros(2, 1, 18, 128, device=DEV), K_prefix=c.Kp, V_prefix=c.Vp,
                                 lens_prefix=i32([64]), max_len_prefix=64)
    assert B.kvc_launch_count() == before


@pytest.mark.parametrize("merged", [False, True])
@pytest.mark.parametrize("B_,G,d", [(13, 5, 128), (32, 4, 128), (16, 4, 64), (43, 3, 64), (32, 8, 128), (37, 7, 128)])
def test_row_counts_at_the_tiles_borders(B_, G, d, merged):
    """64, 65, 128, 129, 256 and 259 query rows a KV head."""
    c = Case(B_, 2, 2, G, d, 400, 30, 16, merged=merged, seed=B_)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()


@pytest.mark.parametrize("B_", [3, 40])
def test_prompts_that_end_at_and_beside_half_tiles(B_):
    ends = [0, 1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257]
    c = Case(B_, len(ends), 1, 4, 128, 257, 20, 16, seed=40, lens_p=ends, merged=B_ == 3)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()


def test_more_layers_than_the_tensor_core_kernel_takes():
    c = Case(2, 130, 1, 2, 64, 40, 20, 16, seed=41, merged=True)
    c.run()
    assert B.kvc_check_status() == 0
    c.check()


@pytest.mark.parametrize("dt", [BF, FP])
def test_calls_on_two_streams_at_once_and_back_to_back(dt):
    """Every call's kernels overlap at their ends: neither another stream's call nor the next on the same
    stream, on the same workspace, may see half a result."""
    cases = [Case(9, 2, 2, 4, 128, 900, 300, 16, seed=s, dt=dt, merged=s % 2 == 1) for s in (42, 43, 44)]
    want = []
    for c in cases:
        c.run()
        want.append(c.o.clone())
    assert B.kvc_check_status() == 0
    kws = [c.kw() for c in cases]
    ws = [B.kvc_prefix_decode_attn(c.m, **kw) for c, kw in zip(cases[:2], kws[:2])]
    torch.cuda.synchronize()
    outs = [[torch.full_like(c.o, float("nan")) for _ in range(8)] for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(8):
        for k, s in enumerate(streams):
            # the second stream's calls alternate between two inputs on one workspace
            j = k if k == 0 or i % 2 == 0 else 2
            B.kvc_prefix_decode_attn(cases[j].m, workspace=ws[k], stream=s, **{**kws[j], "o": outs[j][i]})
    torch.cuda.synchronize()
    assert B.kvc_check_status() == 0
    for i in range(8):
        assert torch.equal(outs[0][i], want[0])
        assert torch.equal(outs[1 if i % 2 == 0 else 2][i], want[1 if i % 2 == 0 else 2])


@pytest.mark.parametrize("G,merged", [(3, False), (1, True), (8, False)])
def test_few_rows_on_a_long_prompt_wait_for_late_loads(G, merged):
    """Bound by HBM, loads come microseconds late and out of order: equal calls give equal bits, right ones."""
    c = Case(3, 4, 6, G, 128, 20011, 28, 128, merged=merged, seed=50 + G)
    ws = c.run()
    assert B.kvc_check_status() == 0
    first = (c.o.clone(), c.lse.clone())
    for _ in range(30):
        c.run(workspace=ws)
    assert B.kvc_check_status() == 0
    assert torch.equal(c.o, first[0]) and torch.equal(c.lse, first[1])
    c.check()


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_a_query_or_a_key_is_seen_and_stays_in_its_rows(dt, d):
    """By the formula: a NaN query makes its row NaN; a NaN key the rows that face it; no other row changes."""
    nan = float("nan")
    kw = dict(dt=dt, lens=[[40, 3], [0, 70], [5, 5]], seed=60)
    ref = Case(3, 2, 2, 4, d, 300, 70, 16, **kw)
    ref.run()
    want = (ref.o.clone(), ref.lse.clone())

    def check(c, bad):
        c.run()
        assert B.kvc_check_status() == 0
        assert bool(torch.isnan(c.o[bad]).all()) and bool(torch.isnan(c.lse[bad]).all())
        assert torch.equal(c.o[~bad], want[0][~bad]) and torch.equal(c.lse[~bad], want[1][~bad])

    bad = lambda: torch.zeros(3, 2, 8, dtype=torch.bool, device=DEV)
    c, b = Case(3, 2, 2, 4, d, 300, 70, 16, **kw), bad()
    c.q[1, 0, 5, 7] = nan                                            # (over the prompt alone)
    c.q[2, 1, 0, :] = nan
    b[1, 0, 5] = b[2, 1, 0] = True
    check(c, b)
    c, b = Case(3, 2, 2, 4, d, 300, 70, 16, **kw), bad()
    c.Kp[0, 1, 17, 3] = nan
    b[:, 0, 4:] = True
    check(c, b)
    c, b = Case(3, 2, 2, 4, d, 300, 70, 16, **kw), bad()
    c.K[int(c.table[0, 0, 1]), 0, 2, 3] = nan                        # own token 18 of sequence 0
    b[0, 0, :4] = True
    check(c, b)
    c, b = Case(3, 2, 2, 4, d, 300, 70, 16, prompt=False, **kw), bad()
    ref = Case(3, 2, 2, 4, d, 300, 70, 16, prompt=False, **kw)
    ref.run()
    want = (ref.o.clone(), ref.lse.clone())
    c.q[0, 1, 2, 0] = nan
    b[0, 1, 2] = True
    check(c, b)


def test_a_prompt_that_takes_seconds():
    """Waits inside a kernel have a limit of two seconds each.  The own rows' kernel is under way while the prompt's ends: what it
    waits for then is not its own, and the limit must not count (4 M keys times 2^20 query rows, some 3 s)."""
    Bn, G, d, P, own = 2 ** 17, 8, 128, 4_000_000, 3
    m = B.model(1, G, 1, d)
    g = torch.Generator(device=DEV).manual_seed(70)
    draw = lambda *s: torch.randn(*s, device=DEV, dtype=BF, generator=g)
    q, Kp, Vp, K, V = draw(Bn, 1, G, d), draw(1, 1, P, d), draw(1, 1, P, d), draw(Bn, 1, 1, own, d), draw(Bn, 1, 1, own, d)
    Kp[0, 0, -5:] *= 3                                               # keys at the end that weigh
    K *= 3
    o, lse = torch.empty(Bn, 1, G, d, device=DEV), torch.empty(Bn, 1, G, device=DEV)
    B.kvc_prefix_decode_attn(m, q=q, o=o, lse=lse, K_prefix=Kp, V_prefix=Vp, lens_prefix=i32([P]), max_len_prefix=P, K=K, V=V,
                             lens=i32(np.full((Bn, 1), own)), max_len=own)
    assert B.kvc_check_status() == 0
    for b in (0, 1, 777, 40000, 99999, Bn - 1):
        z = q[b, 0].double() @ torch.cat([Kp[0, 0], K[b, 0, 0]]).double().t() / d ** 0.5
        w, want = torch.softmax(z, -1), torch.logsumexp(z, -1)
        # logits (below 80) to 2^-17 of them, weights to 2^-16, sums of tiles in fp32: 31250 tiles, 2^-24 of the sum each
        assert float((lse[b, 0] - want).abs().max()) < 80 * 2 ** -17 + 31250 * 2 ** -24 + 2 ** -16
        lim = (2 * (80 * 2 ** -17 + 2 ** -16) + 31250 * 2 ** -23) * (w @ torch.cat([Vp[0, 0], V[b, 0, 0]]).double().abs())
        assert bool(((o[b, 0] - w @ torch.cat([Vp[0, 0], V[b, 0, 0]]).double()).abs() <= lim + 1e-6).all())
