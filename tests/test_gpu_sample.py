"""GPU: token sampling against the fp64 oracle.  Tokens and counts are equal: a border lies within the
kernel's error (2^-32 of a weight for each of them) of a random one with a chance of 10^-6 a row.  logprob is
fp32 of an fp64 value: half a step of fp32 (2^-24 of it) and 10^-9 for the masses (2^-30 at most)."""
import numpy as np
import pytest
import torch

from long_context_kv_obs_b200 import binding as B
from oracle import serving
from tests.helpers import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
INF = float("inf")


def call(logits, u, stream=None, **par):
    n = logits.shape[0]
    dev = lambda x, dt: None if x is None else torch.as_tensor(np.asarray(x), device=DEV).to(dt).expand(n).contiguous()
    token = torch.full((n,), -99, dtype=torch.int32, device=DEV)
    logprob, kept = torch.full((n,), float("nan"), device=DEV), torch.full((n,), -99, dtype=torch.int32, device=DEV)
    kw = {k: dev(v, torch.int32 if k == "top_k" else FP) for k, v in par.items()}
    B.kvc_sample(logits=logits, u=dev(u, FP), token=token, logprob=logprob, kept=kept, stream=stream, **kw)
    return token, logprob, kept, kw


def check(logits, u, **par):
    token, logprob, kept, kw = call(logits, u, **par)
    n = logits.shape[0]
    z = np64(logits)
    uu = np.broadcast_to(np.asarray(u, np.float32), (n,))
    for i in range(n):
        args = {k: (int(v[i]) if k == "top_k" else float(v[i])) for k, v in kw.items() if v is not None}
        et, el, ek = serving.sample(z[i], float(uu[i]), **args)
        assert int(kept[i]) == ek, (i, args, int(kept[i]), ek)
        assert int(token[i]) == et, (i, args, int(token[i]), et)
        if np.isinf(el):
            assert float(logprob[i]) == el
        else:
            assert abs(float(logprob[i]) - el) <= 2.0 ** -24 * abs(el) + 1e-9, (i, args)
    assert B.kvc_check_status() == 0


def rows(n, V, dt, seed, sigma=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = torch.empty(n, 1, device=DEV).uniform_(0.3, 5, generator=g) if sigma is None else sigma
    return (torch.randn(n, V, device=DEV, generator=g) * s).to(dt)


SIZES = [(1, 1), (3, 7), (5, 100), (4, 1000), (7, 4099), (3, 19456), (4, 19457), (3, 32003), (2, 65537), (2, 128256),
         (2, 152064), (1, 262144)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("n,V", SIZES)
def test_each_filter_and_all_of_them(n, V, dt):
    z = rows(n, V, dt, V)
    r = np.random.default_rng(V)
    u = r.random(n).astype(np.float32)
    check(z, u)
    check(z, u, temperature=r.uniform(0.2, 2, n))
    check(z, u, temperature=0.7, top_k=r.integers(1, max(2, V), n))
    check(z, u, temperature=0.7, top_k=50)
    check(z, u, temperature=1.3, top_p=r.uniform(0.05, 0.999, n))
    check(z, u, temperature=0.6, min_p=r.uniform(0.001, 0.5, n))
    check(z, u, temperature=r.uniform(0.2, 2, n), top_k=r.integers(0, V + 5, n), top_p=r.uniform(0.3, 1.05, n),
          min_p=r.uniform(-0.05, 0.1, n))


@pytest.mark.parametrize("dt", [BF, FP])
def test_ties(dt):
    """Few different values: the cuts fall among equal logits and take the lowest indices."""
    r = np.random.default_rng(3)
    for V in (64, 5000, 40000):
        z = torch.as_tensor(r.integers(-2, 3, (6, V)) * 0.5, device=DEV).to(dt)
        z[1] = 1.25                                                  # uniform rows
        z[2] = -3e38
        u = [0.0, 0.5, 0.25, 1 - 2 ** -24, 0.1, 0.9]
        check(z, u, top_k=[1, 7, V // 3, 2, V - 1, V // 2])
        check(z, u, temperature=0.8, top_p=[0.1, 0.5, 0.25, 0.9, 0.3, 0.75])
        check(z, u, temperature=0.8, top_k=V // 2, top_p=[0.1, 0.5, 0.25, 0.99999994, 0.3, 0.75], min_p=0.01)
        check(z, u, min_p=[1.0, 1.0, 2.0, 0.5, 0.3, 1e-30])
        z0 = torch.zeros(2, V, dtype=dt, device=DEV)
        z0[:, ::2] = -0.0                                            # -0 and +0 are equal logits
        check(z0, [0.3, 0.6], top_k=V // 2, top_p=0.7)


@pytest.mark.parametrize("dt", [BF, FP])
def test_masks_infinities_and_nan(dt):
    V = 3001
    low = torch.finfo(dt).min
    z = rows(10, V, dt, 4)
    drop = torch.rand(10, V, device=DEV) < 0.7
    z[:5] = z[:5].masked_fill(drop[:5], -INF)
    z[5] = -INF                                                      # nothing is left
    z[6] = torch.where(drop[6], torch.full_like(z[6], low), z[6])
    z[7, 17], z[7, 2900] = INF, INF
    z[8, ::3] = float("nan")
    z[9] = low
    z[3] = -INF
    z[3, V - 1] = -40.0                                              # one token is left
    u = np.linspace(0, 0.999, 10).astype(np.float32)
    for kw in (dict(), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.02), dict(top_k=100, top_p=0.5, min_p=0.001),
               dict(temperature=0.0), dict(temperature=-1.0, top_k=3)):
        check(z, u, **kw)
    z[:] = float("nan")
    check(z, u, top_p=0.5)


def test_border_parameters():
    z = rows(8, 5003, FP, 5)
    nan = float("nan")
    check(z, [0.0, -3.0, 1.0, 7.0, nan, 0.5, 1 - 2 ** -24, 1e-30], temperature=0.9, top_p=0.8)
    check(z, 0.4, temperature=[0.0, -1.0, nan, 1e-40, 1e-6, 1e6, INF, 30.0], top_p=0.5, top_k=1000)
    check(z, 0.7, temperature=[0.0, -1.0, nan, 1e-40, 1e-6, 1e6, INF, 30.0])
    check(z, 0.7, top_p=[0.0, -1.0, nan, 1.0, 2.0, 1e-30, 0.99999994, 0.5])
    check(z, 0.7, min_p=[0.0, -1.0, nan, 1.0, 2.0, 1e-30, 0.99999994, 0.5])
    check(z, 0.7, top_k=[0, -5, 1, 2, 5002, 5003, 5004, 2 ** 31 - 1])
    zi = z.clone()
    zi[:, 7] = INF
    check(zi, 0.7, temperature=[1.0, 0.5, 2.0, INF, 1e-40, 30.0, 1.0, 1.0], top_p=0.9, min_p=0.1)


@pytest.mark.parametrize("dt", [BF, FP])
def test_wide_scales_near_values_and_drawn_cases(dt):
    """Logits in the thousands, a narrow band around zero, and random parameters on many rows."""
    r = np.random.default_rng(6)
    check(rows(4, 20011, dt, 7, 1000.0), 0.3, top_p=0.9, temperature=[1, 100, 1000, 5000])
    check(rows(4, 20011, dt, 8, 1e-3), r.random(4), top_p=0.6, temperature=[1, 0.001, 0.01, 0.1])
    check(rows(4, 20011, dt, 9, 1e-20), r.random(4), top_k=9999, top_p=0.6)
    n = 96
    check(rows(n, 8011, dt, 10), r.random(n), temperature=r.uniform(0, 2, n), top_k=np.exp(r.uniform(0, 9, n)).astype(int),
          top_p=r.uniform(0.2, 1.1, n), min_p=r.uniform(-0.1, 0.1, n))


@pytest.mark.parametrize("dt", [BF, FP])
def test_strides_and_alignment(dt):
    r = np.random.default_rng(8)
    buf = rows(6, 5100, dt, 11)
    for off, width in ((0, 5000), (1, 5000), (8, 5008), (3, 4097), (17, 1)):
        check(buf[:, off:off + width], r.random(6), temperature=0.8, top_p=0.9)
        check(buf[::2, off:off + width], r.random(3), temperature=0.8, top_k=20)


def test_equal_calls_give_equal_tokens_on_streams_and_in_graphs():
    z = rows(32, 50021, BF, 12)
    u = np.random.default_rng(9).random(32)
    par = dict(temperature=0.8, top_k=3000, top_p=0.9, min_p=0.001)
    first = call(z, u, **par)[:3]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        again = call(z, u, stream=s if k % 2 else None, **par)[:3]
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    ut, token = torch.as_tensor(u, device=DEV).float(), torch.zeros(32, dtype=torch.int32, device=DEV)
    p = torch.full((32,), 0.9, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.kvc_sample(logits=z, u=ut, token=token, top_p=p)
    g.replay()
    torch.cuda.synchronize()
    a = token.clone()
    ut.copy_(torch.flip(ut, (0,)))
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(a, token)
    for i in range(32):
        assert int(token[i]) == serving.sample(np64(z[i]), float(ut[i]), top_p=float(p[i]))[0]


def test_sample_frequencies_follow_the_distribution():
    """An even grid of u over one row: each token is drawn its share of times, off by one at most."""
    V, n = 37, 4096
    z = rows(1, V, FP, 13).expand(n, V)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    token = call(z.contiguous(), u, temperature=1.0)[0].cpu().numpy()
    p = np.exp(np64(z[0]) - np64(z[0]).max())
    p /= p.sum()
    assert (np.abs(np.bincount(token, minlength=V) - n * p) <= 1 + 1e-6).all()
    assert (np.diff(token) >= 0).all()


def test_refusals_launch_nothing():
    z = rows(3, 100, FP, 14)
    u, token = torch.rand(3, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    before = B.kvc_launch_count()
    bad = [dict(logits=z.half()), dict(logits=z.cpu()), dict(logits=z.t()), dict(u=u[:2]), dict(u=u.double()), dict(token=token.long()),
           dict(top_k=u), dict(top_p=token), dict(logits=torch.zeros(1, 262145, device=DEV), u=u[:1], token=token[:1])]
    for change in bad:
        with pytest.raises((ValueError, TypeError, B.KvcError)):
            B.kvc_sample(**{**dict(logits=z, u=u, token=token), **change})
    assert B.kvc_launch_count() == before


def test_bf16_values_of_one_sign_across_zero_and_at_its_borders():
    """bf16 cuts are searched value by value: spans of one sign, spans that cross zero, more values than bins,
    values that differ near zero alone, cuts among ties that several slices of the row share."""
    r = np.random.default_rng(20)
    V = 90001
    g = torch.Generator(device=DEV).manual_seed(21)
    e = torch.rand(12, V, device=DEV, generator=g)
    z = torch.randn(12, V, device=DEV, generator=g)
    z[0] = -torch.exp2(-40 * e[0])                                    # negative, 40 octaves
    z[1] = torch.exp2(-40 * e[1])                                     # positive
    z[2] = torch.where(e[2] < 0.5, -1.0, 1.0) * torch.exp2(-60 * z[2].abs())
    z[3] = z[3] * 1e-6                                                # about zero alone
    z[4] = 9 + z[4] * 0.01
    z[5] = -9 + z[5] * 0.01
    z[6] = torch.where(e[6] < 0.999, torch.full_like(z[6], 2.5), z[6])  # one value holds nearly all
    z[7] = torch.where(e[7] < 0.999, torch.full_like(z[7], -2.5), z[7] * 3)
    z[8] = z[8] * 1e30
    z[9] = -z[9].abs() * 1e-30
    z[10] = z[10].round()                                             # a few values, one of them zero
    z[11, 0] = 30.0                                                   # one token holds nearly all
    z = z.to(BF)
    u = r.random(12).astype(np.float32)
    for T in (0.05, 0.7, 1.0, 20.0):
        for p in (0.3, 0.95, 0.9999):
            check(z, u, temperature=T, top_p=p)
    for k in (600, 5000, V // 2, V // 2 + 1, V - 1):
        check(z, u, temperature=0.8, top_k=k)
        check(z, u, temperature=0.8, top_k=k, top_p=0.8, min_p=1e-4)
    check(z, u, temperature=0.8, min_p=r.uniform(1e-6, 0.9, 12), top_p=r.uniform(0.01, 0.9999, 12))


def test_bf16_border_parameters():
    z = rows(8, 5003, BF, 22)
    nan = float("nan")
    check(z, [0.0, -3.0, 1.0, 7.0, nan, 0.5, 1 - 2 ** -24, 1e-30], temperature=0.9, top_p=0.8)
    check(z, 0.4, temperature=[0.0, -1.0, nan, 1e-40, 1e-6, 1e6, INF, 30.0], top_p=0.5, top_k=1000)
    check(z, 0.7, top_p=[0.0, -1.0, nan, 1.0, 2.0, 1e-30, 0.99999994, 0.5])
    check(z, 0.7, top_p=[0.0, -1.0, nan, 1.0, 2.0, 1e-30, 0.99999994, 0.5], top_k=3000, min_p=0.01)
    check(z, 0.7, top_k=[0, -5, 1, 2, 5002, 5003, 5004, 2 ** 31 - 1])
    zi = z.clone()
    zi[:, 7] = INF
    check(zi, 0.7, temperature=[1.0, 0.5, 2.0, INF, 1e-40, 30.0, 1.0, 1.0], top_p=0.9, min_p=0.1)


def test_calls_on_two_streams_and_captured_twice():
    z = [rows(20, 30011, BF, 30), rows(20, 30011, FP, 31)]
    u = torch.rand(20, device=DEV)
    par = dict(temperature=torch.full((20,), 0.8, device=DEV), top_p=torch.full((20,), 0.9, device=DEV))
    want = []
    for x in z:
        tok = torch.empty(20, dtype=torch.int32, device=DEV)
        B.kvc_sample(logits=x, u=u, token=tok, **par)
        want.append(tok)
    toks = [torch.full((20,), -9, dtype=torch.int32, device=DEV) for _ in z]
    graphs = []
    torch.cuda.synchronize()
    for x, tok in zip(z, toks):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.kvc_sample(logits=x, u=u, token=tok, **par)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(toks, want))
    for s, x, tok in zip(streams, z, toks):
        tok.fill_(-9)
        torch.cuda.synchronize()
        B.kvc_sample(logits=x, u=u, token=tok, stream=s, **par)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(toks, want))
    assert B.kvc_check_status() == 0


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("V", [125515, 131072, 152064, 262144])
def test_large_flat_rows(V, dt):
    """Nearly all tokens of a large vocabulary within one bin of the search: its sums over the row pass 2^32."""
    r = np.random.default_rng(V)
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.zeros(9, V, device=DEV)
    z[1] = 1.5
    z[2, 12345] = 0.01                                               # in the search's first bin, beside the others' value
    z[3] = INF
    z[4] = torch.where(torch.rand(V, device=DEV, generator=g) < 0.5, 0.0, -0.0005)
    z[5] = torch.randn(V, device=DEV, generator=g) * 1e-4
    z[6] = torch.randn(V, device=DEV, generator=g) * 1e-2
    z[7] = torch.where(torch.rand(V, device=DEV, generator=g) < 0.9, 0.0, -0.5)
    z[8] = torch.randn(V, device=DEV, generator=g)
    z = z.to(dt)
    for p in (0.05, 0.5, 0.95, 0.9999):
        check(z, r.random(9), top_p=p)
    check(z, r.random(9), top_p=r.uniform(0.1, 0.999, 9), temperature=[1, 0.3, 1, 1, 0.7, 1e-3, 1, 50, 100], top_k=V - 1000)


@pytest.mark.parametrize("dt", [BF, FP])
def test_large_flat_rows_in_a_large_batch(dt):
    """The same where rows are cut into fewer, longer slices."""
    V, n = 262144, 76
    g = torch.Generator(device=DEV).manual_seed(7)
    z = torch.zeros(4, V, device=DEV)
    z[1] = torch.randn(V, device=DEV, generator=g) * 1e-4
    z[2] = torch.where(torch.rand(V, device=DEV, generator=g) < 0.8, 2.0, 1.9995)
    z[3] = torch.randn(V, device=DEV, generator=g) * 0.1
    z = z.to(dt)
    u = np.array([0.2, 0.55, 0.8, 0.999], np.float32)
    token, logprob, kept, kw = call(z.repeat(n // 4, 1), np.tile(u, n // 4), top_p=0.9)
    zn, p = np64(z), float(kw["top_p"][0])
    for i in range(4):
        et, el, ek = serving.sample(zn[i], float(u[i]), top_p=p)
        assert kept[i::4].tolist() == [ek] * (n // 4) and token[i::4].tolist() == [et] * (n // 4)
        assert np.abs(np64(logprob[i::4]) - el).max() <= 2.0 ** -24 * abs(el) + 1e-9
    assert B.kvc_check_status() == 0


@pytest.mark.parametrize("dt", [BF, FP])
def test_temperatures_at_the_lower_end(dt):
    """Temperatures down to the least of fp32, over logits whose differences are of their size."""
    r = np.random.default_rng(40)
    p = [0.1, 0.3, 0.5, 0.9, 0.99, 0.9999]
    for V in (5003, 40000):
        base = r.standard_normal((6, V))
        for T in (1e-45, 1e-40, 1e-38, 1e-37, 1e-36, 1e-35, 1e-30):
            for s in (0.3, 1.0, 30.0, 1000.0):
                z = torch.as_tensor((base * (T * s)).astype(np.float32), device=DEV).to(dt)
                check(z, r.random(6), top_p=p, temperature=T)


@pytest.mark.parametrize("dt", [BF, FP])
def test_logits_further_apart_than_the_range_of_fp32(dt):
    """Rows from -3.4e38 to 3.4e38 at temperatures that make that a few octaves, or none."""
    r = np.random.default_rng(50)
    p = [0.1, 0.3, 0.5, 0.9, 0.99, 0.9999]
    for V in (1001, 40000):
        base = r.uniform(-1, 1, (6, V))
        base[3] = np.where(r.random(V) < 0.5, -1, 1)
        base[4] = np.where(r.random(V) < 0.5, -1, 1e-38)
        for s in (1e30, 1e37, 2e38, 3.38e38):
            z = torch.as_tensor((base * s).astype(np.float32), device=DEV).to(dt)
            for T in (1.0, 1e35, 1e36, 1e37, 1e38, 3e38, INF):
                u = r.random(6)
                check(z, u, temperature=T, top_p=p)
                check(z, u, temperature=T, top_p=p, top_k=[700, 1, V // 2, V // 3, V - 1, 900], min_p=0.05)
        check(z, u, temperature=1e38)
        check(z, u, temperature=1e38, min_p=0.3)
