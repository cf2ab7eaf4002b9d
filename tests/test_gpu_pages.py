"""GPU: page tables, slot maps and the append into pages against their definitions (integers and
bit-exact rows)."""
import numpy as np
import pytest
import torch

from long_context_kv_obs_b200 import binding as B
from oracle import serving

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(rng, rows, page, most, new_of, spare=5):
    """Tables that hold rows of random length, with the other pages in a ring that wraps."""
    lens = [int(x) for x in rng.integers(0, most + 1, rows)]
    new = [int(new_of(rng, a)) for a in lens]
    pg = lambda n: -(-n // page)
    held = sum(map(pg, lens))
    need = sum(max(0, pg(z) - pg(a)) for a, z in zip(lens, new))
    n_pages = held + need + spare
    ids = rng.permutation(n_pages)
    max_pages = max(1, max(pg(max(a, z)) for a, z in zip(lens, new)))
    table = rng.integers(-9, -1, (rows, max_pages))
    k = 0
    for r in range(rows):
        table[r, :pg(lens[r])] = ids[k:k + pg(lens[r])]
        k += pg(lens[r])
    head = int(rng.integers(0, n_pages))
    ring = rng.integers(-9, -1, n_pages)
    ring[(head + np.arange(n_pages - held)) % n_pages] = ids[held:]
    return lens, new, table, ring, head, n_pages - held


GROW = {"step": lambda r, a: a + 1, "grow": lambda r, a: a + int(r.integers(0, 70)), "same": lambda r, a: a,
        "shrink": lambda r, a: int(r.integers(0, a + 1)), "end": lambda r, a: 0,
        "mixed": lambda r, a: int(r.integers(0, 2 * a + 20))}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,page,most,kind", [
    (1, 16, 0, "step"), (1, 16, 100000, "mixed"), (3, 16, 40, "grow"), (7, 256, 700, "shrink"), (64, 32, 90, "end"),
    (224, 16, 500, "step"), (513, 64, 300, "mixed"), (2049, 16, 60, "mixed"), (300, 128, 1000, "same"),
    (5000, 16, 20, "mixed"), (1, 16, 300, "shrink")])
def test_page_tables_match_the_definition(rows, page, most, kind, in_place):
    rng = np.random.default_rng(rows * 7 + page)
    lens, new, table, ring, head, count = make(rng, rows, page, most, GROW[kind])
    total = sum(max(0, z - a) for a, z in zip(lens, new))
    cap = total + 3
    ok, et, er, es, el, esl, est = serving.page_tables(lens, new, table, ring, head, count, page, cap)
    assert ok
    t_lens, t_state = i32(lens), i32([head, count])
    t_table, t_ring = i32(table), i32(ring)
    lens_out = t_lens if in_place else torch.full((rows,), -7, dtype=torch.int32, device=DEV)
    state_out = t_state if in_place else torch.zeros(2, dtype=torch.int32, device=DEV)
    slots, start = i32(np.full(cap, -5)), i32(np.full(rows + 1, -5))
    before = B.kvc_launch_count()
    B.kvc_page_tables(lens=t_lens, lens_new=i32(new), table=t_table, ring=t_ring, state=t_state, page=page,
                      state_out=None if in_place else state_out, lens_out=lens_out, slots=slots, slot_start=start)
    assert B.kvc_check_status() == 0
    assert B.kvc_launch_count() - before == (2 if in_place else 1)
    for got, want in ((t_table, et), (t_ring, er), (state_out, es), (lens_out, el), (slots, esl), (start, est)):
        np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))
    if not in_place:
        assert t_lens.tolist() == lens and t_state.tolist() == [head, count]


@pytest.mark.parametrize("why", ["pages", "slots", "negative", "long", "head", "count"])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables_refuse_as_a_whole(why, in_place):
    rng = np.random.default_rng(5)
    lens, new, table, ring, head, count = make(rng, 37, 16, 200, GROW["grow"])
    cap = sum(max(0, z - a) for a, z in zip(lens, new))
    if why == "pages":
        need = sum(max(0, -(-z // 16) - -(-a // 16)) for a, z in zip(lens, new))
        count = need - 1
    elif why == "slots":
        cap -= 1
    elif why == "negative":
        new[20] = -1
    elif why == "long":
        new[3] = table.shape[1] * 16 + 1
    elif why == "head":
        head = len(ring)
    else:
        count = len(ring) + 1
    ok, et, er, es, el, esl, est = serving.page_tables(lens, new, table, ring, head, count, 16, cap)
    assert not ok
    t_lens, t_state = i32(lens), i32([head, count])
    t_table, t_ring = i32(table), i32(ring)
    lens_out = t_lens if in_place else torch.full((37,), -7, dtype=torch.int32, device=DEV)
    state_out = t_state if in_place else torch.zeros(2, dtype=torch.int32, device=DEV)
    slots, start = i32(np.full(cap, -5)), i32(np.full(38, -5))
    B.kvc_page_tables(lens=t_lens, lens_new=i32(new), table=t_table, ring=t_ring, state=t_state, page=16,
                      state_out=None if in_place else state_out, lens_out=lens_out, slots=slots, slot_start=start)
    with pytest.raises(B.KvcError) as e:
        B.kvc_check_status()
    assert e.value.status == 6
    for got, want in ((t_table, et), (t_ring, er), (state_out, es), (lens_out, el), (slots, esl), (start, est)):
        np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))


def test_page_ids_outside_the_pool_are_recorded_and_not_used():
    lens, new = [10, 16, 0], [20, 30, 3]
    table = np.array([[2, -1], [77, -1], [-1, -1]])
    ring = np.array([3, 99, 4, 0, 1, 5])
    slots, start = i32(np.full(40, -5)), i32(np.zeros(4))
    B.kvc_page_tables(lens=i32(lens), lens_new=i32(new), table=i32(table), ring=i32(ring), state=i32([0, 3]), page=16,
                      state_out=i32([0, 0]), slots=slots, slot_start=start)
    with pytest.raises(B.KvcError):
        B.kvc_check_status()
    s = slots.tolist()
    assert s[:10] == [2 * 16 + t for t in range(10, 16)] + [3 * 16 + t for t in range(4)]
    assert s[10:24] == [-1] * 14                                     # page 99 does not exist
    assert s[24:27] == [4 * 16, 4 * 16 + 1, 4 * 16 + 2] and s[27:] == [-1] * 13


def test_page_tables_strided_rows_captured_and_replayed():
    """In place, rows of a wider table, in a graph: three replays are three decode steps."""
    rng = np.random.default_rng(11)
    rows, page = 50, 16
    lens, new, table, ring, head, count = make(rng, rows, page, 60, GROW["same"], spare=300)
    wide = np.full((rows, table.shape[1] + 9), -3)
    wide[:, :table.shape[1]] = table
    t_lens, t_state, t_ring = i32(lens), i32([head, count]), i32(ring)
    t_wide = i32(wide)
    t_table = t_wide[:, :table.shape[1] + 4]
    nxt = torch.empty_like(t_lens)
    slots, start = i32(np.zeros(rows)), i32(np.zeros(rows + 1))
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)

    def step():
        torch.add(t_lens, 1, out=nxt)
        B.kvc_page_tables(lens=t_lens, lens_new=nxt, table=t_table, ring=t_ring, state=t_state, page=page,
                          lens_out=t_lens, slots=slots, slot_start=start, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.add(t_lens, 1, out=nxt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    tb = wide[:, :table.shape[1] + 4]
    for _ in range(3):
        g.replay()
        ok, tb, ring, (head, count), lens, sl, st = serving.page_tables(lens, [a + 1 for a in lens], tb, ring, head, count,
                                                                        page, rows)
        assert ok
        torch.cuda.synchronize()
        np.testing.assert_array_equal(t_table.cpu().numpy(), tb)
        np.testing.assert_array_equal(t_ring.cpu().numpy(), ring)
        np.testing.assert_array_equal(slots.cpu().numpy(), sl)
        assert t_state.tolist() == [head, count] and t_lens.tolist() == lens
    assert (t_wide[:, table.shape[1] + 4:] == -3).all()
    assert B.kvc_check_status() == 0


# ----------------------------------------------------------------------------- append

def pools(n_pages, H, page, d, dt, layout, g):
    if layout == "head":
        return [torch.randn(n_pages, H, page, d, device=DEV, generator=g).to(dt) for _ in range(2)]
    return [torch.randn(n_pages, page, H, d, device=DEV, generator=g).to(dt).transpose(1, 2) for _ in range(2)]


@pytest.mark.parametrize("T,H,d,page,dt,layout", [
    (1, 1, 64, 16, torch.bfloat16, "head"), (5, 4, 128, 16, torch.bfloat16, "token"), (300, 7, 64, 32, torch.float32, "head"),
    (129, 8, 128, 256, torch.bfloat16, "head"), (1000, 3, 128, 64, torch.float32, "token"), (0, 2, 64, 16, torch.float32, "head")])
def test_page_append_is_bit_exact(T, H, d, page, dt, layout):
    g = torch.Generator(device=DEV).manual_seed(T + H)
    n_pages = -(-T // page) + 4
    K, V = pools(n_pages, H, page, d, dt, layout, g)
    qkv = torch.randn(T, 3 * H * d + 8, device=DEV, generator=g).to(dt)      # rows of a wider projection
    k, v = qkv[:, H * d:2 * H * d].unflatten(1, (H, d)), qkv[:, 2 * H * d:3 * H * d].unflatten(1, (H, d))
    slots = torch.randperm(n_pages * page, device=DEV, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    slots[3::11] = -2 ** 31
    eK, eV = K.clone(), V.clone()
    keep = slots >= 0
    at = slots[keep].long()
    eK[at // page, :, at % page] = k[keep]
    eV[at // page, :, at % page] = v[keep]
    B.kvc_page_append(B.model(1, H, H, d), k=k, v=v, K=K, V=V, slots=slots)
    assert B.kvc_check_status() == 0
    assert torch.equal(K, eK) and torch.equal(V, eV)


def test_page_append_skips_and_records_slots_past_the_pool():
    g = torch.Generator(device=DEV).manual_seed(1)
    K, V = pools(3, 2, 16, 64, torch.float32, "head", g)
    k, v = torch.randn(4, 2, 64, device=DEV), torch.randn(4, 2, 64, device=DEV)
    eK = K.clone()
    eK[0, :, 5] = k[1]
    B.kvc_page_append(B.model(1, 2, 2, 64), k=k, v=v, K=K, V=V, slots=i32([48, 5, 2 ** 31 - 1, -1]))
    with pytest.raises(B.KvcError) as e:
        B.kvc_check_status()
    assert e.value.status == 6 and torch.equal(K, eK)


def test_page_append_to_a_pool_past_32_bit_offsets():
    """Element offsets above 2^31 (a 5 GB bf16 pool) on the last page."""
    H, d, page = 8, 128, 256
    n_pages = 2 ** 31 // (H * d * page) + 600
    K = torch.zeros(n_pages, H, page, d, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    k = torch.randn(2, H, d, device=DEV).to(torch.bfloat16)
    v = torch.randn(2, H, d, device=DEV).to(torch.bfloat16)
    last = n_pages * page - 1
    B.kvc_page_append(B.model(1, H, H, d), k=k, v=v, K=K, V=V, slots=i32([last, last - page]))
    assert B.kvc_check_status() == 0
    for t, s in ((0, last), (1, last - page)):
        assert torch.equal(K[s // page, :, s % page], k[t]) and torch.equal(V[s // page, :, s % page], v[t])
    assert int(torch.count_nonzero(K)) == int(torch.count_nonzero(k)) and int(torch.count_nonzero(V)) == int(torch.count_nonzero(v))


def test_calls_on_another_stream_and_wrong_arguments():
    g = torch.Generator(device=DEV).manual_seed(2)
    K, V = pools(3, 2, 16, 64, torch.float32, "head", g)
    k, v = torch.randn(4, 2, 64, device=DEV), torch.randn(4, 2, 64, device=DEV)
    m = B.model(1, 2, 2, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.kvc_page_append(m, k=k, v=v, K=K, V=V, slots=i32([0, 17, 40, 3]), stream=s)
    s.synchronize()
    assert torch.equal(K[1, :, 1], k[1])
    before = B.kvc_launch_count()
    with pytest.raises(B.KvcError):                                  # dtypes differ
        B.kvc_page_append(m, k=k.bfloat16(), v=v, K=K, V=V, slots=i32([0, 17, 40, 3]))
    with pytest.raises(ValueError):                                  # host tensor
        B.kvc_page_append(m, k=k.cpu(), v=v, K=K, V=V, slots=i32([0, 17, 40, 3]))
    with pytest.raises(ValueError):                                  # too few slots
        B.kvc_page_append(m, k=k, v=v, K=K, V=V, slots=i32([0, 17, 40]))
    with pytest.raises(B.KvcError):                                  # a page of 8 tokens
        B.kvc_page_append(m, k=k, v=v, K=K[:, :, :8], V=V[:, :, :8], slots=i32([0, 17, 40, 3]))
    with pytest.raises(TypeError):
        B.kvc_page_append(m, k=k, v=v, K=K, V=V, slots=torch.zeros(4, dtype=torch.int64, device=DEV))
    assert B.kvc_launch_count() == before


@pytest.mark.parametrize("rows,skip", [(40001, 0), (9001, 1)])
def test_page_tables_many_rows_one_long_among_short_and_unaligned_lengths(rows, skip):
    """Many rows to a thread, one row as long as a thousand others, lengths at any alignment."""
    rng = np.random.default_rng(rows)
    page = 64

    def new_of(r, a):
        new_of.n += 1
        return 30000 if new_of.n == rows // 3 else int(r.integers(0, 60))

    new_of.n = 0
    lens, new, table, ring, head, count = make(rng, rows, page, 50, new_of)
    total = sum(max(0, z - a) for a, z in zip(lens, new))
    ok, et, er, es, el, esl, est = serving.page_tables(lens, new, table, ring, head, count, page, total + 70)
    assert ok
    off = lambda x: i32(np.concatenate([np.full(skip, -9), x]).astype(np.int64))[skip:]
    t_table, t_ring = i32(table), i32(ring)
    lens_out, state_out = torch.full((rows,), -7, dtype=torch.int32, device=DEV), i32([0, 0])
    slots, start = i32(np.full(total + 70, -5)), i32(np.full(rows + 1, -5))
    B.kvc_page_tables(lens=off(lens), lens_new=off(new), table=t_table, ring=t_ring, state=i32([head, count]), page=page,
                      state_out=state_out, lens_out=lens_out, slots=slots, slot_start=start)
    assert B.kvc_check_status() == 0
    for got, want in ((t_table, et), (t_ring, er), (state_out, es), (lens_out, el), (slots, esl), (start, est)):
        np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))


def test_page_tables_without_slots_and_pools_on_two_streams():
    """Tables alone (no slot map, no starts), two pools resized at once on streams of their own."""
    rng = np.random.default_rng(77)
    runs = []
    for k in range(2):
        lens, new, table, ring, head, count = make(rng, 700 + k, 32, 400, GROW["mixed"])
        ok, et, er, es, el, _, _ = serving.page_tables(lens, new, table, ring, head, count, 32)
        assert ok
        runs.append(dict(lens=i32(lens), lens_new=i32(new), table=i32(table), ring=i32(ring), state=i32([head, count]),
                         state_out=i32([0, 0]), lens_out=i32(np.zeros(len(lens))), want=(et, er, es, el)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r, s in zip(runs, streams):
        B.kvc_page_tables(page=32, stream=s, **{k: v for k, v in r.items() if k != "want"})
    torch.cuda.synchronize()
    assert B.kvc_check_status() == 0
    for r in runs:
        for got, want in zip((r["table"], r["ring"], r["state_out"], r["lens_out"]), r["want"]):
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))
