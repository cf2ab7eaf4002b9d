"""kvc_page_tables, kvc_page_append, kvc_prefix_decode_attn and kvc_sample refuse bad arguments on the host,
before anything is launched (no GPU; fake device addresses, nothing is dereferenced), and the oracle
of the batch steps is held to hand-worked values."""
import ctypes as C

import numpy as np
import pytest

from long_context_kv_obs_b200 import binding as B
from oracle import serving

ARG, UNSUPPORTED, WORKSPACE = 1, 2, 3


def each(args, call, cases):
    before = B.kvc_launch_count()
    for field, bad, code in cases:
        good = getattr(args, field)
        if isinstance(good, C.Structure):                            # a view of the field: keep a copy
            good = type(good).from_buffer_copy(good)
        setattr(args, field, bad)
        assert call() == code, (field, bad, B.lib().kvc_last_error())
        setattr(args, field, good)
    assert B.kvc_launch_count() == before


def test_page_tables_refusals():
    lib = B.lib()
    a = B.PageTablesArgs()
    a.rows, a.page, a.n_pages, a.max_pages, a.table_s_row = 10, 16, 100, 8, 8
    a.len, a.len_new, a.table, a.ring, a.state, a.state_out = 0x1000, 0x2000, 0x3000, 0x8000, 0x9000, 0x9100
    a.len_out = 0xa000
    n = C.c_size_t(7)
    assert lib.kvc_workspace_size(B.OP_PAGE_TABLES, None, C.byref(a), C.byref(n)) == 0 and n.value == 0
    a.len_out = a.len                                                # in place: the verdict needs a workspace
    assert lib.kvc_workspace_size(B.OP_PAGE_TABLES, None, C.byref(a), C.byref(n)) == 0 and n.value > 0
    assert lib.kvc_page_tables(C.byref(a), None, 0, None) == WORKSPACE
    assert lib.kvc_page_tables(C.byref(a), C.c_void_p(0xb000), n.value - 1, None) == WORKSPACE
    a.len_out = 0xa000
    each(a, lambda: lib.kvc_page_tables(C.byref(a), None, 0, None), [
        ("rows", 0, ARG), ("rows", 2 ** 20 + 1, ARG), ("page", 8, UNSUPPORTED), ("page", 48, UNSUPPORTED), ("n_pages", 0, ARG),
        ("n_pages", 2 ** 27, ARG), ("max_pages", 0, ARG), ("table_s_row", 7, ARG), ("len", None, ARG), ("len_new", None, ARG),
        ("table", None, ARG), ("ring", None, ARG), ("state", None, ARG), ("state_out", None, ARG), ("len_out", 0x1004, ARG),
        ("len_out", 0x1ffc, ARG), ("state_out", 0x9004, ARG)])
    a.slots = 0xc000
    each(a, lambda: lib.kvc_page_tables(C.byref(a), None, 0, None), [("slots_cap", -1, ARG)])
    assert lib.kvc_page_tables(None, None, 0, None) == ARG


def test_page_append_refusals():
    lib = B.lib()
    m = B.model(1, 4, 4, 128)
    kv = lambda p, dt=B.KVC_BF16, st=512: B.KV(p, dt, 4 * 16 * 128, 0, 128, st)
    a = B.PageAppendArgs()
    a.T, a.page, a.n_pages, a.slots = 3, 16, 10, 0x1000
    a.k, a.v, a.K, a.V = kv(0x10000), kv(0x20000), kv(0x30000), kv(0x40000)
    each(a, lambda: lib.kvc_page_append(C.byref(m), C.byref(a), None), [
        ("T", -1, ARG), ("page", 17, UNSUPPORTED), ("n_pages", 0, ARG), ("slots", None, ARG), ("k", kv(None), ARG),
        ("v", kv(0x20008), ARG), ("K", kv(0x30000, B.KVC_F32), ARG), ("V", kv(0x40000, st=100), ARG),
        ("k", kv(0x10000, st=516), ARG), ("v", B.KV(0x20000, 7, 0, 0, 128, 512), ARG)])
    a.T = 0                                                          # nothing to do is no error, and no launch
    before = B.kvc_launch_count()
    assert lib.kvc_page_append(C.byref(m), C.byref(a), None) == 0 and B.kvc_launch_count() == before
    assert lib.kvc_page_append(C.byref(B.model(1, 4, 4, 96)), C.byref(a), None) == UNSUPPORTED


def test_prefix_decode_refusals():
    lib = B.lib()
    m = B.model(2, 8, 2, 128)
    cache = lambda p, dt=B.KVC_BF16: B.KV(p, dt, 2 * 2 * 64 * 128, 2 * 64 * 128, 64 * 128, 128)
    a = B.PrefixDecodeArgs()
    a.batch, a.q, a.q_dtype, a.o = 3, 0x1000, B.KVC_BF16, 0x2000
    a.K_prefix, a.V_prefix, a.len_prefix, a.max_len_prefix = cache(0x10000), cache(0x20000), 0x3000, 64
    a.K, a.V, a.len, a.max_len = cache(0x30000), cache(0x40000), 0x4000, 64
    a.table, a.table_s_batch, a.table_s_layer, a.page, a.n_pages = 0x5000, 8, 4, 16, 50
    n = C.c_size_t(0)
    size = lambda: lib.kvc_workspace_size(B.OP_PREFIX_DECODE, C.byref(m), C.byref(a), C.byref(n))
    assert size() == 0 and n.value > 0
    assert lib.kvc_prefix_decode_attn(C.byref(m), C.byref(a), None, 0, None) == WORKSPACE
    assert lib.kvc_prefix_decode_attn(C.byref(m), C.byref(a), C.c_void_p(0x100000), n.value - 1, None) == WORKSPACE
    assert lib.kvc_prefix_decode_attn(C.byref(m), C.byref(a), C.c_void_p(0x100008), n.value, None) == ARG
    none = B.KV()
    each(a, size, [
        ("batch", 0, ARG), ("batch", 2 ** 26, UNSUPPORTED), ("q", None, ARG), ("q", 0x1008, ARG), ("o", 0x2004, ARG),
        ("q_dtype", 5, ARG), ("scale", -1.0, ARG), ("scale", float("inf"), ARG), ("scale", float("nan"), ARG),
        ("lse_stride", -1, ARG), ("K_prefix", cache(0x10008), ARG), ("V_prefix", cache(0x20000, B.KVC_F32), ARG),
        ("len_prefix", None, ARG), ("max_len_prefix", 0, ARG), ("K", cache(0x30000, B.KVC_F32), ARG), ("V", none, ARG),
        ("len", None, ARG), ("max_len", 0, ARG), ("page", 24, UNSUPPORTED), ("n_pages", 0, ARG), ("table_s_layer", -1, ARG),
        ("K", none, ARG)])                                            # a table without K
    a.R, a.alpha_c = 0x6000, float("nan")
    assert size() == ARG
    a.alpha_c = 1.0
    assert size() == 0
    a.K_prefix = none                                                # R without a prompt
    assert size() == ARG
    a.R, a.K, a.table = None, none, None                             # neither side
    assert size() == ARG
    a.K_prefix = cache(0x10000)
    assert lib.kvc_workspace_size(B.OP_PREFIX_DECODE, C.byref(B.model(2, 18, 2, 128)), C.byref(a), C.byref(n)) == UNSUPPORTED
    assert lib.kvc_workspace_size(B.OP_PREFIX_DECODE, None, C.byref(a), C.byref(n)) == ARG


def test_sample_refusals():
    lib = B.lib()
    a = B.SampleArgs()
    a.n, a.V, a.logits, a.dtype, a.row_stride, a.u, a.token = 4, 1000, 0x1000, B.KVC_BF16, 1000, 0x2000, 0x3000
    each(a, lambda: lib.kvc_sample(C.byref(a), None), [
        ("n", 0, ARG), ("V", 0, UNSUPPORTED), ("V", 262145, UNSUPPORTED), ("logits", None, ARG), ("logits", 0x1001, ARG),
        ("dtype", 3, ARG), ("row_stride", 999, ARG), ("u", None, ARG), ("token", None, ARG)])
    assert lib.kvc_sample(None, None) == ARG


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros(2, 10)
    with pytest.raises(ValueError):
        B.kvc_sample(logits=z, u=z[:, 0], token=torch.zeros(2, dtype=torch.int32))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kvc_page_tables(lens=i, lens_new=i, table=torch.zeros(4, 2, dtype=torch.int32), ring=i, state=i[:2], page=16)


def test_prefix_decode_refuses_bounds_whose_sums_pass_32_bits():
    lib = B.lib()
    m = B.model(2, 8, 2, 128)
    cache = lambda p: B.KV(p, B.KVC_BF16, 2 * 2 * 64 * 128, 2 * 64 * 128, 64 * 128, 128)
    a = B.PrefixDecodeArgs()
    a.batch, a.q, a.q_dtype, a.o = 3, 0x1000, B.KVC_BF16, 0x2000
    a.K_prefix, a.V_prefix, a.len_prefix, a.max_len_prefix = cache(0x10000), cache(0x20000), 0x3000, 64
    a.K, a.V, a.len, a.max_len = cache(0x30000), cache(0x40000), 0x4000, 64
    n = C.c_size_t(0)
    size = lambda: lib.kvc_workspace_size(B.OP_PREFIX_DECODE, C.byref(m), C.byref(a), C.byref(n))
    for table in (None, 0x5000):
        a.table, a.table_s_batch, a.table_s_layer, a.page, a.n_pages = table, 8, 4, 16, 50
        each(a, size, [("max_len", 2 ** 30 + 1, UNSUPPORTED), ("max_len", 2 ** 31 - 1, UNSUPPORTED),
                       ("max_len_prefix", 2 ** 30 + 1, UNSUPPORTED), ("max_len_prefix", 2 ** 31 - 1, UNSUPPORTED)])
        a.max_len = a.max_len_prefix = 2 ** 30                       # the most: a workspace of records that fit
        assert size() == 0 and 0 < n.value < 2 ** 34
        a.max_len = a.max_len_prefix = 64
    a.batch, a.max_len_prefix = 2 ** 21, 2 ** 20                      # 2^17 row blocks of 2^13 tiles
    assert size() == UNSUPPORTED
    a.max_len_prefix = 2 ** 10
    assert size() == 0


def test_binding_refuses_halves_of_a_cache():
    import torch
    m = B.model(2, 8, 2, 64)
    q, o = torch.zeros(3, 2, 8, 64), torch.zeros(3, 2, 8, 64)
    cache, own = torch.zeros(2, 2, 10, 64), torch.zeros(3, 2, 2, 10, 64)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    prompt = dict(K_prefix=cache, V_prefix=cache, lens_prefix=i(2), max_len_prefix=10)
    for half in (dict(K_prefix=cache), dict(V_prefix=cache), dict(prompt, K=own), dict(prompt, V=own), dict(prompt, V_prefix=None)):
        with pytest.raises(ValueError, match="belong together"):
            B.kvc_prefix_decode_attn(m, q=q, o=o, lens=i(3, 2), max_len=10, **half)
    with pytest.raises(ValueError, match="table belongs"):
        B.kvc_prefix_decode_attn(m, q=q, o=o, table=i(3, 2, 1), lens=i(3, 2), max_len=10, **prompt)


# ----------------------------------------------------------------------------- the oracle by hand

def test_oracle_page_tables_by_hand():
    table = np.array([[7, -1, -1], [2, 3, 4], [-1, -1, -1]])
    ring = np.array([9, 9, 9, 9, 9, 5, 6, 1, 0, 9])                  # head 5: pages 5, 6, 1, 0 are free
    ok, t, r, state, lens, slots, start = serving.page_tables([15, 40, 0], [18, 16, 17], table, ring, 5, 4, 16, 25)
    assert ok and lens == [18, 16, 17]
    assert t.tolist() == [[7, 5, -1], [2, 3, 4], [6, 1, -1]]
    assert r.tolist() == [4, 9, 9, 9, 9, 5, 6, 1, 0, 3] and state == (8, 3)
    assert start.tolist() == [0, 3, 3, 20]
    assert slots.tolist() == [7 * 16 + 15, 5 * 16, 5 * 16 + 1] + [6 * 16 + i for i in range(16)] + [16] + [-1] * 5
    ok, t, r, state, lens, slots, start = serving.page_tables([15, 40, 0], [18, 16, 70], table, ring, 5, 4, 16, 99)
    assert not ok and lens == [15, 40, 0] and (slots == -1).all() and state == (5, 4)


def test_oracle_sampling_by_hand():
    z = np.log([0.1, 0.4, 0.2, 0.3])
    for u, want in ((0.0, 0), (0.09, 0), (0.11, 1), (0.49, 1), (0.51, 2), (0.71, 3), (0.99, 3)):
        assert serving.sample(z, u)[0] == want
    assert serving.sample(z, 0.5, top_k=2) == (1, pytest.approx(np.log(4 / 7)), 2)
    assert serving.sample(z, 0.9, top_p=0.69)[::2] == (3, 2)         # 0.4 + 0.3 reach 0.69
    assert serving.sample(z, 0.9, top_p=0.71)[::2] == (3, 3)
    assert serving.sample(z, 0.0, min_p=0.6)[::2] == (1, 2)          # 0.3 >= 0.6 * 0.4, 0.2 is below
    assert serving.sample(z, 0.7, temperature=0.0) == (1, 0.0, 1)
    assert serving.sample([1.0, 1.0, 1.0, 1.0], 0.5, top_k=3)[0] == 1   # ties: the first three
    assert serving.sample([-np.inf, np.nan], 0.5) == (-1, -np.inf, 0)
    p2 = np.array([0.1, 0.4, 0.2, 0.3]) ** 2
    assert serving.sample(z, 0.2, temperature=0.5)[1] == pytest.approx(np.log(p2[1] / p2.sum()))


def test_oracle_prefix_attention_is_one_softmax():
    r = np.random.default_rng(0)
    q, kp, vp, ko, vo = r.normal(size=(3, 8)), r.normal(size=(5, 8)), r.normal(size=(5, 8)), r.normal(size=(4, 8)), r.normal(size=(4, 8))
    R = r.uniform(1, 3, 5)
    o, lse, w = serving.prefix_attention(q, kp, vp, ko, vo, R, alpha_c=0.5, scale=0.3)
    z = np.concatenate([q @ kp.T * 0.3 + 0.5 * np.log(R), q @ ko.T * 0.3], axis=1)
    e = np.exp(z)
    np.testing.assert_allclose(w, e / e.sum(1, keepdims=True))
    np.testing.assert_allclose(o, w @ np.concatenate([vp, vo]))
    np.testing.assert_allclose(lse, np.log(e.sum(1)))
    o0, lse0, _ = serving.prefix_attention(q, kp[:0], vp[:0], ko[:0], vo[:0])
    assert (o0 == 0).all() and (lse0 == -np.inf).all()
