"""Paged caches on the CPU: pins of the plain models, struct layouts, and every refusal that comes
before a launch."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from long_context_sparse_rtpurbo_b200 import _lib, rtp
from oracle import paged_oracle as PO

X = 0x1000                                   # an aligned pointer that nothing reads


def _desc(**kw):
    a = dict(B=2, Hq=32, Hkv=8, sinks=4, window=2048, max_seq_len=32768,
             slot_of_kv=rtp.rtp_build_slot_map([1, 0, 0, 0, 0, 1, 0, 0])[0])
    a.update(kw)
    return rtp.LayerDesc(**a)


def _cache(**kw):
    a = dict(kv_type=0, page_size=16, n_pages=100, table_stride=50, k=X, v=X, k_scale=None,
             v_scale=None, page_stride=0, block_table=X)
    a.update(kw)
    return _lib.RtpPagedCache(**a)


def _pool(**kw):
    a = dict(B=2, page_size=16, n_pages=100, table_stride=50, free_pages=X, block_table=X)
    a.update(kw)
    return _lib.RtpPagePool(**a)


# ------------------------------------------------------------------ the plain models

def test_e4m3_values_and_rounding_match_torch():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(PO.e4m3_values(), every.astype(np.float64), equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 4000) * 2.0 ** rng.integers(-12, 9, 4000), [0.0, 448, -448]])
    pos = PO.e4m3_values()[:0x7F]
    x = np.concatenate([x, (pos[1:] + pos[:-1]) / 2]).astype(np.float32)     # every tie
    x = x[np.abs(x) <= 448]
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(PO.e4m3_round(x), got)


def test_e4m3_rows_scale():
    q, s = PO.e4m3_rows(np.array([[0.0] * 4, [1.0, -448.0, 3.0, 0.0], [7.0, 0.25, -3.5, 1.0]]))
    assert s[0] == np.float32(2.0 ** -126) and not q[0].any()
    assert s[1] == 1.0 and np.array_equal(q[1], [1, -448, 3, 0])
    assert s[2] == np.float32(7) / np.float32(448) and q[2, 0] == 448 and q[2, 2] == -224


def test_attend_matches_torch_sdpa():
    rng = np.random.default_rng(1)
    q, K, V = rng.normal(size=128), rng.normal(size=(37, 128)), rng.normal(size=(37, 128))
    o, lse = PO.attend(q, K, V)
    t = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x)[None, None] for x in (q[None], K, V)))[0, 0, 0]
    assert np.allclose(o, t.numpy(), atol=1e-12)
    assert np.isclose(lse, torch.logsumexp(torch.from_numpy(K @ q / np.sqrt(128)), 0).item())
    o, lse = PO.attend(q, K[:0], V[:0])
    assert not o.any() and lse == -np.inf


def test_reserve_model_hand_worked():
    """Pages of 16. Sequence 0 holds 20 tokens (pages 7, 8) and grows to 40 (one page more), 1
    ends with one page, 2 starts with 33 tokens (three pages) which are not there, 3 starts with
    16 tokens: 4 pages lacked up to it, 1 free."""
    table = np.array([[7, 8, -1], [3, -1, -1], [-1] * 3, [-1] * 3])
    free = np.array([5, -1, -1, -1, -1, -1, -1, -1, -1, -1])
    r = PO.reserve(16, 10, table, free, [20, 9, 0, 0], [40, 0, 33, 16], [10, 11], 2)
    assert r["table"].tolist() == [[7, 8, 5], [3, -1, -1], [-1] * 3, [-1] * 3]
    assert r["lens"].tolist() == [40, 0, 0, 0] and r["counters"].tolist() == [11, 12]
    assert r["free"][:3].tolist() == [5, 3, -1]
    assert r["slots"].tolist() == [[8 * 16 + 4, 8 * 16 + 5], [-1, -1], [-1, -1], [-1, -1]]
    assert not r["error"]


def test_reserve_model_keeps_every_page_once():
    """Random rounds: held pages and free pages together are always every page, once."""
    rng = np.random.default_rng(2)
    B, page, n_pages, stride = 5, 16, 23, 9
    table, free = np.full((B, stride), -1), np.arange(n_pages)
    lens, counters = np.zeros(B, int), np.array([0, n_pages])
    for _ in range(60):
        new = rng.integers(0, stride * page + 1, B)
        r = PO.reserve(page, n_pages, table, free, lens, new, counters, 3)
        table, free, lens, counters = r["table"], r["free"], r["lens"], r["counters"]
        held = [int(p) for b in range(B) for p in table[b, :-(-lens[b] // page)]]
        ring = [int(free[i % n_pages]) for i in range(counters[0], counters[1])]
        assert sorted(held + ring) == list(range(n_pages))
        assert not r["error"] and all(x in (a, b) for x, a, b in zip(r["lens"], lens, new))
    assert counters[0] > n_pages                                     # the ring went round


# ------------------------------------------------------------------ structs and refusals

def test_struct_layouts_match_header():
    assert ctypes.sizeof(_lib.RtpPagedCache) == 4 * 4 + 4 * 8 + 8 + 8
    assert ctypes.sizeof(_lib.RtpPagePool) == 4 * 4 + 2 * 8
    assert rtp.RTP_PAGED_CTRL_BYTES == 4096


def test_workspace_bytes():
    need = rtp.rtp_paged_workspace_bytes(_desc())
    assert need > 4096
    assert rtp.rtp_paged_workspace_bytes(_desc(B=4000, max_seq_len=1 << 24)) == need
    assert rtp.rtp_paged_workspace_bytes(_desc(Hq=30)) == 0
    lib = _lib.load()
    assert lib.rtp_paged_workspace_init(None, 4096, None) == _lib.RTP_EWORKSPACE
    assert lib.rtp_paged_workspace_init(X, 4095, None) == _lib.RTP_EWORKSPACE
    assert lib.rtp_paged_workspace_init(X + 16, 4096, None) == _lib.RTP_EWORKSPACE


BAD_CACHES = [
    (dict(k=None), "RTP_EINVAL"), (dict(v=None), "RTP_EINVAL"), (dict(kv_type=2), "RTP_EINVAL"),
    (dict(kv_type=-1), "RTP_EINVAL"), (dict(k=X + 8), "RTP_EINVAL"), (dict(v=X + 8), "RTP_EINVAL"),
    (dict(kv_type=1), "RTP_EINVAL"), (dict(kv_type=1, k_scale=X), "RTP_EINVAL"),
    (dict(kv_type=1, k_scale=X, v_scale=X + 4), "RTP_EINVAL"),
    (dict(page_size=8), "RTP_ESHAPE"), (dict(page_size=48), "RTP_ESHAPE"),
    (dict(page_size=512), "RTP_ESHAPE"), (dict(page_size=0), "RTP_ESHAPE"),
    (dict(n_pages=0), "RTP_ESHAPE"), (dict(n_pages=1 << 27), "RTP_ESHAPE"),
    (dict(page_stride=127), "RTP_ESHAPE"), (dict(page_stride=1 << 25), "RTP_ESHAPE"),
    (dict(n_pages=1 << 24, page_size=64), "RTP_ESHAPE"),
]


def _decode_calls(d, cache, q=X, lens=X, out=X, ws=X, wsb=None, k=X, v=X):
    lib = _lib.load()
    wsb = rtp.rtp_paged_workspace_bytes(d) if wsb is None else wsb
    c = ctypes.byref(cache)
    return (lib.rtp_paged_decode_step(d.ref, c, q, lens, out, None, ws, wsb, None),
            lib.rtp_paged_decode_step_append(d.ref, c, k, v, q, lens, out, None, ws, wsb, None))


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused(kw, code):
    d, c, code = _desc(), _cache(**kw), getattr(_lib, code)
    assert _decode_calls(d, c) == (code, code)
    assert _lib.load().rtp_paged_append_kv(d.ref, ctypes.byref(c), X, X, X, X, 4, X, None) == code


def test_decode_refusals():
    d, c = _desc(), _cache()
    inv, shp, wsp = _lib.RTP_EINVAL, _lib.RTP_ESHAPE, _lib.RTP_EWORKSPACE
    assert _decode_calls(d, c, q=None) == (inv, inv)
    assert _decode_calls(d, c, lens=None) == (inv, inv)
    assert _decode_calls(d, c, out=None) == (inv, inv)
    assert _decode_calls(d, c, q=X + 2) == (inv, inv)
    assert _decode_calls(d, c, out=X + 2) == (inv, inv)
    assert _decode_calls(d, c, k=None, wsb=0) == (wsp, inv)
    assert _decode_calls(d, c, v=X + 2, wsb=0) == (wsp, inv)
    assert _decode_calls(d, _cache(block_table=None)) == (inv, inv)
    assert _decode_calls(d, _cache(table_stride=0)) == (shp, shp)
    assert _decode_calls(d, c, wsb=4096) == (wsp, wsp)
    assert _decode_calls(d, c, ws=None) == (wsp, wsp)
    assert _decode_calls(d, c, ws=X + 16) == (wsp, wsp)
    assert _decode_calls(_desc(Hq=24), c, wsb=1 << 30) == (shp, shp)
    assert _decode_calls(_desc(B=5000), c, wsb=1 << 30) == (shp, shp)
    lib = _lib.load()
    none = ctypes.POINTER(_lib.RtpPagedCache)()
    assert lib.rtp_paged_decode_step(d.ref, none, X, X, X, None, X, 1 << 30, None) == inv


def test_append_refusals():
    d, c, lib = _desc(), _cache(), _lib.load()
    call = lambda k=X, v=X, start=X, slots=X, n=4: lib.rtp_paged_append_kv(
        d.ref, ctypes.byref(c), k, v, start, slots, n, None, None)
    for kw in (dict(k=None), dict(v=None), dict(start=None), dict(slots=None), dict(n=-1),
               dict(k=X + 4), dict(v=X + 4)):
        assert call(**kw) == _lib.RTP_EINVAL, kw
    assert call(n=0) == _lib.RTP_OK
    assert rtp.rtp_last_launch_count() == 0


def test_reserve_refusals():
    lib = _lib.load()
    names = ("lens", "new", "ctr", "lens_out", "ctr_out")

    def call(pool=None, n_new=1, slots=X, ws=X, wsb=4096, **kw):
        p = _pool(**(pool or {}))
        return lib.rtp_paged_reserve(ctypes.byref(p), *(kw.get(n, X) for n in names), slots, n_new,
                                     ws, wsb, None)

    for n in names:
        assert call(**{n: None}) == _lib.RTP_EINVAL, n
    assert call(slots=None) == _lib.RTP_EINVAL
    assert call(n_new=-1) == _lib.RTP_EINVAL
    assert call(dict(free_pages=None)) == _lib.RTP_EINVAL
    assert call(dict(block_table=None)) == _lib.RTP_EINVAL
    for bad in (dict(B=0), dict(B=4097), dict(n_pages=0), dict(page_size=20), dict(table_stride=0),
                dict(page_size=256, n_pages=1 << 23)):
        assert call(bad) == _lib.RTP_ESHAPE, bad
    assert call(ws=None) == _lib.RTP_EWORKSPACE
    assert call(wsb=4095) == _lib.RTP_EWORKSPACE
    assert call(ws=X + 128) == _lib.RTP_EWORKSPACE


def test_injected_failures_come_first():
    d, c, lib = _desc(), _cache(), _lib.load()
    p = _pool()
    calls = [lambda: lib.rtp_paged_decode_step(d.ref, ctypes.byref(c), None, X, X, None, X, 0, None),
             lambda: lib.rtp_paged_decode_step_append(d.ref, ctypes.byref(c), X, X, None, X, X, None,
                                                      X, 0, None),
             lambda: lib.rtp_paged_append_kv(d.ref, ctypes.byref(c), None, X, X, X, 1, None, None),
             lambda: lib.rtp_paged_reserve(ctypes.byref(p), None, X, X, X, X, X, 1, X, 4096, None)]
    for call in calls:
        rtp.rtp_debug_fail_next_call(_lib.RTP_ECUDA)
        assert call() == _lib.RTP_ECUDA
        assert call() == _lib.RTP_EINVAL


# ------------------------------------------------------------------ the binding's own checks

def _cpu_cache(n_pages=3, Hkv=2, page=16, dtype=torch.bfloat16, **kw):
    k = torch.zeros((n_pages, Hkv, page, 128), dtype=dtype)
    a = dict(k=k, v=k.clone(), block_table=torch.zeros((2, 4), dtype=torch.int32))
    a.update(kw)
    return rtp.make_paged_cache(**a)


def test_binding_builds_the_cache_struct():
    c = _cpu_cache()
    assert (c.c.kv_type, c.c.page_size, c.c.n_pages, c.c.table_stride) == (0, 16, 3, 4)
    assert c.c.page_stride == 32
    both = torch.zeros((3, 2, 2, 16, 128), dtype=torch.bfloat16)
    c = _cpu_cache(k=both[:, 0], v=both[:, 1])                       # interleaved pages
    assert c.c.page_stride == 64 and c.c.v - c.c.k == 2 * 16 * 256
    sc = torch.ones((3, 2, 16))
    for dt in (torch.uint8, torch.float8_e4m3fn):
        assert _cpu_cache(dtype=dt, k_scale=sc, v_scale=sc.clone()).c.kv_type == 1


@pytest.mark.parametrize("kw", [
    dict(dtype=torch.float16), dict(dtype=torch.uint8), dict(k_scale=torch.ones((3, 2, 16))),
    dict(v=torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)),
    dict(v=torch.zeros((3, 2, 16, 128))),
    dict(k=torch.zeros((3, 16, 2, 128), dtype=torch.bfloat16).transpose(1, 2),
         v=torch.zeros((3, 16, 2, 128), dtype=torch.bfloat16).transpose(1, 2)),
    dict(k=torch.zeros((1, 2, 16, 128), dtype=torch.bfloat16).expand(3, -1, -1, -1),
         v=torch.zeros((1, 2, 16, 128), dtype=torch.bfloat16).expand(3, -1, -1, -1)),
    dict(block_table=torch.zeros((2, 4))), dict(block_table=torch.zeros(8, dtype=torch.int32)),
    dict(block_table=torch.zeros((4, 2), dtype=torch.int32).t()),
])
def test_binding_refuses_bad_caches(kw):
    with pytest.raises(ValueError):
        _cpu_cache(**kw)


def test_binding_refuses_bad_arguments():
    """Size, dtype and contiguity are checked before the library is called."""
    c = _cpu_cache()
    d = rtp.LayerDesc(2, 4, 2, 4, 64, 64, rtp.rtp_build_slot_map([1, 0])[0])
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(q_pre=bf(2, 4, 128), seq_lens=i32(2), out=bf(2, 4, 128), lse=torch.zeros(2, 4))
    for kw in (dict(q_pre=bf(2, 2, 128)), dict(q_pre=torch.zeros(2, 4, 128)),
               dict(q_pre=bf(4, 2, 128).transpose(0, 1)), dict(seq_lens=i32(3)),
               dict(seq_lens=torch.zeros(2, dtype=torch.int64)), dict(out=bf(2, 4, 64)),
               dict(lse=bf(2, 4))):
        with pytest.raises(ValueError):
            rtp.rtp_paged_decode_step(d, c, **(good | kw))
        with pytest.raises(ValueError):
            rtp.rtp_paged_decode_step_append(d, c, bf(2, 2, 128), bf(2, 2, 128), **(good | kw))
    with pytest.raises(ValueError):
        rtp.rtp_paged_decode_step_append(d, c, bf(2, 1, 128), bf(2, 2, 128), **good)
    other = rtp.LayerDesc(3, 4, 2, 4, 64, 64, rtp.rtp_build_slot_map([1, 0])[0])
    with pytest.raises(ValueError):
        rtp.rtp_paged_decode_step(other, c, **good)
    with pytest.raises(ValueError):
        rtp.rtp_paged_append_kv(d, c, bf(2, 3, 2, 128), bf(2, 3, 2, 128), i32(2), i32(2, 4), 3)
    pool = rtp.make_page_pool(i32(3), i32(2, 4), 16)
    ctr = torch.zeros(2, dtype=torch.int64)
    for a in itertools.combinations(range(5), 1):
        args = [i32(2), i32(2), ctr, i32(2), ctr]
        args[a[0]] = torch.zeros(2)
        with pytest.raises(ValueError):
            rtp.rtp_paged_reserve(pool, *args, i32(2, 1), 1, torch.zeros(4096, dtype=torch.uint8))


def test_append_refuses_a_workspace_without_a_status_word():
    lib, c = _lib.load(), _cache()
    d = _desc()
    assert lib.rtp_paged_append_kv(d.ref, ctypes.byref(c), X, X, X, X, 4, X + 2, None) == _lib.RTP_EWORKSPACE
    c = _cpu_cache()
    d = rtp.LayerDesc(2, 4, 2, 4, 64, 64, rtp.rtp_build_slot_map([1, 0])[0])
    rows = torch.zeros((2, 3, 2, 128), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="status word"):
        rtp.rtp_paged_append_kv(d, c, rows, rows, i32(2), i32(2, 3), 3,
                                torch.zeros(3, dtype=torch.uint8))
