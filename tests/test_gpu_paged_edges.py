"""The paged caches where a serving program meets their edges: pools that run out. The models and the
tolerances of a decode step are those of test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from oracle.rtp_oracle import rope_rotate
from test_gpu_paged import BASE, DEV, Case, _bf, _f64, _mods

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.asarray(a).astype(np.int32)).to(DEV)


# ------------------------------------------------------------------ a pool that runs out

@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,page,stride,n_pages,n_new", [
    (1, 16, 1, 1, 1), (3, 64, 5, 11, 0), (33, 32, 7, 150, 9), (33, 32, 7, 60, 9), (64, 16, 40, 300, 1),
    (513, 16, 9, 1500, 5), (4096, 16, 4, 5000, 1)])
def test_reserve_step_lens(B, page, stride, n_pages, n_new, inplace):
    """step_lens is the new length where a sequence was served and grew, 0 elsewhere; the other
    outputs are those of the call without it."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(B + n_pages)
    table, free, lens = np.full((B, stride), -1), rng.permutation(n_pages), np.zeros(B, int)
    counters = np.array([0, n_pages])
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    for _ in range(6):
        new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, stride * page + 1, B))
        new = np.where(rng.random(B) < 0.5, np.minimum(lens + 1, stride * page), new)
        new = np.where(rng.random(B) < 0.1, lens, new)
        want = PO.reserve(page, n_pages, table, free, lens, new, counters, n_new)
        step = np.where(want["lens"] > lens, want["lens"], 0)
        t, f, l0, l1 = _i32(table), _i32(free), _i32(lens), _i32(new)
        c0 = torch.from_numpy(counters.astype(np.int64)).to(DEV)
        lo, co = (l0, c0) if inplace else (torch.zeros_like(l0), torch.zeros_like(c0))
        slots = torch.full((B, n_new), 77, dtype=torch.int32, device=DEV)
        got = torch.full((B,), 77, dtype=torch.int32, device=DEV)
        rtp.rtp_paged_reserve_step(rtp.make_page_pool(f, t, page), l0, l1, c0, lo, co,
                                   slots if n_new else None, n_new, got, ws)
        assert np.array_equal(got.cpu().numpy(), step)
        for name, x in (("table", t), ("free", f), ("lens", lo), ("counters", co), ("slots", slots)):
            assert np.array_equal(x.cpu().numpy(), want[name]), name
        table, free, lens, counters = want["table"], want["free"], want["lens"], want["counters"]
    assert rtp.rtp_read_device_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("how", ["calls", "graph"])
def test_a_sequence_that_gets_no_page_is_idle(kv, how):
    """Steps of a pool with one page to spare for two sequences at a page's end: the one that is
    refused keeps every row bit for bit, and its outputs are those of an idle place; once another
    has ended it goes on where it stopped."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(70)
    B, Hq, Hkv, page, cap, sinks, window = 4, 8, 2, 16, 64, 2, 20
    t = layer.PageTable(B, 4, page, cap)
    pl = layer.PagedLayer(t, Hq, Hkv, sinks, window, cap, [1, 0],
                          torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn, BASE)
    pools = [x for x in (pl.k, pl.v, pl.k_scale, pl.v_scale) if x is not None]
    for x in pools:
        x.view(torch.uint8).fill_(0x55)
    first = np.array([16, 16, 10, 0])
    kp, vp = (_bf(rng.normal(size=(B, 16, Hkv, 128))) for _ in range(2))
    slots = torch.empty((B, 16), dtype=torch.int32, device=DEV)
    t.reserve(_i32(first), slots)
    pl.append(kp, vp, pl.zeros, slots)
    K = {(b, g): [rope_rotate(_f64(kp)[b, j, g], j, BASE) for j in range(first[b])] for b in range(B) for g in range(Hkv)}
    V = {(b, g): [_f64(vp)[b, j, g] for j in range(first[b])] for b in range(B) for g in range(Hkv)}
    q, k, v = (torch.zeros((B, h, 128), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    out, lse = torch.zeros_like(q), torch.zeros((B, Hq), device=DEV)
    grow, new = torch.zeros_like(t.lens), torch.zeros_like(t.lens)
    c = Case.__new__(Case)
    c.G, c.ret, c.sinks, c.window = Hq // Hkv, [True, False], sinks, window

    def step():
        torch.add(t.lens, grow, out=new)
        t.reserve(new)
        pl.decode_append(k, v, q, t.step_lens, out, lse)

    step()                                                # nobody grows: all idle
    assert not out.any() and t.step_lens.tolist() == [0] * B
    run = step
    if how == "graph":
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    # what each step wishes (None: ends), and who is served
    for wish, served in (([1, 1, 1, 0], [0, 2]), ([1, 1, 0, 0], [0]), ([None, 1, 1, 0], [2]),
                         ([0, 1, 1, 0], [1, 2]), ([0, 1, 1, 0], [1, 2])):
        lens = t.lens.tolist()
        grow.copy_(_i32([-n if w is None else w for w, n in zip(wish, lens)]))
        for x in (q, k, v):
            x.copy_(_bf(rng.normal(size=x.shape)))
        before = [x.clone() for x in pools]
        run()
        want = [n + 1 if b in served else 0 if w is None else n for b, (w, n) in enumerate(zip(wish, lens))]
        assert t.lens.tolist() == want
        assert t.step_lens.tolist() == [want[b] if b in served else 0 for b in range(B)]
        bt = t.block_table.cpu().numpy()
        rows = sorted((int(bt[b, lens[b] // page]), lens[b] % page) for b in served)
        for x, y in zip(pools, before):
            x, y = (z.view(torch.uint8).reshape(4, Hkv, page, -1) for z in (x, y))
            moved = (x != y).any(-1).any(1).nonzero().tolist()
            assert sorted(map(tuple, moved)) == rows
        for b in served:
            for h in range(Hkv):
                K[b, h].append(rope_rotate(_f64(k)[b, h], lens[b], BASE))
                V[b, h].append(_f64(v)[b, h])
        c.q64 = _f64(q)
        c.rows = {name: {key: PO.stored_rows(np.array(r), kv) for key, r in rs.items() if r}
                  for name, rs in (("k", K), ("v", V))}
        for b in range(B):
            for h in range(Hq):
                if b in served:
                    c.agree(_f64(out)[b, h], float(lse[b, h]), b, h, want[b])
                else:
                    assert not out[b, h].any() and float(lse[b, h]) == -np.inf
    assert t.status() == 0 and pl.status() == 0
