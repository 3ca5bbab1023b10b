"""The paged caches where a serving program meets their edges: pools that run out, rows of very
unequal weight over long lines, shared prefixes. Where nothing else is said the models and the
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


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_prompt_that_gets_no_pages_stays_out(kv):
    """Prompts of which the pool holds the first only, then steps of the sequences that the table
    holds, as README has the loop: the refused ones stay idle when pages become free, until their prompt
    is reserved again."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(74)
    B, Hq, Hkv, page, cap = 3, 4, 2, 16, 64
    t = layer.PageTable(B, 3, page, cap)
    pl = layer.PagedLayer(t, Hq, Hkv, 2, 20, cap, [1, 0],
                          torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn, BASE)
    for x in (pl.k, pl.v):                                # what nothing wrote is NaN
        x.view(torch.uint8).fill_(0xFF)
    lens = np.array([20, 30, 10])
    new = lambda n, h: _bf(rng.normal(size=(B, n, h, 128)))
    q, kp, vp = new(30, Hq), new(30, Hkv), new(30, Hkv)
    slots = torch.empty((B, 30), dtype=torch.int32, device=DEV)
    out = torch.zeros_like(q)

    def prompts():
        t.reserve(torch.where(t.lens > 0, t.lens, _i32(lens)), slots)
        pl.prefill(q, kp, vp, _i32(lens), slots, out)

    def steps(n, live):
        for _ in range(n):
            before = t.lens.tolist()
            t.reserve(t.lens + (t.lens > 0))
            want = [m + 1 if b in live else 0 for b, m in enumerate(before)]
            assert t.step_lens.tolist() == want
            qs, ks, vs = (x[:, 0].contiguous() for x in (new(1, Hq), new(1, Hkv), new(1, Hkv)))
            o, lse = torch.zeros_like(qs), torch.zeros((B, Hq), device=DEV)
            pl.decode_append(ks, vs, qs, t.step_lens, o, lse)
            for b in range(B):
                if b in live:
                    assert torch.isfinite(o[b].float()).all() and torch.isfinite(lse[b]).all()
                else:
                    assert not o[b].any() and (lse[b] == -np.inf).all()

    prompts()
    assert t.lens.tolist() == [20, 0, 0]                  # the second lacks a page; nobody passes it
    steps(3, [0])
    t.reserve(_i32([0, 0, 0]))
    steps(2, [])
    lens[0] = 0
    prompts()
    assert t.lens.tolist() == [0, 30, 10]
    steps(2, [1, 2])
    assert t.status() == 0 and pl.status() == 0


# ------------------------------------------------------------------ one row above a long line

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [4096, 131072])
def test_decode_dominating_row_over_a_long_line(n, kv):
    """A first row whose logit is 18 above the others', in groups that lie in a warp or two each: the
    others weigh 2^-26 of it one by one, and several per cent of the output together. (Every page but
    the first is the same one.)

    The tolerance. As in test_gpu_paged.py a logit is off by e = 136 * 2^-23 * max S at most, and a
    weight relatively by d = 2 e + 2^-15 (16-bit terms): that moves the output by d sum_n p_n |v_n - o|.
    The e4m3 step's weights are two fp16 terms of 2^6 times the weight against a reference that some
    row has reached: below fp16's normal numbers the second term is off by 2^-25, so each row adds
    2^-31 max|v|. Sums: two products a tile that may cut, N / 16 * 2^-22 of sum_n p_n |v_n|."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(n)
    page, Hkv, big = 256, 8, 18.0
    warps = torch.cuda.get_device_properties(0).multi_processor_count * (8 if kv == "bf16" else 12)
    B = -(-warps // Hkv)
    q64 = _f64(_bf(rng.normal(size=(Hkv, 128))))
    z = rng.normal(size=(Hkv, 2 * page))
    z[:, 0] = big
    K = np.empty((Hkv, 2 * page, 128))
    V = 1 + 0.1 * rng.normal(size=(Hkv, 2 * page, 128))
    V[:, 0] *= 0.05                                       # a sink: small values, but for one channel,
    V[:, 0, 0] = 1.25                                     # so that its e4m3 scale is the others'
    k, v = (torch.empty((2, Hkv, page, 128), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device=DEV)
            for _ in range(2))
    scales = [None, None] if kv == "bf16" else [torch.empty((2, Hkv, page), device=DEV) for _ in range(2)]
    for g in range(Hkv):
        qr = rope_rotate(q64[g], n - 1, BASE)
        K[g] = z[g, :, None] * 128 ** 0.5 * qr / (qr @ qr)
        for x, dst, sc in ((K, k, scales[0]), (V, v, scales[1])):
            if kv == "bf16":
                dst[:, g] = _bf(PO.stored_rows(x[g], kv)).view(2, page, 128)
            else:
                r, s = PO.e4m3_rows(x[g])
                r8 = torch.from_numpy(r.astype(np.float32)).to(DEV).to(torch.float8_e4m3fn)
                dst[:, g] = r8.view(torch.uint8).view(2, page, 128)
                sc[:, g] = torch.from_numpy(s.reshape(2, page)).to(DEV)
            x[g] = PO.stored_rows(x[g], kv)
    table = np.ones((B, n // page))
    table[:, 0] = 0
    desc = rtp.LayerDesc(B, Hkv, Hkv, 0, 1, n, rtp.rtp_build_slot_map([1] * Hkv)[0], BASE)
    cache = rtp.make_paged_cache(k, v, _i32(table), *scales)
    ws = torch.empty(rtp.rtp_paged_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_workspace_init(ws)
    q = _bf(q64)[None].repeat(B, 1, 1)
    out, lse = torch.zeros_like(q), torch.zeros((B, Hkv), device=DEV)
    rtp.rtp_paged_decode_step(desc, cache, q, _i32(np.full(B, n)), out, lse, ws)
    assert rtp.rtp_read_device_status(ws) == 0
    times = np.r_[np.ones(page), np.full(page, n // page - 1)]
    for g in range(Hkv):
        qr = rope_rotate(q64[g], n - 1, BASE)
        x = K[g] @ qr / 128 ** 0.5
        w = times * np.exp(x - x.max())
        L = w.sum()
        p = w / L
        o, e = p @ V[g], x.max() + np.log(L)
        assert 1 - p[0] > n * 2.0 ** -26                  # the others' share is there to be lost
        err = 136 * 2.0 ** -23 * (np.abs(K[g]) @ np.abs(qr)).max() / 128 ** 0.5
        floor = n * 2.0 ** -31 * np.abs(V[g]).max() if kv == "e4m3" else 0.0
        tol = (2.0 ** -8 * np.abs(o) + (2 * err + 2.0 ** -15) * (p @ np.abs(V[g] - o)) + floor
               + n / 16 * 2.0 ** -22 * (p @ np.abs(V[g])))
        d = np.abs(_f64(out)[:, g] - o)
        assert (d <= tol).all(), (g, (d / np.abs(o)).max(), (d / tol).max())
        t = err + n / 16 * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * abs(e)
        assert np.abs(lse[:, g].double().cpu().numpy() - e).max() <= t


# ------------------------------------------------------------------ layers of several RoPE bases

def test_append_with_many_rope_bases():
    """Appends of layers that take turns with six RoPE bases, more than are kept: rows against the
    formula in 64 bits, half a bf16 step and 2^-40 for the angles."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(71)
    B, n, Hkv, page, start = 1, 900, 4, 64, 5000
    slots = _i32(np.arange(n)[None])
    for i in range(12):
        base = [1e4, 1e6, 5e5, 1e7, 2.0, 1e5][i % 6]
        kp, vp = (_bf(rng.normal(size=(B, n, Hkv, 128))) for _ in range(2))
        k, v = (torch.zeros((-(-n // page), Hkv, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        desc = rtp.LayerDesc(B, Hkv, Hkv, 0, 1, 1 << 20, rtp.rtp_build_slot_map([1] * Hkv)[0], base)
        cache = rtp.make_paged_cache(k, v, torch.zeros((B, 1), dtype=torch.int32, device=DEV))
        rtp.rtp_paged_append_kv(desc, cache, kp, vp, _i32([start]), slots, n)
        a = (start + np.arange(n))[:, None, None] * base ** (-np.arange(64) / 64.0)
        x = _f64(kp)[0]
        want = np.concatenate([x[..., :64] * np.cos(a) - x[..., 64:] * np.sin(a),
                               x[..., :64] * np.sin(a) + x[..., 64:] * np.cos(a)], -1)
        got = _f64(k).swapaxes(1, 2).reshape(-1, Hkv, 128)[:n]
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -40).all(), base


# ------------------------------------------------------------------ nothing to append

def test_calls_of_no_tokens():
    """An empty chunk through the layer: an append of [B][0] tokens, a reservation without new tokens."""
    _, layer, rtp = _mods()
    t = layer.PageTable(2, 4, 16, 64)
    pl = layer.PagedLayer(t, 4, 2, 2, 20, 64, [1, 0])
    pl.k.zero_()
    t.reserve(_i32([5, 0]), torch.empty((2, 0), dtype=torch.int32, device=DEV))
    assert t.lens.tolist() == [5, 0] and t.step_lens.tolist() == [5, 0]
    rows = torch.empty((2, 0, 2, 128), dtype=torch.bfloat16, device=DEV)
    pl.append(rows, rows, t.lens, torch.empty((2, 0), dtype=torch.int32, device=DEV))
    assert rtp.rtp_last_launch_count() == 0
    assert t.status() == 0 and pl.status() == 0 and not pl.k.any()


# ------------------------------------------------------------------ a shared prefix

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_shared_prefix_is_a_sequence_of_its_own(kv):
    """Two sequences behind a common prefix of two pages, as the header has it: the prefix is a third
    sequence of the pool, and a table of the caller's puts its pages before theirs. Steps over that
    table against the model; in the end every page is free once."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(72)
    Hq, Hkv, page, cap, sinks, window, pre = 8, 2, 16, 96, 2, 20, 32
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    t = layer.PageTable(3, 9, page, cap)                  # sequences 0 and 1, the prefix
    pl = layer.PagedLayer(t, Hq, Hkv, sinks, window, cap, [1, 0], dt, BASE)
    kp, vp = (_bf(rng.normal(size=(3, pre, Hkv, 128))) for _ in range(2))
    slots = torch.empty((3, pre), dtype=torch.int32, device=DEV)
    t.reserve(_i32([0, 0, pre]), slots)
    pl.append(kp, vp, pl.zeros, slots)
    both = torch.full((2, 6), -1, dtype=torch.int32, device=DEV)
    both[:, :2] = t.block_table[2, :2]
    cache = rtp.make_paged_cache(pl.k, pl.v, both, pl.k_scale, pl.v_scale)
    desc = rtp.LayerDesc(2, Hq, Hkv, sinks, window, cap, rtp.rtp_build_slot_map([1, 0])[0], BASE)
    K = {(b, g): [rope_rotate(_f64(kp)[2, j, g], j, BASE) for j in range(pre)] for b in range(2) for g in range(Hkv)}
    V = {(b, g): list(_f64(vp)[2, :, g]) for b in range(2) for g in range(Hkv)}
    c = Case.__new__(Case)
    c.G, c.ret, c.sinks, c.window = Hq // Hkv, [True, False], sinks, window
    for i in range(20):
        n = i + 1
        t.reserve(_i32([n, max(0, n - 3), pre]))          # sequence 1 starts three steps later
        both[:, 2:5] = t.block_table[:2, :3]
        lens = torch.where(t.step_lens[:2] > 0, t.step_lens[:2] + pre, 0)
        q, k, v = (_bf(rng.normal(size=(2, h, 128))) for h in (Hq, Hkv, Hkv))
        out, lse = torch.zeros_like(q), torch.zeros((2, Hq), device=DEV)
        rtp.rtp_paged_decode_step_append(desc, cache, k, v, q, lens, out, lse, pl.ws)
        c.q64 = _f64(q)
        for b, m in enumerate(lens.tolist()):
            for g in range(Hkv if m else 0):
                K[b, g].append(rope_rotate(_f64(k)[b, g], m - 1, BASE))
                V[b, g].append(_f64(v)[b, g])
        c.rows = {name: {key: PO.stored_rows(np.array(r), kv) for key, r in rs.items()} for name, rs in (("k", K), ("v", V))}
        for b, m in enumerate(lens.tolist()):
            for h in range(Hq if m else 0):
                c.agree(_f64(out)[b, h], float(lse[b, h]), b, h, m)
    t.reserve(_i32([0, 0, 0]))
    free = [int(t.free_pages[i % 9]) for i in range(*t.counters.tolist())]
    assert sorted(free) == list(range(9)) and t.status() == 0 and pl.status() == 0


# ------------------------------------------------------------------ paged and contiguous appends

@pytest.mark.parametrize("n", [1, 2, 40, 4099])
def test_append_rows_next_to_the_contiguous_ones(n):
    """Rows at far positions against rtp_append_kv's, in calls that share a sine among one, two, four and
    eight tokens. One token: the same bits. Otherwise a key may differ where it lies next to the middle
    of two bf16 values: turned-on angles differ by pos 2^-52 + 2^-50 (two roundings of position *
    theta, and a few of the products), and the value formed here by as much again."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(n)
    B, Hkv, page, start = 1, 4, 128, 1_000_003
    end = start + n
    kp, vp = (_bf(rng.normal(size=(B, n, Hkv, 128))) for _ in range(2))
    lay = layer.DecodeLayer(B, Hkv, Hkv, 4, 64, end, [1] * Hkv, [end], DEV, BASE)
    lay.append(kp, vp, torch.zeros((Hkv, 128, 16), device=DEV), _i32([start]))
    k, v = (torch.zeros((-(-n // page), Hkv, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    desc = rtp.LayerDesc(B, Hkv, Hkv, 4, 64, end, rtp.rtp_build_slot_map([1] * Hkv)[0], BASE)
    cache = rtp.make_paged_cache(k, v, torch.zeros((B, 1), dtype=torch.int32, device=DEV))
    rtp.rtp_paged_append_kv(desc, cache, kp, vp, _i32([start]), _i32(np.arange(n)[None]), n)
    flat = lambda x: _f64(x).swapaxes(1, 2).reshape(-1, Hkv, 128)[:n]
    theirs = lambda x: _f64(x[:, start:end]).swapaxes(0, 1)
    assert np.array_equal(flat(v), theirs(lay.v_ret)) and lay.status() == 0
    a, b = flat(k), theirs(lay.k_ret)
    bad = a != b
    if n == 1:
        assert not bad.any()
    pos = start + np.arange(n)
    ang = pos[:, None, None] * BASE ** (-np.arange(64) / 64.0)
    x = _f64(kp)[0]
    u, w = x[..., :64], x[..., 64:]
    want = np.concatenate([u * np.cos(ang) - w * np.sin(ang), u * np.sin(ang) + w * np.cos(ang)], -1)
    length = np.tile(np.hypot(u, w), 2)
    room = 2 * (2.0 ** -52 * pos[:, None, None] + 2.0 ** -50) * length
    assert (np.abs(want - (a + b) / 2)[bad] <= room[bad]).all()
    assert bad.sum() <= 1e-6 * bad.size + 1


# ------------------------------------------------------------------ more than 32 sequences

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [33, 64, 700])
def test_steps_of_many_short_sequences(B, kv):
    """Batches of more than one block of 32 lengths, some places idle: the fused step's outputs and
    pages are those of append and step, and the model's."""
    _, _, rtp = _mods()
    lens = np.random.default_rng(B).integers(0, 70, B)
    lens[::7] = 0
    c = Case(B, lens, 16, kv, G=2, Hkv=3, ret=(True, False, True), window=9, sinks=2)
    kn, vn = (_bf(c.rng.normal(size=(B, c.Hkv, 128))) for _ in range(2))
    pools = [x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]
    first = [x.view(torch.uint8).clone() for x in pools]
    out, lse = c.outputs()
    rtp.rtp_paged_decode_step_append(c.desc, c.cache, kn, vn, c.q, c.sl, out, lse, c.ws)
    assert c.status() == 0
    fused = [x.view(torch.uint8).clone() for x in pools]
    for x, y in zip(pools, first):
        x.view(torch.uint8).copy_(y)
    slots = [-1 if n == 0 else int(c.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16 for b, n in enumerate(lens)]
    rtp.rtp_paged_append_kv(c.desc, c.cache, kn, vn, c.sl - 1, _i32(slots), 1, c.ws)
    out2, lse2 = c.decode()
    assert c.status() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(pools, fused):
        assert torch.equal(x.view(torch.uint8), y)
    for b, n in enumerate(lens):
        for g in range(c.Hkv if n else 0):
            for name, new in (("k", rope_rotate(_f64(kn[b, g]), n - 1, BASE)), ("v", _f64(vn[b, g]))):
                c.rows[name][b, g][-1] = PO.stored_rows(new, kv)
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("append", [False, True])
def test_steps_of_many_long_sequences(append, kv):
    """41 sequences of up to 60000 tokens, some places idle, retrieval and local heads: a line long
    enough to leave ranges to the CTAs done first (bf16), which start in other blocks of 32 lengths.
    Against 64-bit sums on the GPU; three calls give the same bits."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(73)
    gen = torch.Generator(device=DEV).manual_seed(73)
    B, G, Hkv, page, sinks, window, ret = 41, 2, 4, 64, 4, 500, [1, 0, 1, 1]
    lens = rng.integers(1, 60001, B)
    lens[[0, 13, 31, 32]] = 0
    assert 3 * (lens / 16).sum() > torch.cuda.get_device_properties(0).multi_processor_count * 8 * 128
    need = -(-lens // page)
    n_pages = int(need.sum()) + 1
    ids, table = rng.permutation(n_pages), np.full((B, need.max()), -1)
    for b, at in enumerate(np.cumsum(need) - need):
        table[b, :need[b]] = ids[at:at + need[b]]
    shape = (n_pages, Hkv, page, 128)
    pools = {x: torch.randn(shape, dtype=torch.bfloat16, device=DEV, generator=gen) for x in "kv"}
    scales = dict(k=None, v=None)
    if kv == "e4m3":
        for x, p in pools.items():
            scales[x] = (p.abs().amax(-1).float() / 448.0).contiguous()
            pools[x] = (p.float() / scales[x][..., None]).to(torch.float8_e4m3fn)
    bt, sl = _i32(table), _i32(lens)
    q = (2 * torch.randn((B, G * Hkv, 128), device=DEV, generator=gen)).to(torch.bfloat16)
    kn, vn = (torch.randn((B, Hkv, 128), device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2))
    desc = rtp.LayerDesc(B, G * Hkv, Hkv, sinks, window, 1 << 16, rtp.rtp_build_slot_map(ret)[0], BASE)
    cache = rtp.make_paged_cache(pools["k"], pools["v"], bt, scales["k"], scales["v"])
    ws = torch.empty(rtp.rtp_paged_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_workspace_init(ws)
    outs = []
    for _ in range(3):
        out = torch.full((B, G * Hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, G * Hkv), 7.0, device=DEV)
        if append:
            rtp.rtp_paged_decode_step_append(desc, cache, kn, vn, q, sl, out, lse, ws)
        else:
            rtp.rtp_paged_decode_step(desc, cache, q, sl, out, lse, ws)
        outs.append((out, lse))
    assert rtp.rtp_read_device_status(ws) == 0 and not ws[:4096].any()
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
    out, lse = outs[0]
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            assert not out[b].any() and (lse[b] == -np.inf).all()
            continue
        at = bt[b, :need[b]].long()
        for g in range(Hkv) if b % 8 == 1 else [b % Hkv]:
            K, V = (pools[x][at, g].double() if scales[x] is None
                    else pools[x][at, g].float().double() * scales[x][at, g].double()[..., None] for x in "kv")
            K, V = K.reshape(-1, 128)[:n], V.reshape(-1, 128)[:n]
            if append:
                for x, new in ((K, rope_rotate(_f64(kn[b, g]), n - 1, BASE)), (V, _f64(vn[b, g]))):
                    assert torch.equal(x[-1].cpu(), torch.from_numpy(PO.stored_rows(new, kv)))
            pos = torch.from_numpy(PO.positions(n, not ret[g], sinks, window)).to(DEV)
            K, V = K[pos], V[pos]
            for h in range(G * g, G * g + G):
                qr = torch.from_numpy(rope_rotate(_f64(q[b, h]), n - 1, BASE)).to(DEV)
                z = K @ qr / 128 ** 0.5
                want, e = torch.softmax(z, 0) @ V, torch.logsumexp(z, 0).item()
                # as in test_gpu_paged.py, and the e4m3 weights' 2^-31 a row (see above)
                err = 136 * 2.0 ** -23 * (K.abs() @ qr.abs()).max().item() / 128 ** 0.5
                rows = len(pos)
                atol = (2 * err + 2.0 ** -15 + rows / 16 * 2.0 ** -22 + rows * 2.0 ** -31) * V.abs().max().item()
                d = (out[b, h].double() - want).abs()
                assert (d <= 2.0 ** -8 * want.abs() + atol).all(), (b, h, d.max().item(), atol)
                assert abs(lse[b, h].item() - e) <= err + rows / 16 * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * abs(e)


# ------------------------------------------------------------------ infinite keys

@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_heads_of_an_infinite_key(value):
    """A key with one infinite channel: a head's outputs are non-finite, or, where its logit is -inf,
    those without the row."""
    c = Case(75, [40 + b for b in range(8)], 16, "bf16", G=8, Hkv=2, ret=(True, True))
    rows = [(3 * b) % 40 for b in range(8)]
    for b, r in enumerate(rows):
        c.k[int(c.table[b, r // 16]), 0, r % 16, 17 * b % 128] = value
    out, lse = c.decode()
    assert c.status() == 0
    out, lse = _f64(out), _f64(lse)
    left_out = 0
    for b, n in enumerate(c.lens):
        for h in range(c.Hq):
            if h < c.G and not np.isfinite(out[b, h]).any():
                assert not np.isfinite(lse[b, h])
                continue
            keep = np.delete(np.arange(n), rows[b]) if h < c.G else None
            left_out += h < c.G
            if h < c.G:
                qr = rope_rotate(c.q64[b, h], n - 1, BASE)
                assert np.sign(qr[17 * b % 128]) != np.sign(value)
            c.agree(out[b, h], lse[b, h], b, h, n, keep)
    assert left_out < 32                                  # (a logit of +inf never is)
