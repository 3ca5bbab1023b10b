"""The paged-cache operators on the GPU against plain 64-bit models.

Tolerances of the decode step. Inputs are what the cache holds (exact) and bf16 queries.
Logits: products are exact, a dot product of 128 terms and the query's rotation and split are
off by at most (128 + 8) roundings of 2^-23 of S = sum_i |q_i k_i| / sqrt(128) (the accumulators
may cut instead of rounding, hence 2^-23): e = 136 * 2^-23 * max_n S_n, plus the logit's own last
rounding. Weights then are off by a factor exp(+-2e) (numerator and denominator) and their two
16-bit terms by 2^-16; a row's sum of N weights adds N / 16 * 2^-23 (each lane sums every 16th
row). So |out - ref| <= 2^-8 |ref| (bf16) + (2 e + 2^-15 + N / 16 * 2^-22) max|v|, and lse is off
by at most e + N / 16 * 2^-23 + 2^-21 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from oracle.rtp_oracle import bf16_round, rope_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
BASE = 1e6


def _mods():
    from long_context_sparse_rtpurbo_b200 import _lib, layer, rtp
    return _lib, layer, rtp


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).to(DEV)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _table(rng, lens, page, n_pages=None, stride=None, shuffle=True):
    need = [-(-int(n) // page) for n in lens]
    n_pages = n_pages or sum(need) + 3
    stride = stride or max(1, max(need)) + 1
    pages = rng.permutation(n_pages) if shuffle else np.arange(n_pages)
    t = np.full((len(lens), stride), 0x7fffffff, np.int64)       # behind the end: not a page
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = pages[at:at + k]
        at += k
    return t, n_pages


class Case:
    """A paged cache filled with random rows; every other row of the pool is NaN."""

    def __init__(self, seed, lens, page, kv="bf16", G=4, Hkv=2, ret=(True, False), sinks=4, window=64,
                 interleave=False, max_seq_len=None, q_scale=2.0, n_pages=None, scale_spread=0):
        _, _, rtp = _mods()
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.page, self.kv, self.G, self.Hkv = np.asarray(lens), page, kv, G, Hkv
        self.B, self.Hq, self.ret, self.sinks, self.window = len(lens), G * Hkv, ret, sinks, window
        self.table, self.n_pages = _table(rng, lens, page, n_pages)
        dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        shape = (self.n_pages, Hkv, page, 128)
        if interleave:
            both = torch.empty((self.n_pages, 2, Hkv, page, 128), dtype=dt, device=DEV)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = (torch.empty(shape, dtype=dt, device=DEV) for _ in range(2))
        self.k_scale = self.v_scale = None
        if kv == "e4m3":
            self.k_scale, self.v_scale = (torch.full(shape[:3], float("nan"), device=DEV)
                                          for _ in range(2))
        self.bt = torch.from_numpy(self.table.astype(np.int32)).to(DEV)
        for t in (self.k, self.v):
            if kv == "bf16":
                t.fill_(float("nan"))
            else:
                t.view(torch.uint8).fill_(0x7F)
        self.rows = {"k": {}, "v": {}}
        for b, n in enumerate(self.lens):
            for g in range(Hkv):
                for name in ("k", "v"):
                    x = rng.normal(size=(n, 128))
                    if scale_spread:
                        x = x * 2.0 ** rng.integers(-scale_spread, scale_spread + 1, (n, 1))
                    self.rows[name][b, g] = x
        self.write()
        q = bf16_round(rng.normal(size=(self.B, self.Hq, 128)) * q_scale)
        self.q64, self.q = q, _bf(q)
        slots = rtp.rtp_build_slot_map(ret)[0]
        self.desc = rtp.LayerDesc(self.B, self.Hq, Hkv, sinks, window,
                                  max_seq_len or max(1, int(self.lens.max())), slots, BASE)
        self.cache = rtp.make_paged_cache(self.k, self.v, self.bt, self.k_scale, self.v_scale)
        self.ws = torch.empty(rtp.rtp_paged_workspace_bytes(self.desc), dtype=torch.uint8, device=DEV)
        rtp.rtp_paged_workspace_init(self.ws)
        self.sl = torch.from_numpy(self.lens.astype(np.int32)).to(DEV)

    def write(self):
        """The rows into the pages, as float64 of what is stored back into self.rows."""
        for name, dst, sc in (("k", self.k, self.k_scale), ("v", self.v, self.v_scale)):
            for (b, g), x in self.rows[name].items():
                n = len(x)
                if n == 0:
                    continue
                pos = np.arange(n)
                pg = torch.from_numpy(self.table[b, pos // self.page]).to(DEV)
                r = torch.from_numpy(pos % self.page).to(DEV)
                if self.kv == "bf16":
                    self.rows[name][b, g] = bf16_round(x)
                    dst[pg, g, r] = _bf(bf16_round(x))
                else:
                    q, s = PO.e4m3_rows(x)
                    self.rows[name][b, g] = q * s.astype(np.float64)[:, None]
                    q8 = torch.from_numpy(q.astype(np.float32)).to(DEV).to(torch.float8_e4m3fn)
                    dst.view(torch.uint8)[pg, g, r] = q8.view(torch.uint8)
                    sc[pg, g, r] = torch.from_numpy(s).to(DEV)

    def outputs(self):
        out = torch.full((self.B, self.Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        return out, torch.full((self.B, self.Hq), 7.0, device=DEV)

    def decode(self, sl=None, stream=None):
        _, _, rtp = _mods()
        out, lse = self.outputs()
        rtp.rtp_paged_decode_step(self.desc, self.cache, self.q, self.sl if sl is None else sl, out,
                                  lse, self.ws, stream)
        return out, lse

    def status(self):
        st = _mods()[2].rtp_read_device_status(self.ws)
        assert not self.ws[:4096].any()            # the counters are back at zero
        return st

    def agree(self, out, lse, b, h, n, keep=None):
        """One head's outputs against the model over positions 0..n-1 (or `keep` of them)."""
        g, local = h // self.G, not self.ret[h // self.G]
        pos = PO.positions(n, local, self.sinks, self.window) if keep is None else keep
        K, V = self.rows["k"][b, g][pos], self.rows["v"][b, g][pos]
        q = rope_rotate(self.q64[b, h], n - 1, BASE)
        o, e = PO.attend(q, K, V)
        err = 136 * 2.0 ** -23 * (np.abs(K) @ np.abs(q)).max() / 128 ** 0.5
        atol = (2 * err + 2.0 ** -15 + len(pos) / 16 * 2.0 ** -22) * np.abs(V).max()
        d = np.abs(out - o)
        assert (d <= 2.0 ** -8 * np.abs(o) + atol).all(), (b, h, n, d.max(), atol)
        t = err + len(pos) / 16 * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * abs(e)
        assert abs(lse - e) <= t, (b, h, n, lse, e, t)

    def check(self, out, lse, heads=None, lens=None):
        out, lse = _f64(out), _f64(lse)
        lens = self.lens if lens is None else lens
        for b in range(self.B):
            n = int(lens[b])
            for h in range(self.Hq) if heads is None else heads:
                if n == 0:
                    assert not out[b, h].any() and lse[b, h] == -np.inf
                else:
                    self.agree(out[b, h], lse[b, h], b, h, n)


EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 129, 255, 256, 300]


# ------------------------------------------------------------------ decode step

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_edge_lengths(page, kv):
    """Lengths around tiles and pages, an idle place, rows behind the end NaN, table entries
    behind the end no pages; one dense and one local KV head."""
    c = Case(page, EDGES, page, kv)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,Hkv", [(1, 1), (1, 5), (2, 3), (4, 1), (8, 2), (8, 8)])
def test_decode_head_layouts(G, Hkv, kv):
    ret = [(g % 3) != 1 for g in range(Hkv)]
    c = Case(G * 10 + Hkv, [257, 1, 40], 32, kv, G=G, Hkv=Hkv, ret=ret)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("sinks,window", [(0, 1), (0, 16), (4, 1), (17, 30), (16, 16), (5, 4096),
                                          (300, 7), (33, 100)])
def test_decode_local_masks(sinks, window):
    """Sinks and window that meet, overlap, end inside tiles or cover everything."""
    c = Case(sinks + window, [1, 5, 16, 33, 34, 48, 64, 65, 130, 301], 16, sinks=sinks, window=window,
             ret=(False, False))
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_long_split(kv):
    """One sequence over many CTAs: parts merged through the workspace; lengths that leave the
    CTAs uneven ranges; called three times, the same bits each time."""
    c = Case(3, [20011], 64, kv, G=4, Hkv=2, ret=(True, False), window=2048)
    got = [c.decode() for _ in range(3)]
    assert c.status() == 0
    c.check(*got[0])
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


@pytest.mark.parametrize("G", [1, 8])
def test_decode_one_head_over_all_ctas(G):
    """A single KV head over the whole GPU: the largest merge."""
    c = Case(4, [70003], 256, "bf16", G=G, Hkv=1, ret=(True,))
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


def test_decode_many_short_sequences():
    """More groups than warps, most of them inside one warp's range; some places idle."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 700)
    lens[::7] = 0
    c = Case(6, lens, 16, "bf16", G=2, Hkv=3, ret=(True, False, True), window=9, sinks=2)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


def test_decode_largest_batch():
    lens = np.random.default_rng(8).integers(0, 3, 4096)
    c = Case(9, lens, 16, "bf16", G=1, Hkv=1, ret=(True,))
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [639, 641, 960, 961])
def test_decode_around_one_cta_per_group(n, kv):
    """Lengths around those up to which a group stays in one CTA (40 and 60 tiles of 16 rows)."""
    c = Case(n, [n, 0, 17, n - 1], 16, kv, G=2, Hkv=4, ret=(True, False, True, False), window=700)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("Hkv,n", [(1, 2_500_007), (8, 310_000)])
def test_decode_longest_lines(Hkv, n):
    """Lines long enough to leave a share to the CTAs that are done first: one group in some 300
    parts, and eight groups. Against 64-bit sums on the GPU; three calls give the same bits,
    whichever CTA took which part."""
    _, _, rtp = _mods()
    page, G = 128, 2
    gen = torch.Generator(device=DEV).manual_seed(n)
    n_pages = -(-n // page)
    k, v = (torch.randn((n_pages, Hkv, page, 128), dtype=torch.bfloat16, device=DEV, generator=gen) for _ in range(2))
    table = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)[None].contiguous()
    q = (2 * torch.randn((1, G * Hkv, 128), device=DEV, generator=gen)).to(torch.bfloat16)
    desc = rtp.LayerDesc(1, G * Hkv, Hkv, 0, 1, 1 << 22, rtp.rtp_build_slot_map([1] * Hkv)[0], BASE)
    cache = rtp.make_paged_cache(k, v, table)
    ws = torch.empty(rtp.rtp_paged_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_workspace_init(ws)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        out = torch.full((1, G * Hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((1, G * Hkv), 7.0, device=DEV)
        rtp.rtp_paged_decode_step(desc, cache, q, lens, out, lse, ws)
        assert rtp.rtp_last_launch_count() == 1
        outs.append((out, lse))
    assert rtp.rtp_read_device_status(ws) == 0 and not ws[:4096].any()
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
    q64 = torch.from_numpy(rope_rotate(_f64(q)[0], n - 1, BASE)).to(DEV)
    for h in range(0, G * Hkv, 3):
        K = k[table[0].long(), h // G].reshape(-1, 128)[:n].double()
        S = (K.abs() @ q64[h].abs()).max().item() / 128 ** 0.5
        z = K @ q64[h] / 128 ** 0.5
        del K
        V = v[table[0].long(), h // G].reshape(-1, 128)[:n].double()
        want, e = torch.softmax(z, 0) @ V, torch.logsumexp(z, 0).item()
        # as above; a lane's sum of weights is over the 16 rows' share of one warp's tiles (about
        # n / (16 * 8 * 296)), the parts' sums are joined one after the other, at most 300 of them
        terms = n / (16 * 8 * 296) + 300 + 16
        err = 136 * 2.0 ** -23 * S
        atol = (2 * err + 2.0 ** -15 + terms * 2.0 ** -22) * V.abs().max().item()
        d = (outs[0][0][0, h].double() - want).abs()
        assert (d <= 2.0 ** -8 * want.abs() + atol).all(), (h, d.max().item(), atol)
        assert abs(outs[0][1][0, h].item() - e) <= err + terms * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * abs(e)
        del V, z


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_interleaved_pages(kv):
    """K and V pages side by side in one allocation (page_stride)."""
    c = Case(10, [100, 33, 250], 32, kv, interleave=True)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


def test_decode_far_rows():
    """Pages beyond 2^32 bytes of a pool (only those pages are written)."""
    page, n_pages = 64, 36000                       # 8 KV heads: 131 KB a page, 4.7 GB
    _, _, rtp = _mods()
    assert n_pages * 8 * page * 256 > 1 << 32
    rng = np.random.default_rng(11)
    c = Case.__new__(Case)
    c.rng, c.lens, c.page, c.kv, c.G, c.Hkv = rng, np.array([200]), page, "bf16", 1, 8
    c.B, c.Hq, c.ret, c.sinks, c.window = 1, 8, [True] * 4 + [False] * 4, 4, 32
    c.table, c.n_pages = np.array([[35999, 0, 35998, 33000]]), n_pages
    c.k, c.v = (torch.empty((n_pages, 8, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.k_scale = c.v_scale = None
    c.bt = torch.from_numpy(c.table.astype(np.int32)).to(DEV)
    c.rows = {n: {(0, g): rng.normal(size=(200, 128)) for g in range(8)} for n in "kv"}
    c.write()
    c.q64 = bf16_round(rng.normal(size=(1, 8, 128)) * 2)
    c.q = _bf(c.q64)
    c.desc = rtp.LayerDesc(1, 8, 8, 4, 32, 256, rtp.rtp_build_slot_map(c.ret)[0], BASE)
    c.cache = rtp.make_paged_cache(c.k, c.v, c.bt)
    c.ws = torch.empty(rtp.rtp_paged_workspace_bytes(c.desc), dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_workspace_init(c.ws)
    c.sl = torch.tensor([200], dtype=torch.int32, device=DEV)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


def test_decode_shared_pages():
    """Two sequences with a common prefix of pages."""
    c = Case(12, [96, 96], 32, "bf16")
    c.table[1, :2] = c.table[0, :2]
    c.bt.copy_(torch.from_numpy(c.table.astype(np.int32)))
    for n in "kv":
        for g in range(2):
            x = c.rows[n][1, g].copy()
            x[:64] = c.rows[n][0, g][:64]
            c.rows[n][1, g] = x
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_rows_of_unequal_size(kv):
    """Rows whose sizes differ by 2^24 (scales of an e4m3 cache), and large queries."""
    c = Case(13, [150, 700], 32, kv, scale_spread=12, q_scale=0.01)
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)
    c = Case(14, [150, 700], 32, kv, q_scale=300.0)            # one-hot rows
    out, lse = c.decode()
    c.check(out, lse)


def test_decode_zero_query_and_zero_rows():
    c = Case(15, [50, 17], 16, "e4m3")
    c.q.zero_()
    c.q64 = np.zeros_like(c.q64)
    for n in "kv":
        c.rows[n][0, 0] = np.zeros((50, 128))
    c.write()
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)
    assert not _f64(out)[0, :4].any()


def test_decode_nonfinite_rows_stay_in_their_heads():
    """NaN and infinity in an attended row reach that KV head's outputs and no others."""
    c = Case(16, [40, 40, 40], 16, "bf16", ret=(True, True))
    clean = c.decode()
    c.v[int(c.table[1, 1]), 0, 3] = float("nan")
    c.k[int(c.table[2, 0]), 1, 5] = float("inf")
    out, lse = c.decode()
    o, p = _f64(out), _f64(clean[0])
    assert np.isnan(o[1, :4]).all() and np.array_equal(o[1, 4:], p[1, 4:])
    assert not np.isfinite(o[2, 4:]).any() and np.array_equal(o[2, :4], p[2, :4])
    assert np.array_equal(o[0], p[0])


def test_decode_reports_bad_lengths_and_pages():
    """A length out of range is an idle place; rows of a page that does not exist are left out;
    both are reported, once, and the next call is clean."""
    _lib, _, rtp = _mods()
    c = Case(17, [64, 48, 80], 16, "bf16", ret=(True, True), max_seq_len=90)
    out, lse = c.decode(torch.tensor([64, -1, 91], dtype=torch.int32, device=DEV))
    assert c.status() == _lib.RTP_EDEVICE and c.status() == 0
    assert not _f64(out)[1:].any() and (_f64(lse)[1:] == -np.inf).all()
    c.check(out, lse, lens=[64, 0, 0])
    for wrong in (-1, c.n_pages, 0x7fffffff):
        c.bt[0, 2] = wrong                                     # rows 32..47 of sequence 0
        out, lse = c.decode()
        assert c.status() == _lib.RTP_EDEVICE
        keep = np.r_[0:32, 48:64]
        for h in range(c.Hq):
            c.agree(_f64(out)[0, h], _f64(lse)[0, h], 0, h, 64, keep)
    c.bt[0, :4] = -1                                           # nothing left: zeros
    out, lse = c.decode()
    assert c.status() == _lib.RTP_EDEVICE
    assert not _f64(out)[0].any() and (_f64(lse)[0] == -np.inf).all()
    c.bt.copy_(torch.from_numpy(c.table.astype(np.int32)))
    out, lse = c.decode()
    assert c.status() == 0
    c.check(out, lse)


def test_decode_without_lse_and_past_a_table_row():
    """lse is optional; a length beyond the table row is refused on the device."""
    _lib, _, rtp = _mods()
    c = Case(18, [30, 20], 16, "bf16", max_seq_len=1000)       # rows of 3 entries: 48 tokens
    out, lse = c.decode()
    out2 = torch.zeros_like(out)
    rtp.rtp_paged_decode_step(c.desc, c.cache, c.q, c.sl, out2, None, c.ws)
    assert torch.equal(out, out2)
    c.decode(torch.tensor([49, 20], dtype=torch.int32, device=DEV))
    assert c.status() == _lib.RTP_EDEVICE


def test_decode_graph_and_two_streams():
    """A captured step replayed with other lengths and queries; two workspaces on two streams at
    once; a workspace that served one description serves another."""
    _, _, rtp = _mods()
    c = Case(19, [3000, 900, 0, 17], 32, "bf16", window=128)
    d = Case(20, [5000], 64, "e4m3", G=8, Hkv=2)
    out, lse = c.outputs()
    lens = c.sl.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        rtp.rtp_paged_decode_step(c.desc, c.cache, c.q, lens, out, lse, c.ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        rtp.rtp_paged_decode_step(c.desc, c.cache, c.q, lens, out, lse, c.ws)
    for new in ([3000, 900, 0, 17], [1, 0, 0, 16], [2999, 450, 0, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            od, ld = d.decode()
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse, lens=new)
        d.check(od, ld)
    # a stream given by its address
    out2, lse2 = c.outputs()
    torch.cuda.synchronize()
    rtp.rtp_paged_decode_step(c.desc, c.cache, c.q, lens, out2, lse2, c.ws, s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # another shape on the same workspace
    ws = d.ws
    e = Case(21, [700, 650], 16, "bf16", G=2, Hkv=4, ret=(True, False, True, False))
    e.ws = ws
    for x in (e, d, e):
        o, l = x.decode()
        x.check(o, l)
    assert e.status() == 0 and c.status() == 0


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,n_new", [(16, 1), (64, 37), (256, 300)])
def test_append_rows(page, n_new, kv):
    """Ragged new tokens at near and far positions: stored rows against the 64-bit model; rows
    without a new token stay as they were."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(page + n_new)
    B, Hkv = 3, 5
    cnt = np.array([n_new, max(1, n_new // 3), 0])
    start = np.array([0, 131071, 1 << 20])
    table, n_pages = _table(rng, cnt, page)
    slots = np.full((B, n_new), -1)
    for b in range(B):
        j = np.arange(cnt[b])
        slots[b, :cnt[b]] = table[b, j // page] * page + j % page
    kp, vv = (bf16_round(rng.normal(size=(B, n_new, Hkv, 128))) for _ in range(2))
    kp[0, 0, 0] = 0.0
    vv[0, 0, 1] = 0.0
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    k, v = (torch.full((n_pages, Hkv, page, 128), 0x55, dtype=dt, device=DEV) for _ in range(2))
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (torch.full((n_pages, Hkv, page), 9.0, device=DEV) for _ in range(2))
    desc = rtp.LayerDesc(B, Hkv, Hkv, 0, 1, 1 << 24, rtp.rtp_build_slot_map([1] * Hkv)[0], BASE)
    cache = rtp.make_paged_cache(k, v, torch.zeros((B, 1), dtype=torch.int32, device=DEV), ks, vs)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_append_kv(desc, cache, _bf(kp), _bf(vv),
                            torch.from_numpy(start.astype(np.int32)).to(DEV),
                            torch.from_numpy(slots.astype(np.int32)).to(DEV), n_new, ws)
    assert rtp.rtp_read_device_status(ws) == 0
    touched = np.zeros((n_pages, page), bool)
    for name, x, got, sc in (("k", kp, k, ks), ("v", vv, v, vs)):
        raw = got.float().cpu().numpy() if kv == "bf16" else got.view(torch.float8_e4m3fn).float().cpu().numpy()
        scn = None if sc is None else sc.cpu().numpy()
        wrong = total = 0
        for b in range(B):
            for j in range(cnt[b]):
                pg, r = divmod(int(slots[b, j]), page)
                touched[pg, r] = True
                rows = x[b, j] if name == "v" else rope_rotate(x[b, j], start[b] + j, BASE)
                if kv == "bf16":
                    want = bf16_round(rows)
                else:
                    want, s = PO.e4m3_rows(rows)
                    # the amax may sit on a rounding border of the single-precision row
                    assert (np.abs(scn[pg, :, r] - s) <= 2.0 ** -23 * s).all()
                bad = raw[pg, :, r] != want
                wrong += bad.sum()
                total += bad.size
                # a value on a rounding border: one step off
                step = 2.0 ** -7 if kv == "bf16" else 2.0 ** -3
                assert (np.abs(raw[pg, :, r] - want) <= step * np.abs(want) + 2.0 ** -9)[bad].all()
        assert wrong <= 1e-6 * total, (name, wrong, total)
        left = ~touched
        assert (got.float().cpu().numpy().swapaxes(1, 2)[left] == 0x55).all()


def test_append_equals_contiguous_append_bit_for_bit():
    """The bf16 rows are those of rtp_append_kv."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(30)
    B, n, Hkv, page = 2, 200, 3, 32
    kp, vv = (_bf(rng.normal(size=(B, n, Hkv, 128))) for _ in range(2))
    start = torch.tensor([0, 7], dtype=torch.int32, device=DEV)
    lay = layer.DecodeLayer(B, Hkv, Hkv, 4, 64, 256, [1] * Hkv, [256, 256], DEV, BASE)
    wk = torch.zeros((Hkv, 128, 16), device=DEV)
    lay.append(kp, vv, wk, start)
    t = layer.PageTable(B, 40, page, 256)
    pl = layer.PagedLayer(t, Hkv, Hkv, 4, 64, 256, [1] * Hkv, rope_base=BASE)
    t.reserve(start)
    slots = torch.empty((B, n), dtype=torch.int32, device=DEV)
    t.reserve(start + n, slots)
    pl.append(kp, vv, start, slots)
    bt = t.block_table.cpu().numpy()
    for b in range(B):
        s0 = int(start[b])
        pos = np.arange(s0, s0 + n)
        pg = torch.from_numpy(bt[b, pos // page]).long().to(DEV)
        r = torch.from_numpy(pos % page).to(DEV)
        for g in range(Hkv):
            for mine, theirs in ((pl.k, lay.k_ret), (pl.v, lay.v_ret)):
                want = theirs[g, 256 * b + s0:256 * b + s0 + n]
                assert torch.equal(mine[pg, g, r].view(torch.int16), want.view(torch.int16))
    assert t.status() == 0 and pl.status() == 0


def test_append_skips_and_reports_bad_slots():
    _lib, _, rtp = _mods()
    page, n_pages = 16, 4
    k, v = (torch.zeros((n_pages, 1, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    desc = rtp.LayerDesc(2, 1, 1, 0, 1, 64, rtp.rtp_build_slot_map([1])[0], BASE)
    cache = rtp.make_paged_cache(k, v, torch.zeros((2, 1), dtype=torch.int32, device=DEV))
    x = torch.ones((2, 3, 1, 128), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    rtp.rtp_paged_append_kv(desc, cache, x, x, i32([0, 5]), i32([[-1, 63, -7], [0, -1, 1]]), 3, ws)
    assert rtp.rtp_read_device_status(ws) == 0
    assert sorted(v[..., 0].flatten().nonzero().flatten().tolist()) == [0, 1, 63]
    for start, slots in (([0, 0], [[64, 2, -1], [-1, -1, -1]]), ([0, -1], [[2, -1, -1], [3, -1, -1]])):
        v.zero_()
        rtp.rtp_paged_append_kv(desc, cache, x, x, i32(start), i32(slots), 3, ws)
        assert rtp.rtp_read_device_status(ws) == _lib.RTP_EDEVICE
        assert v[..., 0].flatten().nonzero().flatten().tolist() == [2]
    rtp.rtp_paged_append_kv(desc, cache, x, x, i32([0, 0]), i32([[64, 2, -1], [-1, -1, -1]]), 3)  # no ws


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 128])
def test_fused_append_equals_append_then_decode(page, kv):
    """Outputs, pages and scales of the fused call, bit for bit; at tile and page borders, with an
    idle place; the rest of the pool untouched (NaN included)."""
    _, _, rtp = _mods()
    c = Case(40 + page, [1, 16, 17, 0, 128, 129, 2500], page, kv, window=50)
    kn, vn = (_bf(c.rng.normal(size=(c.B, c.Hkv, 128))) for _ in range(2))
    slots = [-1 if n == 0 else int(c.table[b, (n - 1) // page]) * page + (n - 1) % page
             for b, n in enumerate(c.lens)]
    first = [x.clone() for x in (c.k, c.v)] + [None if x is None else x.clone() for x in (c.k_scale, c.v_scale)]
    rtp.rtp_paged_append_kv(c.desc, c.cache, kn[:, None].contiguous(), vn[:, None].contiguous(), c.sl - 1,
                            torch.tensor(slots, dtype=torch.int32, device=DEV), 1, c.ws)
    out, lse = c.decode()
    assert c.status() == 0
    after = [x if x is None else x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), first):
        if x is not None:
            x.view(torch.uint8).copy_(y.view(torch.uint8))
    out2, lse2 = c.outputs()
    rtp.rtp_paged_decode_step_append(c.desc, c.cache, kn, vn, c.q, c.sl, out2, lse2, c.ws)
    assert c.status() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), after):
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # and against the model: the last row replaced
    for b, n in enumerate(c.lens):
        for g in range(c.Hkv):
            if n:
                for name, new in (("k", rope_rotate(_f64(kn)[b, g], n - 1, BASE)), ("v", _f64(vn)[b, g])):
                    x = c.rows[name][b, g].copy()
                    x[-1] = PO.stored_rows(new, kv)
                    c.rows[name][b, g] = x
    c.check(out2, lse2)


def test_fused_append_on_a_page_that_does_not_exist():
    _lib, _, rtp = _mods()
    c = Case(50, [17, 20], 16, "bf16")
    c.bt[0, 1] = c.n_pages
    before = c.k.view(torch.int16).clone()
    kn, vn = (_bf(c.rng.normal(size=(2, 2, 128))) for _ in range(2))
    out, lse = c.outputs()
    rtp.rtp_paged_decode_step_append(c.desc, c.cache, kn, vn, c.q, c.sl, out, lse, c.ws)
    assert c.status() == _lib.RTP_EDEVICE
    changed = (c.k.view(torch.int16) != before).any(-1).nonzero().tolist()
    assert sorted(changed) == [[int(c.table[1, 1]), 0, 3], [int(c.table[1, 1]), 1, 3]]


# ------------------------------------------------------------------ reservation

def _reserve(rtp, page, n_pages, table, free, lens, new, counters, n_new, inplace):
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).to(DEV)
    t, f = i32(table), i32(free)
    pool = rtp.make_page_pool(f, t, page)
    l0, l1, c0 = i32(lens), i32(new), torch.from_numpy(np.asarray(counters, np.int64)).to(DEV)
    lo, co = (l0, c0) if inplace else (torch.zeros_like(l0), torch.zeros_like(c0))
    B = len(lens)
    slots = torch.full((B, n_new), 77, dtype=torch.int32, device=DEV)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    for _ in range(1 if inplace else 2):               # repeatable while its inputs stay
        rtp.rtp_paged_reserve(pool, l0, l1, c0, lo, co, slots if n_new else None, n_new, ws)
    st = rtp.rtp_read_device_status(ws)
    assert not ws.any()                                # the arrival counter is back at zero
    return dict(table=t.cpu().numpy(), free=f.cpu().numpy(), lens=lo.cpu().numpy(),
                counters=co.cpu().numpy(), slots=slots.cpu().numpy(), error=st != 0)


def _same(a, b):
    for k in ("table", "free", "lens", "counters", "slots"):
        assert np.array_equal(a[k], b[k]), k
    assert a["error"] == b["error"]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,page,stride,n_pages,n_new", [
    (1, 16, 1, 1, 1), (1, 16, 300, 301, 4800), (3, 64, 5, 11, 0), (33, 32, 7, 150, 9),
    (64, 16, 300, 9000, 1), (600, 16, 40, 12000, 2), (5, 16, 3, 9, 4), (512, 32, 3, 900, 4),
    (513, 16, 9, 2500, 5), (4096, 16, 4, 9000, 3), (64, 256, 17, 700, 4097)])
def test_reserve_random_rounds(B, page, stride, n_pages, n_new, inplace):
    """Rounds of starting, growing, shrinking and ending sequences, pages running out, the ring
    going round, at small and huge counters: all outputs equal the model's."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(B + stride)
    table, free = np.full((B, stride), -1), rng.permutation(n_pages)
    lens = np.zeros(B, int)
    h = int(rng.integers(0, 1 << 45)) // n_pages * n_pages
    counters = np.array([h, h + n_pages])
    for r in range(6):
        new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, stride * page + 1, B))
        new = np.where(rng.random(B) < 0.3, np.minimum(lens + 1, stride * page), new)
        want = PO.reserve(page, n_pages, table, free, lens, new, counters, n_new)
        _same(_reserve(rtp, page, n_pages, table, free, lens, new, counters, n_new, inplace), want)
        table, free, lens, counters = want["table"], want["free"], want["lens"], want["counters"]


def test_reserve_into_the_wished_lengths():
    """lens_out may be new_lens."""
    _, _, rtp = _mods()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    lens, new, ctr = i32([0, 5, 40]), i32([33, 6, 0]), torch.tensor([0, 3], device=DEV)
    table, free = i32([[9, 9, 9], [5, 9, 9], [3, 4, 6]]), i32([0, 1, 2, 9, 9, 9, 9])
    slots, ws = i32([[0], [0], [0]]), torch.zeros(4096, dtype=torch.uint8, device=DEV)
    rtp.rtp_paged_reserve(rtp.make_page_pool(free, table, 16), lens, new, ctr, new, ctr, slots, 1, ws)
    assert new.tolist() == [33, 6, 0] and lens.tolist() == [0, 5, 40] and ctr.tolist() == [3, 6]
    assert table.tolist() == [[0, 1, 2], [5, 9, 9], [3, 4, 6]]
    assert free.tolist() == [0, 1, 2, 3, 4, 6, 9] and slots.tolist() == [[0], [85], [-1]]
    assert rtp.rtp_read_device_status(ws) == 0 and rtp.rtp_last_launch_count() == 1


def test_reserve_reports_bad_lengths_and_counters():
    _, _, rtp = _mods()
    page, n_pages = 16, 8
    table = np.array([[0, 1, 7], [2, 7, 7], [7, 7, 7], [7, 7, 7]])
    free = np.array([3, 4, 5, 6, 7, -1, -1, -1])
    for lens, new, counters in (
            ([20, 5, 0, 0], [49, 6, 16, -1], [0, 5]),             # too long, negative
            ([20, -5, 0, 99], [21, 6, 16, 3], [0, 5]),
            ([20, 5, 0, 0], [40, 6, 1, 0], [5, 0]),               # tail before head
            ([20, 5, 0, 0], [40, 6, 1, 0], [-1, 4]),
            ([20, 5, 0, 0], [40, 6, 1, 0], [0, 9]),               # more free pages than pages
            ([20, 5, 0, 0], [0, 0, 1, 0], [0, 6]),                # and with those returned
            ([20, 5, 0, 0], [40, 40, 40, 40], [0, 5])):           # runs out: no error
        want = PO.reserve(page, n_pages, table, free, lens, new, counters, 3)
        _same(_reserve(rtp, page, n_pages, table, free, lens, new, counters, 3, False), want)
        _same(_reserve(rtp, page, n_pages, table, free, lens, new, counters, 3, True), want)


def test_reserve_more_than_counts_hold():
    """Wishes whose sum passes 2^31 pages: nobody after the first overrun is served."""
    _, _, rtp = _mods()
    B, page, stride, n_pages = 1025, 16, 1 << 21, 50
    lens, new = np.zeros(B, int), np.full(B, stride * page)
    new[0], new[-1] = 33, 1
    t = torch.full((B, stride), -1, dtype=torch.int32, device=DEV)            # 8.6 GB
    f = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    pool = rtp.make_page_pool(f, t, page)
    l0, l1 = (torch.from_numpy(x.astype(np.int32)).to(DEV) for x in (lens, new))
    c = torch.tensor([0, n_pages], dtype=torch.int64, device=DEV)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    slots = torch.empty((B, 2), dtype=torch.int32, device=DEV)
    rtp.rtp_paged_reserve(pool, l0, l1, c, l0, c, slots, 2, ws)
    assert rtp.rtp_read_device_status(ws) == 0
    assert l0.nonzero().flatten().tolist() == [0] and int(l0[0]) == 33 and c.tolist() == [3, 50]
    assert t[0, :4].tolist() == [0, 1, 2, -1] and (slots[1:] == -1).all() and slots[0].tolist() == [0, 1]


# ------------------------------------------------------------------ together

def test_serving_run_against_the_contiguous_layer():
    """Prompts, steps, an ending and a starting sequence through PageTable and two PagedLayers; a
    step's outputs against DecodeLayer at p = 1 over the same tokens (dense retrieval heads, the
    same local heads), both in bf16."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(60)
    B, Hq, Hkv, sinks, window, cap, page = 3, 8, 2, 4, 32, 256, 16
    ret = [1, 0]
    t = layer.PageTable(B, 40, page, cap)
    layers = [layer.PagedLayer(t, Hq, Hkv, sinks, window, cap, ret, dt, BASE)
              for dt in (torch.bfloat16, torch.float8_e4m3fn)]
    ref = layer.DecodeLayer(B, Hq, Hkv, sinks, window, cap, ret, [cap] * B, DEV, BASE)
    wk = torch.from_numpy(rng.normal(size=(Hkv, 128, 16)).astype(np.float32)).to(DEV)
    wq = torch.from_numpy(rng.normal(size=(Hq, 128, 16)).astype(np.float32)).to(DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    n_b, n_max = i32([100, 37, 1]), 100
    q, k, v = (_bf(rng.normal(size=(B, n_max, h, 128))) for h in (Hq, Hkv, Hkv))
    slots = torch.empty((B, n_max), dtype=torch.int32, device=DEV)
    t.reserve(n_b, slots)
    assert t.lens.tolist() == [100, 37, 1]
    out = torch.zeros_like(q)
    want = torch.zeros_like(q)
    ref.prefill(q, k, v, wk, n_b, want)
    for pl in layers:
        pl.prefill(q, k, v, n_b, slots, out)
        for b, n in enumerate(n_b.tolist()):
            assert torch.equal(out[b, :n], want[b, :n])        # the same prefill kernel
    lens = t.lens.clone()
    for step in range(40):
        if step == 20:                                         # 1 ends; its pages serve others
            lens[1] = 0
            t.reserve(lens)
        grow = (lens > 0).to(torch.int32)
        if step >= 20:
            grow[1] = 0
        lens = lens + grow
        t.reserve(lens)
        assert torch.equal(t.lens, lens)
        qs, ks, vs = (_bf(rng.normal(size=(B, h, 128))) for h in (Hq, Hkv, Hkv))
        outs = []
        for pl in layers:
            o = torch.zeros((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
            pl.decode_append(ks, vs, qs, t.lens, o)
            outs.append(_f64(o))
        live = [b for b in range(B) if lens[b] > 0]
        w = torch.zeros((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
        cnt = torch.zeros((B, Hq), dtype=torch.int32, device=DEV)
        ref.decode_append(ks, vs, wk, qs, wq, torch.clamp(lens, min=1), 1.0, w, cnt)
        # both outputs are bf16 roundings of the same sum, whose weights are off by 2^-12 at most
        # in the contiguous step (fp16 partials): half a step each, 2^-8 |o|, and 2^-11 max|v|
        d = np.abs(outs[0] - _f64(w))[live]
        assert (d <= 2 * 2.0 ** -8 * np.abs(_f64(w)[live]) + 2.0 ** -11 * 5).all(), d.max()
        # 8 bits: values off by 2^-4 relative, logits by 2^-4 of at most 12: a factor of
        # exp(1.5) in the worst case; checked against the model elsewhere, here for sanity
        assert np.isfinite(outs[1]).all()
    assert t.status() == 0 and all(pl.status() == 0 for pl in layers) and ref.status() == 0
    free = [int(t.free_pages[i % 40]) for i in range(*t.counters.tolist())]
    held = [int(t.block_table[b, j]) for b in range(B) for j in range(-(-int(lens[b]) // page))]
    assert sorted(free + held) == list(range(40))


def test_serving_step_in_one_graph():
    """Reservation and the fused step captured together and replayed: lengths and counters are
    updated in place, pages are taken inside the graph."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(61)
    B, Hq, Hkv, page, cap = 4, 4, 2, 16, 128
    t = layer.PageTable(B, 40, page, cap)
    pl = layer.PagedLayer(t, Hq, Hkv, 2, 20, cap, [1, 0], rope_base=BASE)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    q, k, v = (torch.zeros((B, h, 128), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    out = torch.zeros_like(q)
    lse = torch.zeros((B, Hq), device=DEV)
    c = Case.__new__(Case)                          # the model's side of it
    c.G, c.ret, c.sinks, c.window = 2, [True, False], 2, 20

    def step():
        torch.add(t.lens, 1, out=new)
        t.reserve(new)
        pl.decode_append(k, v, q, t.lens, out, lse)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    # start again from nothing
    t.lens.zero_()
    t.counters.copy_(torch.tensor([0, 40]))
    t.free_pages.copy_(torch.arange(40, dtype=torch.int32))
    K, V = [], []
    for i in range(40):
        for x in (q, k, v):
            x.copy_(_bf(rng.normal(size=x.shape)))
        g.replay()
        K.append(rope_rotate(_f64(k), i, BASE))
        V.append(_f64(v))
        o, l = _f64(out), _f64(lse)
        c.q64 = _f64(q)
        c.rows = {"k": {(b, g): bf16_round(np.stack([x[b, g] for x in K])) for b in range(B) for g in range(Hkv)},
                  "v": {(b, g): np.stack([x[b, g] for x in V]) for b in range(B) for g in range(Hkv)}}
        for b in range(B):
            for h in range(Hq):
                c.agree(o[b, h], l[b, h], b, h, i + 1)
    assert t.lens.tolist() == [40] * B and t.counters.tolist() == [12, 40]
    assert t.status() == 0 and pl.status() == 0


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("how", ["stream", "graph", "branches"])
def test_launches_wait_for_those_before_them(how, kv):
    """A run of reservations, appends and steps that each read what the launch before wrote, in
    buffers that are overwritten between them by kernels, copies and fills: queued without a pause,
    captured into a graph, and on two streams joined by events. The same bits as with the GPU
    waited for after every call."""
    _, layer, rtp = _mods()
    rng = np.random.default_rng(62)
    B, Hq, Hkv, page, cap, n, steps = 5, 8, 2, 16, 2048, 900, 24
    qs, ks, vs = (_bf(rng.normal(size=(steps, B, h, 128))) for h in (Hq, Hkv, Hkv))
    kp, vp = (_bf(rng.normal(size=(B, n, Hkv, 128))) for _ in range(2))
    prompt = torch.tensor([900, 1, 0, 333, 64], dtype=torch.int32, device=DEV)
    start = torch.zeros(B, dtype=torch.int32, device=DEV)

    def run(pause, side=None, captured=False):
        t = layer.PageTable(B, 400, page, cap)
        pl = layer.PagedLayer(t, Hq, Hkv, 2, 100, cap, [1, 0], kv, BASE)
        new, slots = torch.zeros_like(prompt), torch.zeros((B, n), dtype=torch.int32, device=DEV)
        q, k, v = (torch.zeros_like(x[0]) for x in (qs, ks, vs))
        out = torch.zeros_like(q)
        outs = torch.zeros_like(qs)

        def work():
            rtp.rtp_paged_workspace_init(pl.ws)              # (a fill before a launch)
            new.copy_(prompt)                                # (a copy before a launch)
            t.reserve(new, slots); pause()
            pl.append(kp, vp, start, slots); pause()
            slots.fill_(-7)                                  # read by the launch before
            for i in range(steps):
                q.copy_(qs[i]); k.copy_(ks[i]); v.copy_(vs[i])
                torch.add(t.lens, 1, out=new)
                t.reserve(new); pause()
                if side is None:
                    pl.decode_append(k, v, q, t.lens, out); pause()
                    outs[i].copy_(out)
                else:                                        # the step on another stream
                    main = torch.cuda.current_stream()
                    side.wait_stream(main)
                    with torch.cuda.stream(side):
                        pl.decode_append(k, v, q, t.lens, out)
                        outs[i].copy_(out)
                    main.wait_stream(side)
                out.zero_()

        torch.cuda.synchronize()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                work()
            for _ in range(2):                               # twice from the same start
                t.lens.zero_()
                t.counters.copy_(torch.tensor([0, 400]))
                t.free_pages.copy_(torch.arange(400, dtype=torch.int32))
                outs.zero_()
                g.replay()
        else:
            work()
        torch.cuda.synchronize()
        assert t.status() == 0 and pl.status() == 0
        return outs, t.lens.clone(), t.counters.clone()

    run(torch.cuda.synchronize)                              # (loads every kernel)
    want = run(torch.cuda.synchronize)
    for captured in ([False, True] if how == "branches" else [how == "graph"]):
        got = run(lambda: None, torch.cuda.Stream() if how == "branches" else None, captured)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_append_e4m3_rows_of_extreme_size():
    """Rows near both ends of the range, zeros, infinities and NaN at position 0 (where the rotation
    changes no finite value): scale and bytes are those of the definition in single precision."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(63)
    B, Hkv, n, page = 1, 3, 64, 64
    sizes = np.exp2(np.concatenate([np.arange(-133, -101), np.arange(96, 128)]))[:n]
    with np.errstate(over="ignore"):
        x = np.clip(rng.normal(size=(2, B, n, Hkv, 128)) * sizes[None, None, :, None, None],
                    -3.3e38, 3.3e38)
    x[:, 0, 5] = 0.0
    x[1, 0, 6, 0, 3], x[1, 0, 6, 1, 127], x[1, 0, 7, 2, 64] = np.inf, -np.inf, np.nan
    kv = [torch.from_numpy(a).to(DEV, torch.bfloat16) for a in x]
    kv = [a.reshape(n, 1, Hkv, 128).contiguous() for a in kv]
    k, v = (torch.zeros((1, Hkv, page, 128), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((1, Hkv, page), device=DEV) for _ in range(2))
    desc = rtp.LayerDesc(n, Hkv, Hkv, 0, 1, 1 << 24, rtp.rtp_build_slot_map([1] * Hkv)[0], BASE)
    cache = rtp.make_paged_cache(k, v, torch.zeros((n, 1), dtype=torch.int32, device=DEV), ks, vs)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV).reshape(n, 1)
    rtp.rtp_paged_append_kv(desc, cache, kv[0], kv[1], torch.zeros(n, dtype=torch.int32, device=DEV), slots,
                            1, ws)  # each token the first of a sequence
    assert rtp.rtp_read_device_status(ws) == 0
    for rows, got, sc in ((kv[0], k, ks), (kv[1], v, vs)):
        w = rows[:, 0].float().cpu().numpy().swapaxes(0, 1)        # [Hkv][n][128]
        amax = np.fmax.reduce(np.abs(w), axis=-1, initial=0.0).astype(np.float32)
        scale = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))
        assert np.array_equal(sc[0].cpu().numpy(), scale)
        with np.errstate(invalid="ignore"):
            q = w / scale[..., None]
        want = np.where(np.isnan(q), np.nan, PO.e4m3_round(np.nan_to_num(q.astype(np.float64))))
        assert np.array_equal(got[0].float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("Hkv", [1, 3, 4, 5, 8, 9, 13])
@pytest.mark.parametrize("B,n_new", [(7, 16), (3, 701), (5, 1003), (9, 801)])
def test_append_is_the_same_however_it_is_cut(Hkv, B, n_new):
    """Calls of sizes that share a sine among one, two or four tokens, whose blocks of tokens end
    inside a sequence and cross into the next, against the formula in 64 bits: turning
    an angle on by products in double moves it by less than 2^-48, so all but roundings within that
    of a border are the same."""
    _, _, rtp = _mods()
    rng = np.random.default_rng(Hkv * 1000 + n_new)
    page, start = 64, 1000
    per = -(-n_new // page)
    ids = rng.permutation(B * per)
    j = np.arange(n_new)
    slots = np.stack([ids[b * per + j // page] * page + j % page for b in range(B)])
    slots[0, 3] = -1
    kp, vp = (_bf(rng.normal(size=(B, n_new, Hkv, 128))) for _ in range(2))
    k, v = (torch.full((B * per, Hkv, page, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ret = [1] * Hkv
    desc = rtp.LayerDesc(B, Hkv, Hkv, 0, 1, 1 << 24, rtp.rtp_build_slot_map(ret)[0], BASE)
    cache = rtp.make_paged_cache(k, v, torch.zeros((B, 1), dtype=torch.int32, device=DEV))
    pos = torch.full((B,), start, dtype=torch.int32, device=DEV)
    rtp.rtp_paged_append_kv(desc, cache, kp, vp, pos, torch.from_numpy(slots.astype(np.int32)).to(DEV), n_new)
    th = BASE ** (-np.arange(64) / 64.0)
    a = (start + j)[:, None, None] * th
    x = kp.double().cpu().numpy()
    want = np.concatenate([x[..., :64] * np.cos(a) - x[..., 64:] * np.sin(a),
                           x[..., :64] * np.sin(a) + x[..., 64:] * np.cos(a)], -1)
    got_k, got_v = k.float().cpu().numpy(), v.float().cpu().numpy()
    for b in range(B):
        keep = slots[b] >= 0
        pg, r = slots[b, keep] // page, slots[b, keep] % page
        gk = got_k[pg, :, r]
        bad = gk != bf16_round(want[b, keep])
        assert bad.sum() <= 1e-6 * bad.size + 1
        # half a bf16 step, and the angles' error on either side
        assert (np.abs(gk - want[b, keep]) <= 2.0 ** -8 * np.abs(want[b, keep]) + 2.0 ** -40).all()
        assert np.array_equal(got_v[pg, :, r], vp[b].float().cpu().numpy()[keep])
    touched = np.zeros((B * per, page), bool)
    touched.reshape(-1)[slots[slots >= 0]] = True
    assert (got_k.swapaxes(1, 2)[~touched] == 7.0).all() and (got_v.swapaxes(1, 2)[~touched] == 7.0).all()
