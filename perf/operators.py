"""Cases that measure the paged-cache operators: page reservation (block tables and slot maps), the
append of new tokens into pages, and the decode step of one layer over a paged cache.

``run`` computes an operator either in its plain form (elementary torch operations, 32-bit floats,
64-bit angles) or, with ``own`` set, through the package's entry points.

Layouts: K and V pages are [n_pages][Hkv][page][128] in bf16, or e4m3 bytes with one float scale per
row in [n_pages][Hkv][page]. Row r of page i holds position j * page + r of the sequence whose
block-table entry j is i. KV heads are retrieval heads (attend to every position) or local heads
(attention sinks plus a sliding window). Free pages form a ring read at ``counters[0]`` and
written at ``counters[1]`` (both only ever grow; entries are at the counter modulo the ring's size).
"""
import math

import numpy as np
import torch

own = False

D = 128
ROPE_BASE = 1e6
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # decode steps: one token per sequence against its cached context
        # one small layer, one dense and one local KV head: the latency of a single call
        dict(name="step-4k-append", op="decode", append=True, B=1, Hq=4, Hkv=2, n_ret=1, sinks=4,
             window=256, lo=4096, hi=4096, page=16, kv="bf16", idle=0),
        # an 8B-model layer at 32K: one dense head, the others sinks + window
        dict(name="step-32k", op="decode", append=False, B=1, Hq=32, Hkv=8, n_ret=1, sinks=4,
             window=2048, lo=32768, hi=32768, page=64, kv="bf16", idle=0),
        # the same layer with every head dense, 128K x 4, 8-bit cache
        dict(name="step-128k-x4-e4m3", op="decode", append=False, B=4, Hq=32, Hkv=8, n_ret=8,
             sinks=4, window=2048, lo=131072, hi=131072, page=64, kv="e4m3", idle=0),
        # one sequence of a million tokens, every head dense: the longest stream
        dict(name="step-1m", op="decode", append=False, B=1, Hq=32, Hkv=8, n_ret=8, sinks=4,
             window=2048, lo=1048576, hi=1048576, page=128, kv="bf16", idle=0),
        # a serving batch of unequal contexts, small pages, 8-bit cache, dense and local heads
        dict(name="step-ragged-64-e4m3", op="decode", append=False, B=64, Hq=32, Hkv=8, n_ret=2,
             sinks=4, window=2048, lo=8192, hi=65536, page=16, kv="e4m3", idle=0),
        # many short chats, 8 query heads per KV head, some batch slots idle, fused append
        dict(name="step-short-256-append", op="decode", append=True, B=256, Hq=64, Hkv=8, n_ret=8,
             sinks=4, window=2048, lo=1, hi=1024, page=32, kv="bf16", idle=16),
        # appends: new tokens into the slots that the reservation handed out
        # the token of a decode step
        dict(name="append-token-64", op="append", B=64, Hkv=8, n_new=1, short=1, start=65535,
             page=16, kv="bf16"),
        # one whole prompt
        dict(name="append-32k", op="append", B=1, Hkv=8, n_new=32768, short=32768, start=0,
             page=64, kv="bf16"),
        # unequal prompt chunks at far positions into an 8-bit cache
        dict(name="append-ragged-8-e4m3", op="append", B=8, Hkv=8, n_new=4095, short=1,
             start=1000000, page=32, kv="e4m3"),
        # reservations: one per step for all layers of a model
        # a decode step of 64 sequences
        dict(name="reserve-step-64", op="reserve", B=64, lo=8192, hi=65536, grow=1, fresh=0.0,
             gone=0.0, n_new=1, page=16, spare=1.0),
        # 64 new prompts of 8K-64K tokens
        dict(name="reserve-prompts-64", op="reserve", B=64, lo=8192, hi=65536, grow=65536,
             fresh=1.0, gone=0.0, n_new=65536, page=16, spare=1.0),
        # a large batch in which sequences end, start and grow while the pool runs out
        dict(name="reserve-turnover-4096", op="reserve", B=4096, lo=1, hi=2048, grow=64,
             fresh=0.05, gone=0.05, n_new=64, page=16, spare=0.5),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "reserve"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 8])
        n_ret = rng.randint(0, Hkv)
        hi = _log(rng, 1, 1 << 20)
        # at most the rows of the largest listed cases: dense rows, and rows held
        B = _log(rng, 1, max(1, min(512, (8 << 20) // (hi * max(n_ret, 1)), (32 << 20) // (hi * Hkv))))
        append = rng.random() < 0.5 and B * hi * Hkv <= 4 << 20
        return dict(op="decode", append=append, B=B, Hq=G * Hkv, Hkv=Hkv, n_ret=n_ret,
                    sinks=rng.choice([0, 1, 4, 17]), window=_log(rng, 1, 4096),
                    lo=rng.randint(1, hi), hi=hi, page=page, kv=rng.choice(["bf16", "e4m3"]),
                    idle=rng.randint(0, B // 4))
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        n_new = _log(rng, 1, 32768)
        B = _log(rng, 1, max(1, min(256, 32768 // n_new)))
        return dict(op="append", B=B, Hkv=Hkv, n_new=n_new, short=rng.randint(1, n_new),
                    start=_log(rng, 1, 1 << 20) - 1, page=page, kv=rng.choice(["bf16", "e4m3"]))
    B = _log(rng, 1, 4096)
    hi = _log(rng, 1, max(1, min(65536, (4 << 20) // B)))
    n_new = _log(rng, 1, hi)
    return dict(op="reserve", B=B, lo=rng.randint(1, hi), hi=hi, grow=n_new,
                fresh=rng.choice([0.0, 0.1, 1.0]), gone=rng.choice([0.0, 0.1]), n_new=n_new,
                page=page, spare=rng.choice([0.3, 1.0]))


# --------------------------------------------------------------------------------------- inputs

def _is_ret(Hkv, n_ret):
    """Which KV heads are retrieval heads: n_ret of them, spread over the layer."""
    return [(g * n_ret) % Hkv < n_ret for g in range(Hkv)]


def _lens(case, seed):
    """Context lengths of the sequences, the case's own in the seed's order; `idle` batch slots
    hold none."""
    lens = np.random.default_rng(1).integers(case["lo"], case["hi"] + 1, case["B"])
    lens[:case["idle"]] = 0
    return np.random.default_rng([seed, 1]).permutation(lens)


def _tables(lens, page, rng, spare=8):
    """Block tables of sequences of these lengths over a shuffled pool."""
    need = -(-lens // page)
    n_pages = int(need.sum()) + spare
    pages = rng.permutation(n_pages).astype(np.int32)
    stride = max(1, int(need.max()))
    col = np.arange(stride)
    first = np.concatenate([[0], np.cumsum(need)[:-1]])
    at = np.minimum(first[:, None] + col, n_pages - 1)
    table = np.where(col < need[:, None], pages[at], 0).astype(np.int32)
    return table, n_pages


def _pages(gen, shape, kv):
    """Random cache rows as the append leaves them."""
    x = torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=gen)
    return (x, None) if kv == "bf16" else _quantise(x.float())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, 2])
    s = dict(case=case)
    page = case["page"]

    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    if case["op"] == "reserve":
        r = _reserve_inputs(case, seed)
        for k in ("lens", "new_lens", "table", "free", "counters"):
            s[k] = dev(r[k])
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["counters_out"] = torch.zeros_like(s["counters"])
        s["slots"] = torch.full((case["B"], case["n_new"]), -1, dtype=torch.int32, device="cuda")
        return s

    B, Hkv = case["B"], case["Hkv"]
    if case["op"] == "append":
        n_new = case["n_new"]
        lens = np.random.default_rng(1).integers(case["short"], n_new + 1, B)
        lens[0] = n_new
        lens = rng.permutation(lens)
        # the slots of whole pages in shuffled order; tokens past a sequence's end have none
        table, n_pages = _tables(lens, page, rng)
        j = np.arange(n_new)
        slots = np.where(j < lens[:, None],
                         table[np.arange(B)[:, None], np.minimum(j // page, table.shape[1] - 1)]
                         * page + j % page, -1)
        s["slots"] = dev(slots.astype(np.int32))
        s["start"] = dev(rng.integers(0, case["start"] + 1, B).astype(np.int32))
        s["k_pre"] = torch.randn((B, n_new, Hkv, D), dtype=torch.bfloat16, device="cuda", generator=gen)
        s["v_new"] = torch.randn((B, n_new, Hkv, D), dtype=torch.bfloat16, device="cuda", generator=gen)
        s["table"] = dev(table)
    else:
        lens = _lens(case, seed)
        table, n_pages = _tables(lens, page, rng)
        s["table"], s["lens"] = dev(table), dev(lens.astype(np.int32))
        # logits of standard deviation 2: peaked rows that are not one-hot
        q = torch.randn((B, case["Hq"], D), dtype=torch.float32, device="cuda", generator=gen)
        s["q"] = (2.0 * q).to(torch.bfloat16)
        s["out"] = torch.zeros((B, case["Hq"], D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((B, case["Hq"]), dtype=torch.float32, device="cuda")
        if case["append"]:
            s["k_pre"] = torch.randn((B, Hkv, D), dtype=torch.bfloat16, device="cuda", generator=gen)
            s["v_new"] = torch.randn((B, Hkv, D), dtype=torch.bfloat16, device="cuda", generator=gen)
    shape = (n_pages, Hkv, page, D)
    s["k"], s["k_scale"] = _pages(gen, shape, case["kv"])
    s["v"], s["v_scale"] = _pages(gen, shape, case["kv"])
    return s


def _reserve_inputs(case, seed):
    """Lengths, wished lengths, tables, the ring of free pages and its counters (host arrays).
    The lengths are the case's own, in the seed's order."""
    rng = np.random.default_rng(1)
    B, page = case["B"], case["page"]
    lens = rng.integers(case["lo"], case["hi"] + 1, B)
    new = lens + rng.integers(1, case["grow"] + 1, B)
    fresh = rng.random(B) < case["fresh"]             # sequences that start: nothing held yet
    new = np.where(fresh, lens, new)
    lens = np.where(fresh, 0, lens)
    gone = rng.random(B) < case["gone"]               # sequences that end
    new = np.where(gone, 0, new)
    rng = np.random.default_rng([seed, 3])
    order = rng.permutation(B)
    lens, new = lens[order], new[order]
    held = -(-lens // page)
    need = np.maximum(-(-new // page) - held, 0)
    free_n = int(need.sum() * case["spare"]) + 1      # spare < 1: not everybody is served
    n_pages = int(held.sum()) + free_n
    pages = rng.permutation(n_pages).astype(np.int32)
    stride = int(max((-(-lens // page)).max(), (-(-new // page)).max(), 1))
    col = np.arange(stride)
    first = np.concatenate([[0], np.cumsum(held)[:-1]])
    table = np.where(col < held[:, None], pages[np.minimum(first[:, None] + col, n_pages - 1)], -1)
    head = int(rng.integers(0, 1 << 40))
    ring = np.full(n_pages, -1, np.int32)
    ring[(head + np.arange(free_n)) % n_pages] = pages[n_pages - free_n:]
    return dict(lens=lens.astype(np.int32), new_lens=new.astype(np.int32),
                table=table.astype(np.int32), free=ring,
                counters=np.array([head, head + free_n], np.int64))


# ---------------------------------------------------------------------------------- plain forms

def _quantise(x):
    """Rows of 32-bit floats -> e4m3 values and a scale per row."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _rotate(x, pos):
    """R(pos) x in 64 bits; channels are paired (i, i + 64). pos broadcasts over x's leading axes."""
    i = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    a = pos.double()[..., None] * torch.exp(-math.log(ROPE_BASE) * 2.0 * i / D)
    c, s = torch.cos(a), torch.sin(a)
    u, w = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat([u * c - w * s, u * s + w * c], -1)


def _store(s, slots, k_rot, v):
    """Rows [n][Hkv][128] into the pages at `slots`."""
    ps = s["case"]["page"]
    at = (slots // ps)[:, None], torch.arange(k_rot.shape[1], device=k_rot.device), (slots % ps)[:, None]
    for name, x in (("k", k_rot.float()), ("v", v.float())):
        if s["case"]["kv"] == "bf16":
            s[name][at] = x.to(torch.bfloat16)
        else:
            x8, scale = _quantise(x)
            s[name].view(torch.uint8)[at] = x8.view(torch.uint8)
            s[name + "_scale"][at] = scale


def _rows(s, name, pos, heads):
    """Cache rows of positions [B][L] for some KV heads: [B][len(heads)][L][128] in 32 bits."""
    ps, table = s["case"]["page"], s["table"]
    p = pos.clamp(0, table.shape[1] * ps - 1)
    at = table.gather(1, p // ps).long()[:, None], heads[None, :, None], (p % ps)[:, None]
    if s["case"]["kv"] == "bf16":
        return s[name][at].float()
    x8 = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn)
    return x8.float() * s[name + "_scale"][at][..., None]


def _attend(s, q, pos, ok, heads):
    """Attention of the query heads of some KV heads over positions [B][L] where `ok`."""
    B, Hkv, G, _ = q.shape
    z = torch.matmul(q[:, heads], _rows(s, "k", pos, heads).transpose(-1, -2)) / math.sqrt(D)
    z = torch.where(ok[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = torch.where(ok[:, None, :, None], _rows(s, "v", pos, heads), 0.0)
    o = torch.where(l > 0, torch.matmul(p, v) / l, 0.0)
    s["out"].view(B, Hkv, G, D)[:, heads] = o.to(torch.bfloat16)
    s["lse"].view(B, Hkv, G)[:, heads] = (m + torch.log(l))[..., 0]


def _plain_decode(s):
    c = s["case"]
    B, Hkv, G = c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    n = s["lens"].long()[:, None]
    m = n[:, 0] - 1
    if c["append"]:
        live = torch.nonzero(m >= 0)[:, 0]
        page = s["table"][live].gather(1, m[live, None] // c["page"])[:, 0].long()
        _store(s, page * c["page"] + m[live] % c["page"],
               _rotate(s["k_pre"][live], m[live, None]), s["v_new"][live])
    q = _rotate(s["q"], m[:, None]).float().view(B, Hkv, G, D)
    is_ret = torch.tensor(_is_ret(Hkv, c["n_ret"]), device=q.device)
    ret, loc = torch.nonzero(is_ret)[:, 0], torch.nonzero(~is_ret)[:, 0]
    if c["n_ret"]:
        pos = torch.arange(s["table"].shape[1] * c["page"], device=q.device).expand(B, -1)
        _attend(s, q, pos, pos < n, ret)
    if c["n_ret"] < Hkv:
        sink = torch.arange(c["sinks"], device=q.device).expand(B, -1)
        win = n - 1 - torch.arange(c["window"], device=q.device)
        pos = torch.cat([sink, win], 1)
        ok = torch.cat([sink < torch.minimum(n, (n - c["window"]).clamp_min(0)), win >= 0], 1)
        _attend(s, q, pos, ok, loc)


def _plain_append(s):
    c = s["case"]
    b, j = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    pos = s["start"].long()[b] + j
    _store(s, s["slots"][b, j].long(), _rotate(s["k_pre"][b, j], pos[:, None]), s["v_new"][b, j])


def _plain_reserve(s):
    c = s["case"]
    page, n_pages = c["page"], s["free"].numel()
    lens, new = s["lens"].long(), s["new_lens"].long()
    head, tail = s["counters"][0], s["counters"][1]
    have, want = (lens + page - 1) // page, (new + page - 1) // page
    need = (want - have).clamp_min(0)
    upto = need.cumsum(0)
    granted = (need == 0) | (upto <= tail - head)
    # pages that are taken, then pages that are given back
    first = upto - need
    col = torch.arange(s["table"].shape[1], device=lens.device)
    take = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    at = (head + first[:, None] + col - have[:, None]) % n_pages
    s["table"].copy_(torch.where(take, s["free"][at], s["table"]))
    back = (have - want).clamp_min(0)
    b, j = torch.nonzero((col >= want[:, None]) & (col < have[:, None]), as_tuple=True)
    s["free"][(tail + (back.cumsum(0) - back)[b] + j - want[b]) % n_pages] = s["table"][b, j]
    s["lens_out"].copy_(torch.where(granted, new, lens))
    s["counters_out"][0] = head + torch.where(granted, need, 0).sum()
    s["counters_out"][1] = tail + back.sum()
    # slots of the new tokens
    pos = lens[:, None] + torch.arange(c["n_new"], device=lens.device)
    p = s["table"].gather(1, (pos // page).clamp_max(s["table"].shape[1] - 1))
    s["slots"].copy_(torch.where(pos < s["lens_out"][:, None], p * page + pos % page, -1))


# ---------------------------------------------------------------------- the package's operators

def _handle(s):
    """What a program keeps: the description, the cache struct and the workspace."""
    from long_context_sparse_rtpurbo_b200 import rtp
    c = s["case"]
    h = s["handle"] = dict(rtp=rtp)
    if c["op"] == "reserve":
        h["pool"] = rtp.make_page_pool(s["free"], s["table"], c["page"])
        size = rtp.RTP_PAGED_CTRL_BYTES
    else:
        Hq = c.get("Hq", c["Hkv"])
        slots = rtp.rtp_build_slot_map(_is_ret(c["Hkv"], c.get("n_ret", c["Hkv"])))[0]
        h["desc"] = rtp.LayerDesc(c["B"], Hq, c["Hkv"], c.get("sinks", 0), c.get("window", 1),
                                  c["hi"] if c["op"] == "decode" else 1 << 24, slots, ROPE_BASE)
        h["cache"] = rtp.make_paged_cache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
        size = rtp.rtp_paged_workspace_bytes(h["desc"])
    h["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    rtp.rtp_paged_workspace_init(h["ws"])
    return h


def _own_run(s):
    c = s["case"]
    h = s.get("handle") or _handle(s)
    rtp = h["rtp"]
    if c["op"] == "reserve":
        rtp.rtp_paged_reserve(h["pool"], s["lens"], s["new_lens"], s["counters"], s["lens_out"],
                              s["counters_out"], s["slots"], c["n_new"], h["ws"])
    elif c["op"] == "append":
        rtp.rtp_paged_append_kv(h["desc"], h["cache"], s["k_pre"], s["v_new"], s["start"],
                                s["slots"], c["n_new"], h["ws"])
    elif c["append"]:
        rtp.rtp_paged_decode_step_append(h["desc"], h["cache"], s["k_pre"], s["v_new"], s["q"],
                                         s["lens"], s["out"], s["lse"], h["ws"])
    else:
        rtp.rtp_paged_decode_step(h["desc"], h["cache"], s["q"], s["lens"], s["out"], s["lse"],
                                  h["ws"])


def run(state):
    c = state["case"]
    if own:
        _own_run(state)
    elif c["op"] == "reserve":
        _plain_reserve(state)
    elif c["op"] == "append":
        _plain_append(state)
    else:
        _plain_decode(state)
    if c["op"] == "reserve":
        return {k: state[k] for k in ("table", "free", "slots", "lens_out", "counters_out")}
    got = {}
    if c["op"] == "append" or c["append"]:
        got = {k: state[k] for k in ("k", "v", "k_scale", "v_scale")}
    if c["op"] == "decode":
        got |= {"out": state["out"], "lse": state["lse"]}
    return got


# ------------------------------------------------------------------------------------ work, exact

def work(case):
    if case["op"] == "reserve":
        r = _reserve_inputs(case, 0)
        page = case["page"]
        have, want = -(-r["lens"] // page), -(-r["new_lens"] // page)
        moved = int(np.abs(want - have).sum())        # ring to table, or table to ring
        return {"bytes": 12 * case["B"] + 32 + 8 * moved + 4 * case["B"] * case["n_new"], "flops": 0}
    row = 2 * D * 2 if case["kv"] == "bf16" else 2 * (D + 4)       # K and V of one token and head
    if case["op"] == "append":
        tokens = case["n_new"] + (case["B"] - 1) * (case["short"] + case["n_new"]) / 2
        return {"bytes": tokens * case["Hkv"] * (4 * D + row) + 4 * case["B"] * (case["n_new"] + 1),
                "flops": 3 * D * tokens * case["Hkv"]}
    n = _lens(case, 0).astype(np.float64)
    G = case["Hq"] // case["Hkv"]
    rows = case["n_ret"] * n.sum() + (case["Hkv"] - case["n_ret"]) * np.minimum(
        n, case["sinks"] + case["window"]).sum()
    table = 4 * np.ceil(n / case["page"]).sum()
    io = case["B"] * (case["Hq"] * (4 * D + 4) + 4)
    if case["append"]:
        io += (n > 0).sum() * case["Hkv"] * (4 * D + row)
    return {"bytes": float(rows * row + table + io), "flops": float(4 * D * G * rows)}


def exact(case, seed):
    if case["op"] == "reserve":
        return None                                   # whole numbers: the plain form's are exact
    s = prepare(case, seed)
    page, Hkv, B = case["page"], case["Hkv"], case["B"]
    inv = torch.tensor([ROPE_BASE ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64,
                       device="cuda")

    def turned(x, p):
        """x [..., 128] in 64 bits as complex numbers, turned by the angles of position p [...]."""
        z = torch.complex(x[..., :64].double(), x[..., 64:].double())
        ang = p.double()[..., None] * inv
        z = z * torch.complex(torch.cos(ang), torch.sin(ang))
        return torch.cat([z.real, z.imag], -1)

    # the new rows, as real numbers (a cache holds them rounded)
    updates = {}
    if case["op"] == "append":
        b, j = torch.nonzero(s["slots"] >= 0, as_tuple=True)
        slot = s["slots"][b, j].long()
        updates["k"] = turned(s["k_pre"][b, j], (s["start"][b].long() + j)[:, None].expand(-1, Hkv))
        updates["v"] = s["v_new"][b, j].double()
    elif case["append"]:
        lens = s["lens"].long()
        b = torch.nonzero(lens > 0)[:, 0]
        m = lens[b] - 1
        slot = s["table"][b, m // page].long() * page + m % page
        updates["k"] = turned(s["k_pre"][b], m[:, None].expand(-1, Hkv))
        updates["v"] = s["v_new"][b].double()
    got, rounded = {}, {}
    for name, x in updates.items():
        full = s[name].double()
        pg, r = slot // page, slot % page
        scale = s[name + "_scale"]
        if scale is None:
            rounded[name] = x.to(torch.bfloat16).double()
            for g in range(Hkv):
                full[pg, g, r] = x[:, g]
            got[name + "_scale"] = None
        else:
            sc = (x.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)
            # the scale and the quotient are defined in 32 bits: quotients on the border of two
            # e4m3 values are common where a row was not turned
            x32 = x.float()
            sc32 = (x32.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)
            rounded[name] = (x32 / sc32[..., None]).to(torch.float8_e4m3fn).double() * sc32[..., None].double()
            scale = scale.double()
            for g in range(Hkv):
                full[pg, g, r] = x[:, g] / sc[:, g, None]
                scale[pg, g, r] = sc[:, g]
            got[name + "_scale"] = scale
        got[name] = full
    if case["op"] == "append":
        return got
    # attention, one sequence and KV head at a time, over the rows as the cache holds them
    G, is_ret = case["Hq"] // Hkv, _is_ret(Hkv, case["n_ret"])
    out = torch.zeros((B, case["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    live = 0
    for bb, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        every = torch.arange(n, device="cuda")
        near = every[(every < case["sinks"]) | (every >= n - case["window"])]
        qs = turned(s["q"][bb], torch.full((case["Hq"],), n - 1, device="cuda"))
        for g in range(Hkv):
            pos = every if is_ret[g] else near
            pid = s["table"][bb, pos // page].long()
            rows = {}
            for name in ("k", "v"):
                x = s[name].view(torch.uint8 if s["k_scale"] is not None else torch.bfloat16)[pid, g, pos % page]
                if s["k_scale"] is not None:
                    x = x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][pid, g, pos % page].double()[:, None]
                rows[name] = x.double()
                if case["append"]:
                    rows[name][-1] = rounded[name][live, g]
            z = qs[g * G:(g + 1) * G] @ rows["k"].T / math.sqrt(D)
            lse[bb, g * G:(g + 1) * G] = torch.logsumexp(z, -1)
            out[bb, g * G:(g + 1) * G] = torch.softmax(z, -1) @ rows["v"]
        live += 1
    return got | {"out": out, "lse": lse}
