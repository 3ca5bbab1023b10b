"""DecodeLayer.prefill and PagedLayer.prefill as a serving program calls them: on other streams, in
captured graphs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, CAP = 4, 2, 4096


class Prefill:
    """A layer (two sequences, one retrieval and one local KV head) and prompts of n tokens."""

    def __init__(self, kind, n):
        from long_context_sparse_rtpurbo_b200 import layer, rtp
        self.rtp, self.kind, self.n = rtp, kind, n
        if kind == "paged":
            self.t = layer.PageTable(2, 2 * CAP // 64, 64, CAP)
            self.layer = layer.PagedLayer(self.t, HQ, HKV, 4, 128, CAP, [1, 0])
        else:
            self.layer = layer.DecodeLayer(2, HQ, HKV, 4, 128, CAP, [1, 0], [CAP, CAP], DEV)
            self.wk = torch.zeros((HKV, 128, 16), device=DEV)
        self.inputs(n)

    def inputs(self, n):
        gen = torch.Generator(device=DEV).manual_seed(n)
        self.q, self.k, self.v = (torch.randn((2, n, h, 128), dtype=torch.bfloat16, device=DEV, generator=gen)
                                  for h in (HQ, HKV, HKV))
        self.n_b = torch.tensor([n, n // 2 + 1], dtype=torch.int32, device=DEV)
        self.out = torch.zeros_like(self.q)
        if self.kind == "paged":
            self.slots = torch.empty((2, n), dtype=torch.int32, device=DEV)
            self.t.reserve(torch.zeros_like(self.n_b))
            self.t.reserve(self.n_b, self.slots)

    def run(self, stream=None):
        if self.kind == "paged":
            self.layer.prefill(self.q, self.k, self.v, self.n_b, self.slots, self.out, stream)
        else:
            self.layer.prefill(self.q, self.k, self.v, self.wk, self.n_b, self.out, stream)

    def cache(self):
        names = ("k", "v") if self.kind == "paged" else ("k_ret", "v_ret", "k_loc", "v_loc")
        return [getattr(self.layer, x) for x in names]

    def clear(self):
        for x in (self.out, *self.cache()):
            x.zero_()

    def results(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.out, *self.cache())]

    def ok(self):
        assert self.layer.status() == 0 and self.rtp.rtp_read_device_status(self.layer.pf_ws) == 0


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", ["contiguous", "paged"])
def test_prefill_needs_nothing_of_the_current_stream(kind):
    """A prompt on another stream while the current one is busy for milliseconds: all that the call reads
    was there before."""
    n = 700
    ref = Prefill(kind, n)
    ref.clear()
    ref.run()
    want = ref.results()
    p = Prefill(kind, n)
    p.clear()
    s = torch.cuda.Stream()
    busy = torch.zeros((8192, 8192), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy
    p.run(s)
    assert _same(p.results(), want)
    p.ok()


@pytest.mark.parametrize("kind", ["contiguous", "paged"])
@pytest.mark.parametrize("how", ["stream", "address", "current"])
def test_scratch_comes_from_the_calls_stream(kind, how):
    """A block of the scratch's very size that the current stream has let go of, with work on it maybe
    still queued there, is not the one that a call on another stream gets."""
    n = 3000
    ref = Prefill(kind, n)
    ref.clear()
    ref.run()
    want = ref.results()
    p = Prefill(kind, n)
    p.clear()
    size = p.rtp.rtp_prefill_workspace_bytes(p.layer.desc, n) + 256
    block = torch.zeros(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    lo = block.data_ptr()
    del block
    s = torch.cuda.Stream()
    if how == "current":
        with torch.cuda.stream(s):
            p.run()
    else:
        p.run(s if how == "stream" else s.cuda_stream)
    assert not lo <= p.layer.pf_ws.data_ptr() < lo + size
    assert _same(p.results(), want)
    p.ok()


@pytest.mark.parametrize("kind", ["contiguous", "paged"])
def test_address_of_the_default_stream(kind):
    """The default stream's address is 0: the scratch is marked as used there, not on a new stream."""
    n = 3000
    p = Prefill(kind, n)
    p.run()
    want = p.results()
    p.layer.pf_ws = None
    at = []
    real = torch.Tensor.record_stream
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.Tensor, "record_stream", lambda x, s: (at.append(s), real(x, s))[1])
        p.out.zero_()
        p.run(torch.cuda.default_stream().cuda_stream)
    assert torch.cuda.default_stream().cuda_stream == 0
    assert at == [torch.cuda.default_stream()]
    assert _same(p.results(), want)
    p.ok()


@pytest.mark.parametrize("kind", ["contiguous", "paged"])
@pytest.mark.parametrize("warm", [True, False])
def test_a_graphs_scratch_outlives_a_longer_prompt(kind, warm):
    """A captured prompt, then a longer one that needs more scratch, then tensors of the size of the
    first scratch: a replay gives the results again and writes to none of them. The scratch is made
    before the capture or in it."""
    Prefill(kind, 500).run()                              # (loads every kernel)
    p, ref = Prefill(kind, 500), Prefill(kind, 500)
    ref.clear()
    ref.run()
    want = ref.results()
    if warm:
        p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    first = p.layer.pf_ws
    lo, size = first.data_ptr(), first.numel()
    del first
    kept = {x: getattr(p, x) for x in ("q", "k", "v", "n_b", "out") + (("slots",) if kind == "paged" else ())}
    p.inputs(1500)
    p.run()
    assert p.layer.pf_ws.numel() > size
    others = [torch.full((size + 256 * i,), 0xA5, dtype=torch.uint8, device=DEV) for i in (0, 1, 1, 1)]
    assert not any(x.data_ptr() < lo + size and lo < x.data_ptr() + x.numel() for x in others)
    torch.cuda.synchronize()
    for x, t in kept.items():
        setattr(p, x, t)
    if kind == "paged":                                   # the prompt's own pages again
        p.t.reserve(torch.zeros_like(p.n_b))
        p.t.reserve(p.n_b, p.slots)
    p.clear()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want[0])
    if kind == "contiguous":                              # (pages are other ones by now)
        assert _same(p.cache(), want[1:])
    assert all((x == 0xA5).all() for x in others)
    p.ok()
