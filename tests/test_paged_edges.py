"""Refusals and host-side rules of the paged calls at their edges (CPU)."""
import ctypes
import os
import time

import pytest
import torch

from long_context_sparse_rtpurbo_b200 import _lib, rtp
from test_paged_host import X, _cache, _desc, _pool


def test_reserve_step_refusals():
    """Those of rtp_paged_reserve; step_lens itself may be null."""
    lib = _lib.load()
    names = ("lens", "new", "ctr", "lens_out", "ctr_out")

    def call(pool=None, n_new=1, slots=X, step=X, ws=X, wsb=4096, **kw):
        p = _pool(**(pool or {}))
        return lib.rtp_paged_reserve_step(ctypes.byref(p), *(kw.get(n, X) for n in names), slots, n_new,
                                          step, ws, wsb, None)

    for step in (None, X):
        for n in names:
            assert call(step=step, **{n: None}) == _lib.RTP_EINVAL, n
        assert call(step=step, slots=None) == _lib.RTP_EINVAL
        assert call(dict(B=4097), step=step) == _lib.RTP_ESHAPE
        assert call(step=step, wsb=4095) == _lib.RTP_EWORKSPACE
    rtp.rtp_debug_fail_next_call(_lib.RTP_ECUDA)
    assert call(lens=None) == _lib.RTP_ECUDA
    assert call(lens=None) == _lib.RTP_EINVAL


def test_reserve_step_checks_its_tensor():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = rtp.make_page_pool(i32(3), i32(2, 4), 16)
    ctr = torch.zeros(2, dtype=torch.int64)
    for bad in (i32(3), torch.zeros(2), torch.zeros(2, dtype=torch.int64), i32(4)[::2], 5):
        with pytest.raises(ValueError, match="step_lens"):
            rtp.rtp_paged_reserve_step(pool, i32(2), i32(2), ctr, i32(2), ctr, i32(2, 1), 1, bad,
                                       torch.zeros(4096, dtype=torch.uint8))


def test_layers_of_two_rope_bases_cost_no_more():
    """A description's check costs the same whether the call before had another RoPE base or not (it
    took 6 times as long while one base's tables were kept). The least of many runs, with a factor of
    three for noise."""
    slots = rtp.rtp_build_slot_map([1, 0])[0]
    a, b = (rtp.LayerDesc(1, 4, 2, 4, 64, 64, slots, base) for base in (1e4, 1e6))
    check = _lib.load().rtp_paged_workspace_bytes

    def cost(first, second):
        best = 1e9
        for _ in range(40):
            t0 = time.perf_counter()
            for _ in range(100):
                check(first.ref)
                check(second.ref)
            best = min(best, time.perf_counter() - t0)
        return best

    assert check(a.ref) == check(b.ref) > 0
    assert cost(a, b) < 3 * cost(a, a)


def test_append_of_no_tokens_does_nothing():
    """Arrays of no elements have no address. The description and the cache are checked all the same."""
    lib, d, c = _lib.load(), _desc(), _cache()
    call = lambda c: lib.rtp_paged_append_kv(d.ref, ctypes.byref(c), None, None, X, None, 0, None, None)
    assert call(c) == _lib.RTP_OK and rtp.rtp_last_launch_count() == 0
    assert call(_cache(page_size=8)) == _lib.RTP_ESHAPE


def test_binding_is_built_with_the_toolkit_of_nvcc(tmp_path, monkeypatch):
    """A toolkit in another place than /usr/local/cuda, named by NVCC or found through the path."""
    from long_context_sparse_rtpurbo_b200 import build
    home = tmp_path / "cuda"
    for d in ("bin", "include"):
        (home / d).mkdir(parents=True)
    (home / "bin" / "nvcc").write_text("#!/bin/sh\n")
    (home / "bin" / "nvcc").chmod(0o755)
    (home / "include" / "cuda_runtime_api.h").write_text("")
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    monkeypatch.setenv("NVCC", str(home / "bin" / "nvcc"))
    build.build_binding()
    assert f"-I{home / 'include'}" in ran[0] and "-I/usr/local/cuda/include" not in ran[0]
    link = tmp_path / "nvcc"                                 # a link to it somewhere on the path
    os.symlink(home / "bin" / "nvcc", link)
    monkeypatch.setenv("NVCC", str(link))
    assert build.cuda_include() == str(home / "include")
    (home / "include" / "cuda_runtime_api.h").unlink()
    inner = home / "targets" / "x86_64-linux" / "include"
    inner.mkdir(parents=True)
    (inner / "cuda_runtime_api.h").write_text("")
    assert build.cuda_include() == str(inner)


def test_workspace_init_refuses_other_devices(monkeypatch):
    """Host memory, and a device that is not the current one (whose stream would clear it out of order
    with that device's)."""
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="current device"):
        rtp.rtp_paged_workspace_init(ws)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    with pytest.raises(ValueError, match="current device"):
        rtp.rtp_paged_workspace_init(ws)
