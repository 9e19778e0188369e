"""Prompt attention, page weights and page eviction without a GPU: the C entry
points refuse bad arguments on the host before any CUDA call, the binding
refuses host tensors, and the plain 64-bit forms that the GPU tests compare
with are pinned by closed forms."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import plain64
from quantized_kv_cache_09_gb300 import kvq

P = ctypes.c_void_p(16)
ODD = ctypes.c_void_p(24)


def _cache(**kw):
    a = dict(fmt=0, num_heads=2, head_dim=128, page_tokens=64, num_pages=4, max_seqs=1, k_codes=16, v_codes=16,
             k_scales=16, v_scales=16, k_tail=None, v_tail=None, status=None)
    a.update(kw)
    return kvq.kvq_cache(*a.values())


def test_prompt_attention_refusals():
    f = kvq.lib().kvq_prompt_attention

    def call(dt=0, q=P, qs=1024, k=P, ks=256, v=P, vs=256, hq=8, h=2, d=128, cu=P, total=64, mx=64, n=1, scale=0.1,
             out=P, lse=None):
        return f(dt, q, qs, k, ks, v, vs, hq, h, d, cu, total, mx, n, scale, out, lse, None, None)

    assert call(dt=2) == 2 and call(dt=-1) == 2 and call(d=64) == 2
    assert call(n=-1) == 1 and call(mx=-1) == 1 and call(total=-1) == 1
    assert call(scale=math.inf) == 1 and call(scale=math.nan) == 1
    assert call(hq=7) == 1 and call(hq=0) == 1 and call(h=0) == 1 and call(hq=-8) == 1
    assert call(qs=1016) == 1 and call(ks=248) == 1 and call(vs=0) == 1      # rows that overlap
    assert call(qs=1028) == 1 and call(ks=260) == 1 and call(vs=257) == 1    # rows off 16 bytes
    assert call(hq=258, h=2, qs=258 * 128) == 2                              # 129 query heads per cache head
    assert call(n=65536) == 2 and call(total=2 ** 31) == 2
    assert call(qs=1 << 39) == 2
    for name in ("q", "k", "v", "out"):
        assert call(**{name: None}) == 1 and call(**{name: ODD}) == 1, name
    assert call(cu=None) == 1
    for name in ("n", "mx", "total"):   # nothing to do
        assert call(**{name: 0}, q=None, k=None, v=None, out=None, cu=None) == 0, name


def test_page_weights_refusals():
    lib = kvq.lib()
    f = lib.kvq_page_weights

    def call(c=None, q=P, hq=8, cu=P, total=4, mx=1, bt=P, mb=4, lens=P, n=4, scale=0.1, decay=1.0, win=None, wout=P,
             ws=P, nws=1 << 20):
        return f(ctypes.byref(_cache() if c is None else c), q, hq, cu, total, mx, bt, mb, lens, n, scale, decay, win,
                 wout, ws, nws, None)

    assert f(None, P, 8, P, 4, 1, P, 4, P, 4, 0.1, 1.0, None, P, P, 1 << 20, None) == 1
    assert call(_cache(fmt=3)) == 2 and call(_cache(head_dim=64)) == 2 and call(_cache(k_codes=24)) == 1
    assert call(n=-1) == 1 and call(mx=-1) == 1 and call(total=-1) == 1 and call(mb=0) == 1
    assert call(scale=math.nan) == 1 and call(decay=math.inf) == 1 and call(hq=3) == 1 and call(hq=0) == 1
    assert call(mb=(1 << 22) + 1) == 2 and call(mx=1 << 28) == 2
    assert call(mb=1 << 22, mx=1 << 20, total=1) == 2                        # units of one sequence
    assert call(n=0, q=None, cu=None, bt=None, lens=None, wout=None, ws=None) == 0
    for name in ("q", "cu", "bt", "lens", "wout"):
        assert call(**{name: None}) == 1, name
    assert call(q=ODD) == 1
    assert call(ws=None) == 6 and call(ws=ODD) == 6
    need = lib.kvq_page_weights_workspace_bytes(4, 8, 4)
    assert need >= 4 * 8 * 4 * 4 and call(nws=need - 1) == 6
    for bad in ((0, 8, 4), (4, 0, 4), (4, 8, 0), (-1, 8, 4)):
        assert lib.kvq_page_weights_workspace_bytes(*bad) == 0
    assert lib.kvq_page_weights_workspace_bytes(1 << 20, 64, 1 << 14) > 1 << 42   # sizes in 64 bits


def test_evict_pages_refusals():
    f = kvq.lib().kvq_evict_pages

    def call(bt=P, mb=4, lens=P, w=P, n=2, keep=P, sink=1, recent=1, to=P, lo=P, wo=P, gone=P):
        return f(bt, mb, lens, w, n, keep, sink, recent, to, lo, wo, gone, None, None)

    assert call(n=-1) == 1 and call(mb=0) == 1 and call(sink=-1) == 1 and call(recent=-1) == 1
    assert call(mb=32769) == 2 and call(n=(1 << 27) + 1) == 2
    assert call(n=0, bt=None, lens=None, w=None, keep=None, to=None, lo=None, wo=None, gone=None) == 0
    for name in ("bt", "lens", "w", "keep", "to", "lo", "wo", "gone"):
        assert call(**{name: None}) == 1, name


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 128, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    w = torch.zeros(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_prompt_attention(x, x, x, i, 4, 0.1, x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_prompt_attention(x.float(), x.float(), x.float(), i, 4, 0.1, x.float())
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_page_weights(None, x, i, 1, i.view(1, 2), i, 0.1, 1.0, None, w, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_evict_pages(i.view(1, 2), i[:1], w, i[:1], 0, 1, i.view(1, 2), i[:1], w, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        c = torch.zeros(1, 2, 64, 64, dtype=torch.uint8)
        kvq.PagedKVCache.over(0, c, c, torch.zeros(1, 2), torch.zeros(1, 2))


def test_nvtx_ranges_wrap_the_entry_points():
    code = ("from quantized_kv_cache_09_gb300 import kvq\n"
            "print(*(hasattr(getattr(kvq, n), '__wrapped__') for n in "
            "('kvq_prompt_attention', 'kvq_page_weights', 'kvq_evict_pages')))\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for value, want in (("1", "True True True"), ("0", "False False False")):
        run = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, KVQ_NVTX=value),
                             capture_output=True, text=True, check=True)
        assert run.stdout.strip() == want


def test_plain_prompt_closed_forms():
    """One token returns its value; equal keys average the prefix; lse counts them."""
    g = torch.Generator().manual_seed(1)
    v = torch.randn(5, 1, 128, generator=g).half()
    z = torch.zeros(5, 2, 128, dtype=torch.float16)
    out, lse, tol, _ = plain64.prompt(z, z[:, :1], v, [0, 1, 5], 0.3)
    assert torch.equal(out[0, 1], v[0, 0].double())
    want = torch.stack([v[1:2 + i, 0].double().mean(0) for i in range(4)])
    assert torch.allclose(out[1:, 0], want, rtol=0, atol=1e-15)
    assert torch.allclose(lse[1:, 1], torch.log(torch.arange(1, 5).double()))
    assert (tol > 0).all() and (tol < 1e-2).all()


def test_plain_page_weights_closed_forms():
    """Zero queries weigh every key alike; the masses of a row sum to 1."""
    codes = torch.arange(3 * 64 * 64).remainder(251).to(torch.uint8).view(3, 1, 64, 64)
    sc = torch.ones(3, 1)
    table = torch.tensor([[2, 0, 1]])
    q = torch.zeros(2, 2, 128, dtype=torch.float16)
    w, _ = plain64.page_weights(0, codes, sc, q, [0, 2], table, [130], 0.1, 0.5, torch.tensor([[2.0, 4.0, 6.0]]))
    want = [0.5 * o + 2 * (min(64, 129 - a) / 129 + min(64, 130 - a) / 130) for o, a in ((2, 0), (4, 64), (6, 128))]
    assert torch.allclose(w[0], torch.tensor(want, dtype=torch.float64), rtol=1e-14)
    q = torch.randn(2, 2, 128, generator=torch.Generator().manual_seed(2)).half()
    w, tol = plain64.page_weights(0, codes, sc, q, [0, 2], table, [130], 0.01, 1.0, None)
    assert abs(w.sum() - 4) < 1e-12 and (tol[0] < 1e-2).all()


def test_plain_evict_by_hand():
    table, w = [[10, 11, 12, 13, 14, 15, 16]], [[0.0, 3.0, 1.0, 3.0, 2.0, 9.0, 9.0]]
    # 5 pages used (the last holds 3 tokens), one sink, the open page: of 3.0, 1.0, 3.0 one stays
    assert plain64.evict(table, [4 * 64 + 3], w, [3], 1, 1) == ([[10, 11, 14, 15, 16, 12, 13]], [2 * 64 + 3],
                                                               [[0.0, 3.0, 2.0, 0.0, 0.0, 0.0, 0.0]], [2])
    assert plain64.evict(table, [4 * 64 + 3], w, [0], 0, 0)[0] == [[14, 15, 16, 10, 11, 12, 13]]
    assert plain64.evict(table, [0], w, [3], 1, 1) == (table, [0], [[0.0] * 7], [0])
    assert plain64.evict(table, [64], w, [9], 2, 3)[3] == [0]
