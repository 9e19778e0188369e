"""The operators around a prompt as they are used together: prompt attention
beside the append of the same rows, the weights of the prompt's last queries,
eviction, and decode steps over what is left -- each stage against plain 64-bit
forms, and the whole of it captured once and replayed."""
import math

import numpy as np
import pytest
import torch

import plain64
from oracle import oracle as orc
from quantized_kv_cache_09_gb300 import kvq

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(128)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Prompts:
    """Prompts of the given lengths on their way into a cache with room for growth."""

    def __init__(self, fmt, lens, H, g, window, keep, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.fmt, self.lens, self.H, self.Hq, self.window = fmt, lens, H, H * g, window
        T, B = sum(lens), len(lens)
        self.mb = max(lens) // 64 + 3
        rows = torch.randn(T, self.Hq + 2 * H, 128, generator=gen, device="cuda")
        rows[:, self.Hq:, 7] *= 10.0
        self.rows = rows.half()
        self.cu_host = [0] + list(np.cumsum(lens))
        self.cu = _i32(self.cu_host)
        self.cache = kvq.PagedKVCache(fmt, B * self.mb, H, max_seqs=B)
        self.table = torch.randperm(B * self.mb, generator=gen, device="cuda").to(torch.int32).view(B, self.mb)
        self.lengths, self.keep = _i32(lens), _i32(keep)
        self.weights = torch.zeros(B, self.mb, device="cuda")
        self.gone = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cu_w = _i32(list(np.cumsum([0] + [min(window, n) for n in lens])))
        self.last = torch.cat([torch.arange(z - min(window, z - a), z) for a, z in
                               zip(self.cu_host[:-1], self.cu_host[1:])]).cuda()
        self.out = torch.empty(T, self.Hq, 128, dtype=torch.float16, device="cuda")
        self.ws = kvq.page_weights_workspace(self.last.numel(), self.Hq, self.mb)
        self.zero = torch.zeros_like(self.lengths)
        self.step_q = torch.randn(B, self.Hq, 128, generator=gen, device="cuda").half()
        self.step_kv = torch.randn(2, B, H, 128, generator=gen, device="cuda").half()
        self.step_out = torch.empty(B, self.Hq, 128, dtype=torch.float16, device="cuda")
        self.step_ws = self.cache.workspace(self.Hq)
        self.one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        self.before = torch.empty_like(self.lengths)

    def run(self):
        Hq, H = self.Hq, self.H
        q, k, v = self.rows[:, :Hq], self.rows[:, Hq:Hq + H], self.rows[:, Hq + H:]
        kvq.kvq_prompt_attention(q, k, v, self.cu, max(self.lens), SM, self.out, status=self.cache.status)
        kvq.kvq_append(self.cache, k.contiguous(), v.contiguous(), self.cu, self.table, self.zero, max(self.lens))
        kvq.kvq_page_weights(self.cache, q[self.last].contiguous(), self.cu_w, self.window, self.table, self.lengths,
                             SM, 1.0, None, self.weights, self.ws)
        self.evict()
        self.step()

    def evict(self):
        kvq.kvq_evict_pages(self.table, self.lengths, self.weights, self.keep, 1, 2, self.table, self.lengths,
                            self.weights, self.gone, status=self.cache.status)

    def step(self):
        """A token per sequence behind the kept pages, attention over them, and the pages' new weights."""
        self.before.copy_(self.lengths)
        self.lengths += 1
        kvq.kvq_append(self.cache, self.step_kv[0], self.step_kv[1], self.one, self.table, self.before, 1)
        kvq.kvq_decode_attention_gqa(self.cache, self.step_q, self.table, self.lengths, SM, self.step_out, self.step_ws)
        kvq.kvq_page_weights(self.cache, self.step_q, self.one, 1, self.table, self.lengths, SM, 0.9, self.weights,
                             self.weights, self.ws)


@pytest.mark.parametrize("fmt", [kvq.KVQ_INT4_B64, kvq.KVQ_INT8_PAGE, kvq.KVQ_FP8_E4M3])
def test_prompt_to_decode(cuda_ok, fmt):
    lens, keep = [700, 64, 130, 1000, 5], [5, 4, 1, 9, 2]
    p = Prompts(fmt, lens, 2, 4, 32, keep, seed=1)
    table0 = p.table.clone()
    p.run()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_status(p.cache) == (0, 0)
    Hq, H = p.Hq, p.H
    ref, _, tol, _ = plain64.prompt(p.rows[:, :Hq], p.rows[:, Hq:Hq + H], p.rows[:, Hq + H:], p.cu_host, SM)
    assert ((p.out.double() - ref).abs() <= tol).all()
    # which pages stay: by the 64-bit weights over the cache as it was before the step (the step
    # rewrites only open pages, so the full pages' codes still stand)
    B = len(lens)
    for b in range(B):
        nb = (lens[b] + 63) // 64
        protected = min(nb, 1) + min(max(nb - 1, 0), 2)
        stay = min(nb, max(keep[b], protected))
        assert int(p.gone[b]) == nb - stay and int(p.lengths[b]) == lens[b] - 64 * (nb - stay) + 1
        row = p.table[b].tolist()
        assert sorted(row) == sorted(table0[b].tolist())          # a permutation of the row
        kept = [table0[b].tolist().index(x) for x in row[:stay]]
        assert kept == sorted(kept) and kept[0] == 0 and kept[-1] == nb - 1
        assert row[stay + p.mb - nb:] == [x for i, x in enumerate(table0[b].tolist()) if i < nb and i not in kept]
    # decode over the kept pages against the oracle on the cache as it is
    c = p.cache
    arrays = [t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
    tab, ln = p.table.cpu().numpy(), p.lengths.cpu().numpy()
    ref = orc.decode_attention(fmt, *arrays, tab, ln, p.step_q.cpu().numpy().view(np.uint16), np.float32(SM))
    vmax = orc.value_absmax(fmt, arrays[1], arrays[3], tab, ln, H, 128)
    assert orc.normalized_error(p.step_out.float().cpu().numpy(), ref, np.repeat(vmax, Hq // H, axis=1)) <= 2e-3
    # and the running weights: each new query adds a mass of 1 per head
    total = p.weights.double().sum(1).cpu()
    assert (total >= Hq * (1 - 1e-4)).all()


def test_kept_pages_are_those_of_most_weight(cuda_ok):
    """The weights of the window, by the plain form, choose the same pages wherever the margin is above their bound."""
    lens, keep = [900, 1200], [6, 7]
    p = Prompts(kvq.KVQ_INT8_PAGE, lens, 2, 4, 16, keep, seed=2)
    table0 = p.table.clone()
    p.run()
    torch.cuda.synchronize()
    q = p.rows[:, :p.Hq][p.last].contiguous()
    # (the step rewrote each open page, which eviction keeps whatever its weight: leave it out below)
    ref, tol = plain64.page_weights(p.fmt, p.cache.k_codes, p.cache.k_scales, q, p.cu_w.tolist(), table0, lens, SM,
                                    1.0, None)
    for b in range(2):
        nb = (lens[b] + 63) // 64
        kept = {table0[b].tolist().index(x) for x in p.table[b].tolist()[:keep[b]]}
        free = [j for j in range(1, nb - 2)]
        least_kept = min(ref[b, j] for j in free if j in kept)
        most_gone = max(ref[b, j] for j in free if j not in kept)
        # masses within a row share one denominator, whose open page the step has changed by little
        assert least_kept > most_gone * (1 - 1e-2) - 2 * tol[b].max()


def test_captured_and_replayed(cuda_ok):
    """The whole run as one graph: every replay from the same start gives the same bits."""
    p = Prompts(kvq.KVQ_INT4_B64, [400, 130, 70], 2, 2, 8, [3, 1, 1], seed=3)
    start = p.table.clone(), p.lengths.clone()

    def reset():
        p.table.copy_(start[0]), p.lengths.copy_(start[1])

    p.run()   # (also loads every kernel before the capture)
    torch.cuda.synchronize()
    want = [t.clone() for t in (p.out, p.table, p.lengths, p.weights, p.gone, p.step_out)]
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        got = (p.out, p.table, p.lengths, p.weights, p.gone, p.step_out)
        # (decode attention joins its splits in the order they finish, so its output is compared by value)
        assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3])) and torch.equal(want[4], got[4])
        assert torch.allclose(want[3], got[3]) and torch.allclose(want[5].float(), got[5].float(), atol=2e-3)
    assert kvq.kvq_get_device_status(p.cache) == (0, 0)


def test_freed_pages_serve_another_sequence(cuda_ok):
    """A page that left one row and went into another is written by its new owner alone."""
    p = Prompts(kvq.KVQ_FP8_E4M3, [640, 100], 1, 2, 8, [3, 9], seed=4)
    p.run()
    torch.cuda.synchronize()
    gone = int(p.gone[0])
    assert gone == 7
    out1 = p.step_out.clone()
    # the second sequence's spare entries now are the first one's freed pages
    p.table[1, 2] = p.table[0, -1]
    q1 = p.step_q.clone()
    k = torch.randn(70, 1, 128, device="cuda").half()
    before = p.lengths.clone()
    cu = _i32([0, 0, 70])
    kvq.kvq_append(p.cache, k, k, cu, p.table, before, 70)
    p.lengths[1] += 70
    kvq.kvq_decode_attention_gqa(p.cache, q1, p.table, p.lengths, SM, p.step_out, p.step_ws)
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_status(p.cache) == (0, 0)
    assert torch.allclose(p.step_out[0].float(), out1[0].float(), atol=2e-3)   # the first is as it was
    assert not torch.allclose(p.step_out[1].float(), out1[1].float(), atol=2e-3)
