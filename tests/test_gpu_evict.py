"""kvq_evict_pages against the plain form: every output is a whole number or a
copied weight, so all of them have to be equal."""
import math

import pytest
import torch

import plain64
from quantized_kv_cache_09_gb300 import kvq

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(table, lens, weights, keep, sink, recent, in_place=False, stream=None):
    status = _i32([0])
    if in_place:
        t, n, w = table.clone(), lens.clone(), weights.clone()
        to, no, wo = t, n, w
    else:
        t, n, w = table, lens, weights
        to, no, wo = torch.full_like(t, -7), torch.full_like(n, -7), torch.full_like(w, -7.0)
    gone = torch.full_like(n, -7)
    kvq.kvq_evict_pages(t, n, w, keep, sink, recent, to, no, wo, gone, status=status, stream=stream)
    torch.cuda.synchronize()
    return to, no, wo, gone, int(status)


def _check(table, lens, weights, keep, sink, recent, **kw):
    to, no, wo, gone, status = _run(table, lens, weights, keep, sink, recent, **kw)
    T, L, W, G = plain64.evict(table.tolist(), lens.tolist(), weights.tolist(), keep.tolist(), sink, recent)
    assert to.tolist() == T and no.tolist() == L and gone.tolist() == G and status == 0
    assert torch.equal(wo, torch.tensor(W, device="cuda")) or (
        torch.equal(torch.nan_to_num(wo, nan=-3.0), torch.nan_to_num(torch.tensor(W, device="cuda"), nan=-3.0)))


def _case(seed, blocks, spare, levels=None):
    g = torch.Generator().manual_seed(seed)
    B, mb = len(blocks), max(max(blocks) + spare, 1)
    table = torch.randperm(B * mb, generator=g).to(torch.int32).view(B, mb)
    w = torch.rand(B, mb, generator=g) if levels is None else torch.randint(0, levels, (B, mb), generator=g).float()
    lens = [max(0, (nb - 1) * 64 + int(torch.randint(1, 65, (1,), generator=g))) if nb else 0 for nb in blocks]
    return table.cuda(), _i32(lens), w.cuda()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sink,recent", [(0, 0), (1, 2), (4, 1), (1000, 7), (0, 100000)])
def test_ragged_rows(cuda_ok, sink, recent, in_place):
    blocks = [0, 1, 2, 3, 7, 31, 32, 33, 64, 129, 300, 17]
    table, lens, w = _case(1, blocks, 5)
    for keep in ([0] * 12, [1] * 12, [-3] * 12, [5] * 12, [nb // 2 + 1 for nb in blocks], [10 ** 9] * 12):
        _check(table, lens, w, _i32(keep), sink, recent, in_place=in_place)


@pytest.mark.parametrize("mb", [1, 127, 128, 129, 511, 512, 513, 1023, 1024, 1025, 4096, 4097, 16385, 18432, 18433, 32768])
def test_row_lengths_around_the_instances(cuda_ok, mb):
    """Rows as long as each instance of the kernel takes, and one more; full and nearly full."""
    table, lens, w = _case(2, [mb, max(1, mb - 3), mb // 2 + 1], 0)
    _check(table, lens, w, _i32([max(1, mb // 3), mb - 1, 2]), 1, 2, in_place=mb % 2 == 0)


def test_ties_go_to_the_lower_index(cuda_ok):
    for levels in (1, 2, 5):
        table, lens, w = _case(3, [500, 1500, 64], 3, levels)
        _check(table, lens, w, _i32([123, 700, 32]), 2, 3)


def test_special_weights(cuda_ok):
    """Infinities, NaN, both zeros, subnormals, negative weights: ordered, copied, a NaN the least."""
    vals = [math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0, -1.0]
    g = torch.Generator().manual_seed(4)
    table, lens, _ = _case(5, [200, 130], 2)
    w = torch.tensor(vals)[torch.randint(0, len(vals), table.shape, generator=g)].cuda()
    for keep in (1, 20, 64, 100, 128, 190):
        _check(table, lens, w, _i32([keep, keep]), 1, 1)


def test_again_is_a_no_op_and_pages_are_permuted(cuda_ok):
    table, lens, w = _case(6, [90, 40], 6)
    keep = _i32([30, 30])
    t1, n1, w1, g1, _ = _run(table, lens, w, keep, 1, 2)
    t2, n2, w2, g2, _ = _run(t1, n1, w1, keep, 1, 2)
    assert g1.tolist() == [60, 10] and g2.tolist() == [0, 0]
    assert torch.equal(t1, t2) and torch.equal(n1, n2) and torch.equal(w1, w2)
    assert torch.equal(t1.sort(1).values, table.sort(1).values)


def test_bad_lengths_are_copied_and_flagged(cuda_ok):
    table, lens, w = _case(7, [20, 20, 20, 20], 0)
    lens[0], lens[2] = -1, 20 * 64 + 1
    to, no, wo, gone, status = _run(table, lens, w, _i32([5] * 4), 1, 1)
    assert status == kvq.KVQ_FLAG_BAD_LENGTH
    for b in (0, 2):
        assert torch.equal(to[b], table[b]) and torch.equal(wo[b], w[b]) and no[b] == lens[b] and gone[b] == 0
    assert gone[1] == 15 and gone[3] == 15


def test_empty_batch_and_refusals(cuda_ok):
    z = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    e = _i32([])
    kvq.kvq_evict_pages(z, e, z.float(), e, 1, 1, z.clone(), e.clone(), z.float(), e.clone())
    big = torch.zeros(1, 32769, dtype=torch.int32, device="cuda")
    with pytest.raises(kvq.KvqError) as err:
        kvq.kvq_evict_pages(big, _i32([1]), big.float(), _i32([1]), 1, 1, big, _i32([1]), big.float(), _i32([1]))
    assert err.value.status == 2
    t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="shapes"):
        kvq.kvq_evict_pages(t, _i32([1]), t.float(), _i32([1, 1]), 1, 1, t, _i32([1, 1]), t.float(), _i32([1, 1]))


def test_other_stream_and_graph(cuda_ok):
    table, lens, w = _case(8, [70, 50], 2)
    keep = _i32([20, 20])
    want = _run(table, lens, w, keep, 1, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(table, lens, w, keep, 1, 2, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(want[:4], got[:4]))
    t, n, x, gone = table.clone(), lens.clone(), w.clone(), _i32([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_evict_pages(t, n, x, keep, 1, 2, t, n, x, gone)
    for _ in range(2):  # each replay on fresh rows
        t.copy_(table), n.copy_(lens), x.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t, want[0]) and torch.equal(n, want[1]) and torch.equal(x, want[2])
