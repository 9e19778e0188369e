"""kvq_page_weights against the plain 64-bit form, within the bound counted
there from the operands' magnitudes."""
import math
import types

import pytest
import torch

import plain64
from quantized_kv_cache_09_gb300 import kvq

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(128)
FMTS = [kvq.KVQ_INT4_B64, kvq.KVQ_INT8_PAGE, kvq.KVQ_FP8_E4M3]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """A cache with sequences of the given lengths (codes by kvq_append, permuted pages) and new queries."""

    def __init__(self, fmt, lens, rows, H, g, spare=1, seed=0, q_scale=1.0, hot=10.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.fmt, self.lens_host, self.B = fmt, list(lens), len(lens)
        mb = max((max(lens) + 63) // 64 + spare, 1)
        self.cache = kvq.PagedKVCache(fmt, self.B * mb + 2, H, max_seqs=self.B)
        self.table = (torch.randperm(self.B * mb, generator=gen, device="cuda") + 2).to(torch.int32).view(self.B, mb)
        k = torch.randn(sum(lens), H, 128, generator=gen, device="cuda")
        k[:, :, 3] *= hot
        cu = _i32([0] + list(torch.tensor(lens).cumsum(0).tolist()))
        kvq.kvq_append(self.cache, k.half(), k.half(), cu, self.table, torch.zeros_like(cu[:-1]), max(max(lens), 1))
        self.cu_host = [0] + list(torch.tensor(rows).cumsum(0).tolist())
        self.cu, self.lens, self.max_rows = _i32(self.cu_host), _i32(lens), max(rows)
        self.q = (torch.randn(sum(rows), H * g, 128, generator=gen, device="cuda") * q_scale).half()
        self.before = torch.rand(self.B, mb, generator=gen, device="cuda")
        self.before *= torch.arange(mb, device="cuda") < ((self.lens + 63) // 64)[:, None]
        self.ws = kvq.page_weights_workspace(self.q.shape[0], H * g, mb)
        self.ws.fill_(0xFF)  # any contents

    def run(self, before="own", decay=1.0, scale=SM, out=None, stream=None):
        before = self.before if isinstance(before, str) else before
        out = torch.full_like(self.before, math.nan) if out is None else out
        kvq.kvq_page_weights(self.cache, self.q, self.cu, self.max_rows, self.table, self.lens, scale, decay, before,
                             out, self.ws, stream=stream)
        return out

    def check(self, before="own", decay=1.0, scale=SM, **kw):
        before = self.before if isinstance(before, str) else before
        got = self.run(before, decay, scale, **kw)
        torch.cuda.synchronize()
        ref, tol = plain64.page_weights(self.fmt, self.cache.k_codes, self.cache.k_scales, self.q, self.cu_host,
                                        self.table, self.lens_host, scale, decay, before)
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])
        assert kvq.kvq_get_device_status(self.cache) == (0, 0)
        return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,g", [(4, 1), (1, 8), (2, 3), (1, 32), (3, 16)])
def test_decode_rows(cuda_ok, fmt, H, g):
    b = Batch(fmt, [1, 63, 64, 65, 257, 700, 2111], [1] * 7, H, g, seed=1)
    b.check()
    b.check(before=None)
    b.check(decay=0.75)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,g", [(2, 1), (2, 4), (1, 5), (4, 64)])
def test_windows_of_rows(cuda_ok, fmt, H, g):
    """Chunks of different lengths, a sequence without new rows, chunks that span several pages."""
    b = Batch(fmt, [40, 300, 129, 500, 64, 1000], [3, 32, 129, 0, 64, 70], H, g, seed=2)
    got = b.check(decay=0.5)
    assert torch.equal(got[3], b.before[3])   # no new rows: as it was, without decay


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33])
def test_row_counts_around_the_tiles(cuda_ok, rows):
    Batch(kvq.KVQ_INT4_B64, [200, 333], [rows, max(1, rows - 1)], 2, 2, seed=3).check()


def test_mass_is_the_number_of_rows(cuda_ok):
    b = Batch(kvq.KVQ_INT8_PAGE, [1500, 90], [4, 2], 2, 4, seed=4)
    got = b.check(before=None).double().sum(1)
    assert torch.allclose(got.cpu(), torch.tensor([32.0, 16.0], dtype=torch.float64), rtol=1e-5)


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_and_peaky_scores(cuda_ok, fmt):
    """A negative scale, a zero one (every key alike), scores spread over hundreds of units."""
    b = Batch(fmt, [150, 900], [1, 7], 2, 4, seed=5, q_scale=6.0)
    for scale in (-SM, 0.0, SM, 1.0):
        b.check(scale=scale)


def test_in_place_and_repeatable(cuda_ok):
    b = Batch(kvq.KVQ_FP8_E4M3, [700, 64, 1], [5, 1, 1], 2, 8, seed=6)
    want = b.check(decay=0.9)
    for _ in range(3):
        assert torch.equal(b.run(decay=0.9), want)
    w = b.before.clone()
    assert torch.equal(b.run(before=w, decay=0.9, out=w), want)


def test_many_sequences(cuda_ok):
    """More sequences than one launch takes (512), more than one warp scans at once."""
    lens = [1 + (i * 37) % 190 for i in range(700)]
    Batch(kvq.KVQ_INT4_B64, lens, [1 if i % 11 else 0 for i in range(700)], 1, 2, seed=7).check()


def test_long_context(cuda_ok):
    Batch(kvq.KVQ_INT4_B64, [70001], [1], 1, 2, seed=8).check()


def test_bad_tables_and_lengths(cuda_ok):
    b = Batch(kvq.KVQ_INT4_B64, [300, 200, 100], [2, 1, 1], 2, 2, seed=9)
    want = b.check()
    b.lens[1] = b.table.shape[1] * 64 + 1      # beyond the table: skipped, its row untouched
    got = b.run()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_status(b.cache)[1] == kvq.KVQ_FLAG_BAD_LENGTH
    assert got[1].isnan().all() and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    b.lens[1] = 200
    b.table[2, 0] = b.cache.num_pages          # out of range: page 0 is read instead
    got = b.run()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_status(b.cache)[1] == kvq.KVQ_FLAG_BAD_PAGE
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_rows_than_the_bound_are_flagged(cuda_ok):
    b = Batch(kvq.KVQ_INT4_B64, [300, 200], [3, 2], 2, 2, seed=13)
    want = b.check()
    b.max_rows = 2
    got = b.run()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_status(b.cache)[1] == kvq.KVQ_FLAG_BAD_LENGTH
    assert got[0].isnan().all() and torch.equal(got[1], want[1])


def test_no_rows_at_all(cuda_ok):
    """A call without a single query keeps every weight."""
    b = Batch(kvq.KVQ_INT4_B64, [300, 200], [1, 1], 2, 2, seed=14)
    out = torch.full_like(b.before, math.nan)
    kvq.kvq_page_weights(b.cache, b.q[:0], _i32([0, 0, 0]), 4, b.table, b.lens, SM, 0.5, b.before, out, b.ws)
    kvq.kvq_page_weights(b.cache, b.q[:0], _i32([0, 0, 0]), 0, b.table, b.lens, SM, 0.5, b.before, out, b.ws)
    torch.cuda.synchronize()
    assert torch.equal(out, b.before) and kvq.kvq_get_device_status(b.cache) == (0, 0)


@pytest.mark.parametrize("rows", [1, 40])
def test_large_groups(cuda_ok, rows):
    """A single cache head under 200 query heads."""
    Batch(kvq.KVQ_FP8_E4M3, [130, 700], [rows, 1], 1, 200, seed=15).check()


def test_two_calls_at_once(cuda_ok):
    """Two streams, each with its own workspace, over one cache."""
    b = Batch(kvq.KVQ_INT8_PAGE, [3000, 900, 64], [20, 3, 1], 4, 4, seed=16)
    want = b.check()
    other = kvq.page_weights_workspace(b.q.shape[0], b.q.shape[1], b.table.shape[1])
    outs = [torch.empty_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, o, w in zip(streams, outs, (b.ws, other)):
            kvq.kvq_page_weights(b.cache, b.q, b.cu, b.max_rows, b.table, b.lens, SM, 1.0, b.before, o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_nan_in_keys_after_the_positions(cuda_ok):
    """Rows of an open page past the sequence's end are read but carry no weight, whatever they hold."""
    b = Batch(kvq.KVQ_FP8_E4M3, [100], [1], 1, 1, seed=10)
    want = b.check()
    b.cache.k_codes[b.table[0, 1].long(), :, 36:] = 0x7F  # NaN codes
    assert torch.equal(b.run(), want)


def test_refusals(cuda_ok):
    b = Batch(kvq.KVQ_INT4_B64, [100], [1], 1, 1, seed=11)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_page_weights(b.cache, b.q, b.cu, 1, b.table, b.lens, SM, 1.0, None, torch.empty_like(b.before), small)
    assert e.value.status == 6
    with pytest.raises(ValueError, match="shapes"):
        kvq.kvq_page_weights(b.cache, b.q, b.cu, 1, b.table, b.lens, SM, 1.0, b.before[:, :1].contiguous(),
                             torch.empty_like(b.before), b.ws)


def test_a_cache_on_another_device_is_refused(cuda_ok):
    b = Batch(kvq.KVQ_INT8_PAGE, [100], [1], 1, 1, seed=11)
    other = types.SimpleNamespace(struct=b.cache.struct, k_codes=types.SimpleNamespace(get_device=lambda: 1))
    with pytest.raises(ValueError, match="another device"):
        kvq.kvq_page_weights(other, b.q, b.cu, 1, b.table, b.lens, SM, 1.0, None, torch.empty_like(b.before), b.ws)


def test_other_stream_and_graph(cuda_ok):
    b = Batch(kvq.KVQ_INT4_B64, [700, 64], [3, 1], 2, 8, seed=12)
    want = b.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
