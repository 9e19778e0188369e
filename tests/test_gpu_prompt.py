"""kvq_prompt_attention against the plain 64-bit form, within the bound counted
there: the operands' rounding of P, binary32 scores and sums, the output's own
rounding."""
import math

import pytest
import torch

import plain64
from quantized_kv_cache_09_gb300 import kvq

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(128)
TYPES = [torch.float16, torch.bfloat16]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(lens, Hq, H, dtype, seed=0, q_scale=1.0, pad=0, fused=False, hot=10.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + pad
    x = torch.randn(T, Hq + 2 * H, 128, generator=g, device="cuda")
    x[:, :Hq] *= q_scale
    x[:, Hq:, 5] *= hot
    x = x.to(dtype)
    parts = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return (parts if fused else tuple(t.contiguous() for t in parts)) + (cu,)


def _run(q, k, v, cu, scale=SM, max_n=None, lse=True, stream=None, out=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    ls = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    status = _i32([0])
    mx = max([b - a for a, b in zip(cu[:-1], cu[1:])] + [0]) if max_n is None else max_n
    kvq.kvq_prompt_attention(q, k, v, _i32(cu), mx, scale, out, lse=ls, status=status, stream=stream)
    torch.cuda.synchronize()
    return out, ls, int(status)


def _check(q, k, v, cu, scale=SM, **kw):
    out, lse, status = _run(q, k, v, cu, scale, **kw)
    assert status == 0
    ref, ref_lse, tol, tol_lse = plain64.prompt(q, k, v, cu, scale)
    inside = ~ref_lse.isnan()
    bad = inside[:, :, None] & ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), out[bad][:4], ref[bad][:4], tol[bad][:4])
    if lse is not None:
        bad = inside & ~((lse.double() - ref_lse).abs() <= tol_lse)
        assert not bad.any(), (bad.nonzero()[:4].tolist(), lse[bad][:4], ref_lse[bad][:4], tol_lse[bad][:4])
        assert (lse[~inside] == 7.0).all()
    assert (out[~inside] == 7.0).all()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 2), (8, 2)])
def test_one_sequence(cuda_ok, dtype, Hq, H):
    for n in (1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 400, 777):
        _check(*_inputs([n], Hq, H, dtype, seed=n))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,H", [(2, 2), (3, 1), (10, 2), (7, 1), (32, 1), (128, 1), (100, 1), (66, 2)])
def test_ragged_groups(cuda_ok, dtype, Hq, H):
    """Group sizes that divide a tile's 128 rows and that do not, lengths cut anywhere, empty sequences."""
    _check(*_inputs([5, 0, 130, 1, 64, 300, 0, 17, 129], Hq, H, dtype, seed=Hq))


@pytest.mark.parametrize("dtype", TYPES)
def test_views_of_a_fused_projection_and_padding(cuda_ok, dtype):
    """Rows with gaps; rows behind the last sequence hold NaN and are left alone; cu starts past row 0."""
    q, k, v, cu = _inputs([100, 33, 200], 8, 2, dtype, seed=3, pad=70, fused=True)
    for t in (q, k, v):
        t[cu[-1]:] = math.nan
    assert not q.is_contiguous()
    want = _check(q, k, v, cu)
    for t in (q, k, v):
        t[:cu[1]] = math.inf     # the first sequence's rows belong to nobody now
    got = _check(q, k, v, cu[1:])
    assert torch.equal(got[cu[1]:], want[cu[1]:])


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_in_their_rows(cuda_ok, dtype):
    """An infinity or NaN in v at token t changes the rows from t on alone, in its own element, within its own
    sequence; NaN in k at t makes the rows from t on NaN."""
    q, k, v, cu = _inputs([70, 300, 129], 4, 2, dtype, seed=4)
    want, wl, _ = _run(q, k, v, cu)
    v2, k2 = v.clone(), k.clone()
    at = cu[1] + 200
    v2[at, 0, 3], v2[at, 0, 9], v2[cu[2] + 128, 1, 60] = math.inf, math.nan, -math.inf
    got, gl, status = _run(q, k, v2, cu)
    hit = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    hit[at:cu[2], 0:2, 3] = True
    hit[at:cu[2], 0:2, 9] = True
    hit[cu[2] + 128, 2:4, 60] = True
    assert status == 0 and torch.equal(got[~hit], want[~hit]) and torch.equal(gl, wl)
    assert not got[hit].isfinite().any()
    assert (got[at:cu[2], 0:2, 3] == math.inf).all() and got[at:cu[2], 0:2, 9].isnan().all()
    k2[at, 1, 7] = math.nan
    got, gl, _ = _run(q, k2, v, cu)
    hit = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    hit[at:cu[2], 2:4] = True
    assert torch.equal(got[~hit], want[~hit]) and got[hit].isnan().all() and gl[hit[:, :, 0]].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_scales_and_growing_maxima(cuda_ok, dtype):
    """Negative and zero scales; scores that grow along the sequence, so that the running maximum moves often."""
    q, k, v, cu = _inputs([520, 140], 4, 2, dtype, seed=5, q_scale=3.0)
    for scale in (-SM, 0.0, 0.5, 1e-30):
        _check(q, k, v, cu, scale)
    ramp = torch.linspace(-3, 3, 660, device="cuda")[:, None]
    q[:, :, 0] = 8.0
    k[:, :, 0] = (ramp * 20).to(dtype)
    _check(q, k, v, cu, 0.25)
    _check(q, k, v, cu, -0.25)


def test_long_prompt(cuda_ok):
    """More units than SMs: every CTA takes several, tiles of both parities."""
    _check(*_inputs([4100, 900, 2050, 3], 8, 4, torch.bfloat16, seed=6))


def test_many_sequences(cuda_ok):
    """More sequences than one warp holds lengths of."""
    _check(*_inputs([1 + (i * 53) % 140 for i in range(90)], 4, 1, torch.float16, seed=7))


def test_thousands_of_short_prompts(cuda_ok):
    """A batch whose every prompt is a few tokens, some empty, in several head groups of units."""
    lens = [(i * 7) % 12 for i in range(3000)]
    _check(*_inputs(lens, 2, 2, torch.float16, seed=14))


def test_few_rows_in_a_large_buffer(cuda_ok):
    """Bounds that allow for many more units than there are: the buffers of a captured step, for instance."""
    for lens in ([5, 0, 130, 1], [0, 0], [300]):
        _check(*_inputs(lens, 4, 4, torch.bfloat16, seed=15, pad=40000), max_n=40000)


def test_units_of_very_different_lengths(cuda_ok):
    """More units than SMs, long and short: which CTA has one depends on timing, the bits do not."""
    lens = [1900, 3, 640, 1, 129, 2500, 77, 300]
    q, k, v, cu = _inputs(lens, 8, 8, torch.float16, seed=16)
    want = _check(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(_run(q, k, v, cu)[0], want)


def test_many_sequences_of_many_lengths(cuda_ok):
    """Levels of few units each, in several groups of heads: units come out of order by more than a level."""
    lens = [1 + (i * 97) % 1210 for i in range(150)]
    _check(*_inputs(lens, 12, 12, torch.float16, seed=17))


def test_without_lse_and_repeatable(cuda_ok):
    q, k, v, cu = _inputs([600, 128], 8, 1, torch.float16, seed=8)
    want, _, _ = _run(q, k, v, cu)
    for _ in range(3):
        got, _, _ = _run(q, k, v, cu, lse=False)
        assert torch.equal(got, want)
    got, _, _ = _run(q, k, v, cu, max_n=5000)   # a loose bound on the lengths
    assert torch.equal(got, want)


def test_bad_lengths_are_flagged(cuda_ok):
    q, k, v, cu = _inputs([100, 50, 60], 2, 2, torch.float16, seed=9)
    want, _, _ = _run(q, k, v, cu)
    got, _, status = _run(q, k, v, cu, max_n=99)    # the first is longer than the bound
    assert status == kvq.KVQ_FLAG_BAD_LENGTH
    assert (got[:100] == 7.0).all() and torch.equal(got[100:], want[100:])
    got, _, status = _run(q, k, v, [0, 100, 150, 211], max_n=100)   # the last ends past the rows
    assert status == kvq.KVQ_FLAG_BAD_LENGTH
    assert (got[150:] == 7.0).all() and torch.equal(got[:150], want[:150])
    got, _, status = _run(q, k, v, [0, 100, 50, 110], max_n=100)    # one runs backwards
    assert status == kvq.KVQ_FLAG_BAD_LENGTH
    assert torch.equal(got[:50], want[:50])


def test_empty_calls_and_refusals(cuda_ok):
    q, k, v, cu = _inputs([10], 2, 2, torch.float16)
    out = torch.full_like(q, 7.0)
    kvq.kvq_prompt_attention(q, k, v, _i32([0]), 10, SM, out)
    kvq.kvq_prompt_attention(q, k, v, _i32([0, 0]), 0, SM, out)
    kvq.kvq_prompt_attention(q[:0], k[:0], v[:0], _i32([0, 0]), 4, SM, out[:0])
    kvq.kvq_prompt_attention(q, k, v, _i32([3, 3]), 10, SM, out)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    with pytest.raises(ValueError, match="side by side"):
        kvq.kvq_prompt_attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, _i32(cu), 10, SM, out)
    with pytest.raises(ValueError):
        kvq.kvq_prompt_attention(q, k.bfloat16(), v, _i32(cu), 10, SM, out)
    with pytest.raises(ValueError, match="shapes"):
        kvq.kvq_prompt_attention(q, k[:5], v[:5], _i32(cu), 10, SM, out)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_prompt_attention(q[:, :1], k[:, :2], v[:, :2], _i32(cu), 10, SM, out[:, :1].contiguous())
    assert e.value.status == 1   # 1 query head over 2 cache heads
    wide = torch.zeros(4, 129, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_prompt_attention(wide, wide[:, :1], wide[:, :1], _i32([0, 4]), 4, SM, wide.clone())
    assert e.value.status == 2


def test_other_stream_two_at_once_and_graph(cuda_ok):
    a, b = _inputs([700, 64], 8, 2, torch.float16, seed=12), _inputs([333, 900], 4, 4, torch.bfloat16, seed=13)
    wa, wb = _run(*a)[0], _run(*b)[0]
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    cua, cub = _i32(a[3]), _i32(b[3])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        kvq.kvq_prompt_attention(*a[:3], cua, 700, SM, oa, stream=s1)
        kvq.kvq_prompt_attention(*b[:3], cub, 900, SM, ob, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_prompt_attention(*a[:3], cua, 700, SM, oa)
        kvq.kvq_prompt_attention(*b[:3], cub, 900, SM, ob)
    for _ in range(2):
        oa.zero_(), ob.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
