"""What is measured of the operators around a prompt and of eviction from the paged cache.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and as the framework's call:

  prompt   kvq_prompt_attention: causal attention of whole prompts, packed
           sequences of different lengths, grouped query heads, over their own
           fp16 or bf16 rows (before kvq_append quantizes them).
  weights  kvq_page_weights: the softmax weight that every page of the
           quantized cache receives from the newest queries of its sequence,
           summed over heads and queries, added to a running total.
  evict    kvq_evict_pages: the pages of least total weight leave each block
           table; the kept ones close ranks, the freed ones go to the row's end.

`own` chooses which form `run` takes.
"""
import math

import numpy as np
import torch

own = False

D = 128
PAGE = 64
FMT = {"int4": 0, "int8": 1, "fp8": 2}
CODE_MAX = {"int4": 7.5, "int8": 127.0, "fp8": 448.0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths from lo to hi, spread over their logarithm, odd ones among them, in a mixed order."""
    if n == 1:
        return [hi]
    out = []
    for i in range(n):
        j = (i * 7) % n if n % 7 else (i * 5) % n
        x = int(round(lo * (hi / lo) ** (j / (n - 1))))
        out.append(min(hi, max(lo, x | 1 if lo < x < hi else x)))
    return out


def _prompt(name, lens, heads, kv_heads, dtype, lse=False, fused=False, pad=0):
    return {"name": name, "op": "prompt", "lens": ",".join(str(n) for n in lens), "heads": heads,
            "kv_heads": kv_heads, "dtype": dtype, "lse": lse, "fused": fused, "pad": pad}


def _weights(name, fmt, lens, heads, kv_heads, rows=1, decay=1.0, spare=1):
    return {"name": name, "op": "weights", "fmt": fmt, "lens": ",".join(str(n) for n in lens), "heads": heads,
            "kv_heads": kv_heads, "rows": rows, "decay": decay, "spare": spare}


def _evict(name, blocks, keep, sink, recent, spare=0):
    return {"name": name, "op": "evict", "blocks": ",".join(str(n) for n in blocks), "keep": keep, "sink": sink,
            "recent": recent, "spare": spare}


def listed():
    return [
        # a handful of one-line requests that arrive together: the smallest call, where latency counts
        _prompt("prompt-short-lines", [1, 7, 33, 64, 96, 130], 32, 8, "fp16"),
        # a batch of full prompts through one layer of the Llama-2-7B shape (32 heads, no groups); the
        # logarithms of the sums are kept, as for joining with attention over a cached prefix
        _prompt("prompt-7b-layer", [2048] * 8, 32, 32, "fp16", lse=True),
        # a continuous-batching step's prompts of the Llama-3-8B shape in bf16, cut as views out of one fused
        # projection whose buffer is padded behind the last sequence
        _prompt("prompt-8b-ragged", _spread(65, 8192, 16), 32, 8, "bf16", fused=True, pad=45),
        # one long document through a layer of the Llama-3-70B shape
        _prompt("prompt-70b-document", [16384], 64, 8, "fp16"),
        # the page weights of the smallest decode step, after its 257th token, over an FP8 cache
        _weights("weights-tiny", "fp8", [257, 257], 4, 4),
        # one decode step of the 7B layer, int4: a query per head and sequence
        _weights("weights-7b-layer", "int4", [8193] * 8, 32, 32),
        # one decode step of the 70B-shaped layer over an FP8 cache: 8 query heads share each cache head,
        # older steps fade
        _weights("weights-70b-layer-fp8", "fp8", [8192 - 37 * b for b in range(32)], 64, 8, decay=0.98),
        # one decode step over long contexts, int4
        _weights("weights-long-context", "int4", [32768 - 129 * b for b in range(16)], 32, 32),
        # the last 32 tokens of each prompt judge its pages before the first answer token, int8, ragged
        _weights("weights-window", "int8", _spread(512, 16384, 16), 32, 8, rows=32),
        # a small batch over its budget by a few pages
        _evict("evict-small", [9, 5, 17, 12], 0.6, 1, 2, spare=3),
        # a serving batch that goes back to half of its pages
        _evict("evict-batch", _spread(64, 256, 64), 0.5, 1, 4, spare=8),
        # contexts of up to a million tokens
        _evict("evict-million", _spread(4096, 16384, 16), 0.25, 2, 16, spare=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "weights", "weights", "evict"])
    if op == "prompt":
        kv, g = rng.choice([(1, 32), (2, 4), (4, 1), (4, 7), (8, 3), (8, 4), (8, 8), (32, 1), (6, 5), (16, 2)])
        top = _log_int(rng, 1, 8192)
        n = rng.randint(1, 24)
        lens = [_log_int(rng, 1, top) for _ in range(n - 1)] + [top]
        rng.shuffle(lens)
        while sum(x * x for x in lens) * kv * g > 16384 * 16384 * 64 // 2:
            lens.remove(max(lens))
        c = _prompt("", lens, kv * g, kv, rng.choice(["fp16", "bf16"]), rng.random() < 0.5, rng.random() < 0.5,
                    rng.choice([0, rng.randint(1, 200)]))
    elif op == "weights":
        kv, g = rng.choice([(1, 32), (2, 3), (4, 1), (8, 4), (8, 8), (8, 5), (16, 2), (32, 1)])
        rows = rng.choice([1, 1, _log_int(rng, 2, 64)])
        top = _log_int(rng, rows, 16384)
        n = rng.randint(1, 32)
        while n > 1 and n * kv * top > (1 << 21):
            n -= 1
        while rows > 1 and n * kv * g * top * rows > (1 << 29):
            rows -= 1
        lens = [_log_int(rng, rows, top) for _ in range(n - 1)] + [top]
        c = _weights("", rng.choice(["int4", "int8", "fp8"]), lens, kv * g, kv, rows,
                     rng.choice([1.0, 0.9, rng.uniform(0.5, 1.0)]), rng.randint(0, 4))
    else:
        top = _log_int(rng, 3, 16384)
        n = rng.randint(1, 16)
        c = _evict("", [_log_int(rng, 1, top) for _ in range(n - 1)] + [top], rng.uniform(0.05, 1.0),
                   rng.randint(0, 4), rng.randint(0, 16), rng.randint(0, 40))
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, heads, outliers=True):
    """n rows of normal values; four channels of each head are ten times as large, as keys and values have them."""
    x = torch.randn((n, heads, D), generator=g, device="cuda", dtype=torch.float32)
    if outliers:
        hot = torch.randint(0, D, (heads, 4), generator=g, device="cuda")
        m = torch.ones((heads, D), device="cuda").scatter_(1, hot, 10.0)
        x *= m
    return x


def _prepare_prompt(case, seed):
    g = _gen(seed)
    lens = _ints(case["lens"])
    H, Hq = case["kv_heads"], case["heads"]
    dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
    T = sum(lens) + case["pad"]
    q, k, v = _rows(g, T, Hq, False).to(dt), _rows(g, T, H).to(dt), _rows(g, T, H).to(dt)
    if case["fused"]:
        rows = torch.cat([q, k, v], 1)  # one projection's output: [T][heads + 2 kv_heads][128]
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return {"op": "prompt", "q": q, "k": k, "v": v, "cu_host": cu, "max": max(lens),
            "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
            "scale": 1.0 / math.sqrt(D),
            "out": torch.zeros((T, Hq, D), dtype=dt, device="cuda"),
            "lse": torch.zeros((T, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None,
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _quantize(fmt, x):
    """Blocks of 64 rows x 128 values -> codes as the cache stores them, and their scales."""
    a = x.abs().amax((-2, -1))
    s = a / CODE_MAX[fmt]
    y = x / torch.where(s > 0, s, 1.0)[..., None, None]
    if fmt == "fp8":
        return y.to(torch.float8_e4m3fn).view(torch.uint8), s
    if fmt == "int8":
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8), s
    c = y.round().clamp(-8, 7).to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8), s


def _prepare_weights(case, seed):
    g = _gen(seed)
    lens = _ints(case["lens"])
    H, Hq, n, B = case["kv_heads"], case["heads"], case["rows"], len(lens)
    blocks = [(L + PAGE - 1) // PAGE for L in lens]
    mb = max(blocks) + case["spare"]
    pages = B * mb
    rb = D // 2 if case["fmt"] == "int4" else D
    k_codes = torch.zeros((pages, H, PAGE, rb), dtype=torch.uint8, device="cuda")
    k_scales = torch.zeros((pages, H), dtype=torch.float32, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(B, mb)
    hot = torch.ones((H, D), device="cuda").scatter_(1, torch.randint(0, D, (H, 4), generator=g, device="cuda"), 10.0)
    for b, L in enumerate(lens):
        x = torch.randn((blocks[b], H, PAGE, D), generator=g, device="cuda") * hot[:, None, :]
        x = x.half().float()
        if L % PAGE:
            x[-1, :, L % PAGE:] = 0.0  # the open page's unused rows hold zero
        codes, scales = _quantize(case["fmt"], x)
        at = table[b, :blocks[b]].long()
        k_codes[at] = codes
        k_scales[at] = scales
    total = B * n
    before = torch.rand((B, mb), generator=g, device="cuda") * 2.0
    before *= torch.arange(mb, device="cuda") < torch.tensor(blocks, device="cuda")[:, None]
    return {"op": "weights", "fmt": case["fmt"], "k_codes": k_codes, "k_scales": k_scales,
            "v_codes": torch.zeros_like(k_codes), "v_scales": torch.zeros_like(k_scales),
            "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "rows": n,
            "cu": torch.arange(0, total + 1, n, dtype=torch.int32, device="cuda"),
            "q": _rows(g, total, Hq, False).half(), "scale": 1.0 / math.sqrt(D), "decay": case["decay"],
            "before": before, "after": torch.zeros_like(before),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_evict(case, seed):
    g = _gen(seed)
    blocks = _ints(case["blocks"])
    B, mb = len(blocks), max(blocks) + case["spare"]
    table = torch.randperm(B * mb, generator=g, device="cuda").to(torch.int32).view(B, mb)
    nb = torch.tensor(blocks, device="cuda")
    open_rows = torch.randint(1, PAGE + 1, (B,), generator=g, device="cuda")
    # attention weight decays as a power over a page's rank and lies anywhere in the sequence
    w = torch.rand((B, mb), generator=g, device="cuda").pow(-0.7) * 0.01
    w *= torch.arange(mb, device="cuda") < nb[:, None]
    return {"op": "evict", "table": table, "lens": ((nb - 1) * PAGE + open_rows).to(torch.int32), "weights": w,
            "keep": (nb * case["keep"]).ceil().to(torch.int32), "sink": case["sink"], "recent": case["recent"],
            "table_out": torch.zeros_like(table), "lens_out": torch.zeros(B, dtype=torch.int32, device="cuda"),
            "weights_out": torch.zeros_like(w), "evicted": torch.zeros(B, dtype=torch.int32, device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    return {"prompt": _prepare_prompt, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu_host"]
    Hq, H = q.shape[1], k.shape[1]
    g = Hq // H
    for a, z in zip(cu[:-1], cu[1:]):
        n = z - a
        kk = k[a:z].float().permute(1, 2, 0)  # [H][128][n]
        vv = v[a:z].float().permute(1, 0, 2)  # [H][n][128]
        step = max(128, (1 << 29) // (Hq * n))  # query rows whose scores are held at once
        for i in range(0, n, step):
            e = min(n, i + step)
            qq = q[a + i:a + e].float().view(e - i, H, g, D).permute(1, 2, 0, 3).reshape(H, g * (e - i), D)
            x = torch.matmul(qq, kk[:, :, :e]).view(H, g, e - i, e) * s["scale"]
            late = torch.arange(e, device=q.device)[None, :] > torch.arange(i, e, device=q.device)[:, None]
            x.masked_fill_(late, -math.inf)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - m)
            t = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(H, g * (e - i), e), vv[:, :e]).view(H, g, e - i, D) / t
            s["out"][a + i:a + e] = o.permute(2, 0, 1, 3).reshape(e - i, Hq, D).to(q.dtype)
            if s["lse"] is not None:
                s["lse"][a + i:a + e] = (m + torch.log(t))[..., 0].permute(2, 0, 1).reshape(e - i, Hq)
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _widen(fmt, codes):
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).float()
    if fmt == "int8":
        return codes.view(torch.int8).float()
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return ((pair ^ 8).to(torch.int8) - 8).float()


def _plain_weights(s):
    B, mb = s["table"].shape
    H, Hq, n = s["k_codes"].shape[1], s["q"].shape[1], s["rows"]
    g = Hq // H
    at = s["table"].long()
    k = _widen(s["fmt"], s["k_codes"][at]) * s["k_scales"][at][..., None, None]  # [B][mb][H][64][128]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, H, mb * PAGE, D)
    q = s["q"].float().view(B, n, H, g, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * g, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, H, n, g, mb * PAGE) * s["scale"]
    pos = s["lens"][:, None] - n + torch.arange(n, device=at.device)  # [B][n]
    late = torch.arange(mb * PAGE, device=at.device) > pos[..., None]
    x.masked_fill_(late[:, None, :, None, :], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    s["after"].copy_(s["decay"] * s["before"] + p.view(B, H * n * g, mb, PAGE).sum((1, 3)))
    return {"weights": s["after"]}


def _plain_evict(s):
    B, mb = s["table"].shape
    j = torch.arange(mb, device="cuda").expand(B, mb)
    nb = ((s["lens"] + PAGE - 1) // PAGE)[:, None]
    valid = j < nb
    safe = valid & ((j < s["sink"]) | (j >= nb - max(s["recent"], 1)))
    keep = torch.maximum(s["keep"][:, None].long(), safe.sum(1, keepdim=True)).minimum(nb)
    w = torch.where(s["weights"].isnan(), -math.inf, s["weights"])  # a NaN counts as the least weight
    by_weight = torch.sort(w, dim=1, descending=True, stable=True).indices
    rank_class = torch.where(safe, 0, torch.where(valid, 1, 2)).gather(1, by_weight)
    order = by_weight.gather(1, torch.sort(rank_class, dim=1, stable=True).indices)  # protected, then by weight
    kept = torch.zeros_like(valid).scatter_(1, order, j < keep)
    new = torch.sort(torch.where(kept, 0, torch.where(valid, 2, 1)), dim=1, stable=True).indices  # kept, spare, freed
    gone = (nb - keep).to(torch.int32)[:, 0]
    s["table_out"].copy_(s["table"].gather(1, new))
    s["weights_out"].copy_(torch.where(j < keep, s["weights"].gather(1, new), 0.0))
    s["lens_out"].copy_(s["lens"] - PAGE * gone)
    s["evicted"].copy_(gone)
    return {"table": s["table_out"], "lens": s["lens_out"], "weights": s["weights_out"], "evicted": s["evicted"]}


def _cache(s, kvq):
    """The cache's descriptor, which a user's program keeps beside its buffers."""
    if "cache" not in s:
        s["cache"] = kvq.PagedKVCache.over(FMT[s["fmt"]], s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"],
                                           status=s["status"])
    return s["cache"]


def _own_prompt(s, kvq):
    kvq.kvq_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["max"], s["scale"], s["out"], lse=s["lse"],
                             status=s["status"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _own_weights(s, kvq):
    cache = _cache(s, kvq)
    if "workspace" not in s:
        s["workspace"] = kvq.page_weights_workspace(s["q"].shape[0], s["q"].shape[1], s["table"].shape[1])
    kvq.kvq_page_weights(cache, s["q"], s["cu"], s["rows"], s["table"], s["lens"], s["scale"], s["decay"],
                         s["before"], s["after"], s["workspace"])
    return {"weights": s["after"]}


def _own_evict(s, kvq):
    kvq.kvq_evict_pages(s["table"], s["lens"], s["weights"], s["keep"], s["sink"], s["recent"],
                        s["table_out"], s["lens_out"], s["weights_out"], s["evicted"], status=s["status"])
    return {"table": s["table_out"], "lens": s["lens_out"], "weights": s["weights_out"], "evicted": s["evicted"]}


def run(state):
    if own:
        from quantized_kv_cache_09_gb300 import kvq
        return {"prompt": _own_prompt, "weights": _own_weights, "evict": _own_evict}[state["op"]](state, kvq)
    return {"prompt": _plain_prompt, "weights": _plain_weights, "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "prompt":
        lens, H, Hq = _ints(case["lens"]), case["kv_heads"], case["heads"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        rows = sum(lens)
        return {"bytes": rows * D * 2 * (2 * Hq + 2 * H) + (4 * rows * Hq if case["lse"] else 0) + 4 * len(lens),
                "flops": 4 * D * Hq * pairs}
    if case["op"] == "weights":
        lens, H, Hq, n = _ints(case["lens"]), case["kv_heads"], case["heads"], case["rows"]
        pages = sum((L + PAGE - 1) // PAGE for L in lens)
        row = D // 2 if case["fmt"] == "int4" else D
        pairs = sum(n * L - n * (n - 1) // 2 for L in lens)
        return {"bytes": sum(lens) * H * row + pages * (4 * H + 4 + 8) + len(lens) * n * Hq * D * 2,
                "flops": 2 * D * Hq * pairs}
    blocks = _ints(case["blocks"])
    rows = len(blocks) * (max(blocks) + case["spare"])
    return {"bytes": rows * 8 + sum(blocks) * 4 + rows * 4 + len(blocks) * 16, "flops": sum(blocks)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_prompt(case, s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu_host"]
    g = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for a, z in zip(cu[:-1], cu[1:]):
        for h in range(q.shape[1]):
            kh, vh = k[a:z, h // g].double(), v[a:z, h // g].double()
            for i in range(0, z - a, 2048):
                e = min(z - a, i + 2048)
                x = s["scale"] * (q[a + i:a + e, h].double() @ kh[:e].T)
                x = x + torch.full_like(x, -math.inf).triu(i + 1)
                t = torch.logsumexp(x, 1)
                out[a + i:a + e, h] = torch.exp(x - t[:, None]) @ vh[:e]
                lse[a + i:a + e, h] = t
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_weights(case, s):
    H, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    n = case["rows"]
    res = torch.zeros(s["before"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(_ints(case["lens"])):
        nb = (L + PAGE - 1) // PAGE
        raw = s["k_codes"][s["table"][b, :nb].long()]
        if case["fmt"] == "int4":
            x = raw.to(torch.int64)
            val = torch.empty(raw.shape[:-1] + (D,), dtype=torch.float64, device="cuda")
            val[..., 0::2], val[..., 1::2] = (x + 8) % 16 - 8, (x // 16 + 8) % 16 - 8
        elif case["fmt"] == "int8":
            x = raw.to(torch.int64)
            val = torch.where(x > 127, x - 256, x).double()
        else:
            val = raw.view(torch.float8_e4m3fn).double()
        val *= s["k_scales"][s["table"][b, :nb].long()].double()[:, :, None, None]
        q = s["q"][b * n:(b + 1) * n].double().view(n, H, g, D)
        x = s["scale"] * torch.einsum("nhgd,phtd->nhgpt", q, val).reshape(n, H, g, nb * PAGE)
        for i in range(n):
            x[i, :, :, L - n + i + 1:] = -math.inf
        w = torch.softmax(x, -1).sum((0, 1, 2)).view(nb, PAGE).sum(1)
        res[b, :nb] = case["decay"] * s["before"][b, :nb].double() + w
    return {"weights": res}


def _exact_evict(case, s):
    table, w = s["table"].cpu().numpy(), s["weights"].double().cpu().numpy()
    lens, keep = s["lens"].cpu().numpy().copy(), s["keep"].cpu().numpy()
    new, left, gone = table.copy(), np.zeros_like(w), np.zeros_like(lens)
    for b, nb in enumerate(_ints(case["blocks"])):
        last = max(case["recent"], 1)
        safe = [i for i in range(nb) if i < case["sink"] or i >= nb - last]
        rest = [i for i in range(nb) if case["sink"] <= i < nb - last]
        room = max(0, min(int(keep[b]), nb) - len(safe))
        rest.sort(key=lambda i: (-w[b, i], i))
        stay, go = sorted(safe + rest[:room]), sorted(rest[room:])
        new[b] = table[b, stay + list(range(nb, table.shape[1])) + go]
        left[b, :len(stay)] = w[b, stay]
        gone[b] = len(go)
        lens[b] -= PAGE * len(go)
    return {"table": torch.from_numpy(new), "lens": torch.from_numpy(lens), "weights": torch.from_numpy(left),
            "evicted": torch.from_numpy(gone)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, s)
