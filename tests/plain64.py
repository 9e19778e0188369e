"""Plain 64-bit forms of prompt attention, page weights and page eviction,
written from their definitions, with the error bounds the tests hold the
kernels to.

Half a rounding step is u = eps / 2 relative to the value (fp16 2^-11, bf16
2^-8, fp32 2^-24).  GAMMA counts the binary32 accumulation of a 128-element dot
product on the tensor cores: at most 16 additions of partial sums, each within
2^-23 of the sum of magnitudes (the tensor cores may truncate, a full step)."""
import math

import torch

D = 128
PAGE = 64
GAMMA = 16 * 2.0 ** -23
EXP2 = 2.0 ** -21    # ex2.approx (2^-22), and the rounding of its argument's scale
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def prompt(q, k, v, cu, scale):
    """(out, lse, out's bound, lse's bound) in float64; rows outside every sequence are NaN."""
    T, Hq, _ = q.shape
    g = Hq // k.shape[1]
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=q.device)
    tol, tol_lse = out.clone(), lse.clone()
    u = U[q.dtype]
    for a, z in zip(cu[:-1], cu[1:]):
        n = z - a
        if n == 0:
            continue
        seen = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        for h in range(Hq):
            x, y, w = q[a:z, h].double(), k[a:z, h // g].double(), v[a:z, h // g].double()
            s = (x @ y.T * scale).masked_fill(~seen, -math.inf)
            mag = (x.abs() @ y.abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(1, keepdim=True)
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            tot = p.sum(1, keepdim=True)
            out[a:z, h] = p @ w / tot
            lse[a:z, h] = (m + torch.log(tot))[:, 0]
            # a score is off by GAMMA of its magnitudes and by one rounding of its scaled value
            err = GAMMA * mag + 2.0 ** -23 * (mag + s.masked_fill(~seen, 0.0).abs().amax(1, keepdim=True)) + EXP2
            err_l = err + n * 2.0 ** -24
            avg = p @ w.abs() / tot
            # P as an operand: u of its value, or (fp16) half the subnormal step 2^-25 beside a largest P >= 1
            low = 2.0 ** -25 * w.abs().cumsum(0) if q.dtype == torch.float16 else 0.0
            bound = (u + err + err_l + n * 2.0 ** -23) * avg + low
            tol[a:z, h] = 1.01 * (bound + u * (out[a:z, h].abs() + bound)) + 2.0 ** -24
            tol_lse[a:z, h] = 1.01 * (err_l + 2.0 ** -22 * (1 + lse[a:z, h:h + 1].abs()))[:, 0]
    return out, lse, tol, tol_lse


def widen(fmt, codes):
    """The values codes stand for (before the scale): fmt 0 int4, 1 int8, 2 FP8 E4M3."""
    if fmt == 2:
        return codes.view(torch.float8_e4m3fn).double()
    x = codes.to(torch.int64)
    if fmt == 1:
        return torch.where(x > 127, x - 256, x).double()
    out = torch.empty(codes.shape[:-1] + (D,), dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = (x + 8) % 16 - 8, (x // 16 + 8) % 16 - 8
    return out


def page_weights(fmt, k_codes, k_scales, q, cu, table, lens, scale, decay, before):
    """(weights, bound) in float64, as kvq_page_weights defines them."""
    B, mb = table.shape
    H, Hq = k_codes.shape[1], q.shape[1]
    g = Hq // H
    res = torch.zeros((B, mb), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(res)
    for b in range(B):
        L, n = lens[b], cu[b + 1] - cu[b]
        nb = (L + PAGE - 1) // PAGE
        old = torch.zeros(nb, dtype=torch.float64, device=q.device) if before is None else before[b, :nb].double()
        if n == 0:
            res[b, :nb] = old
            continue
        at = table[b, :nb].long()
        c, sk = widen(fmt, k_codes[at]), k_scales[at].double()
        new = torch.zeros(nb, dtype=torch.float64, device=q.device)
        err_new = torch.zeros_like(new)
        pos = L - n + torch.arange(n, device=q.device)
        late = torch.arange(nb * PAGE, device=q.device)[None, :] > pos[:, None]
        for h in range(Hq):
            x = q[cu[b]:cu[b + 1], h].double()
            raw = torch.einsum("nd,ptd->npt", x, c[:, h // g])
            # int4 codes enter shifted by up to 8, which comes out afterwards
            mag = torch.einsum("nd,ptd->npt", x.abs(), c[:, h // g].abs() + (8 if fmt == 0 else 0))
            s = (raw * sk[:, h // g, None] * scale).reshape(n, -1).masked_fill(late, -math.inf)
            d = (2 * GAMMA * mag * sk[:, h // g, None] * abs(scale)).reshape(n, -1).masked_fill(late, 0.0)
            err = d.amax(1) + 2.0 ** -22 * s.masked_fill(late, 0.0).abs().amax(1) + 4 * EXP2 + nb * 2.0 ** -24
            w = torch.softmax(s, 1).view(n, nb, PAGE).sum(2)
            new += w.sum(0)
            # numerator and denominator
            err_new += (2 * err[:, None] * w).sum(0)
        res[b, :nb] = decay * old + new
        rows = n * Hq
        tol[b, :nb] = 1.01 * (err_new + rows * 2.0 ** -24 * new) + 2.0 ** -22 * (res[b, :nb].abs() + abs(decay) * old.abs())
        tol[b, :nb] += rows * 2.0 ** -120  # a page whose mass binary32 cannot hold
    return res, tol


def evict(table, lens, weights, keep, sink, recent):
    """(table, lens, weights, evicted) as lists of rows, as kvq_evict_pages defines them."""
    T, Ls, W, gone = [], [], [], []
    for row, L, w, kb in zip(table, lens, weights, keep):
        nb, mb = (L + PAGE - 1) // PAGE, len(row)
        last = max(recent, 1)
        safe = [j for j in range(nb) if j < sink or j >= nb - last]
        rest = [j for j in range(nb) if sink <= j < nb - last]
        room = max(0, min(kb, nb) - len(safe))
        rest.sort(key=lambda j: (-w[j] if w[j] == w[j] else math.inf, j))  # a NaN: the least weight
        stay, go = sorted(safe + rest[:room]), sorted(rest[room:])
        T.append([row[j] for j in stay + list(range(nb, mb)) + go])
        W.append([w[j] for j in stay] + [0.0] * (mb - len(stay)))
        gone.append(len(go))
        Ls.append(L - PAGE * len(go))
    return T, Ls, W, gone
