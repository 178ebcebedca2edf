"""The serving operators' definitions in 64 bits (torch double, on the tensors' device), and the error bounds that the
kernels' arithmetic allows.

Bounds.  u = torch.finfo(dtype).eps / 2 is a rounding's relative error.  With w_j the softmax weights, A = sum_j w_j |v_j|
(per channel), and e_s the largest error of a score:
  |o - o*| <= u |o*| + (u_P + 2 e_s + (n + 16) 2^-23) A + abs_P
  |lse - lse*| <= e_s + (n + 16) 2^-23 + 2^-22 |lse*|
u_P is P's rounding before the product with V (numerator only; the row sum is of the unrounded values, or of the same
rounded ones, which changes the quotient by at most another u_P: callers pass the sum).  Sums over n keys are fp32 with
at most n roundings of 2^-24; 16 more steps of 2^-23 cover the exponential, its argument's products, and the quotient.
e_s = (d + 16) 2^-23 S with S = max_j scale sum_c |q_c k_jc|: d products summed in fp32, in any order, by hardware that may
truncate (2^-23 a step), and the argument's own rounding, whose size |s| is at most S.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def softmax_row(s, v):
    """s [r, n], v [n, d] double -> o, lse, A; empty rows give 0, -inf."""
    if s.shape[1] == 0:
        z = torch.zeros((s.shape[0], v.shape[1]), dtype=torch.float64, device=s.device)
        return z, torch.full((s.shape[0],), -math.inf, dtype=torch.float64, device=s.device), z.clone()
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    v0 = torch.nan_to_num(v, 0, 0, 0)  # a weight of 0 has masked the key: what it holds does not count
    bad = ~torch.isfinite(v)
    o = w @ v0
    if bad.any():
        hit = ((w > 0).double() @ bad.double()) > 0
        o = torch.where(hit, torch.full_like(o, math.nan), o)
    return o, lse, w @ v0.abs()


def prompt(q, k, v, q_offsets, kv_offsets, causal, scale=None):
    """-> out, lse (double), tolerance of each; rows of no sequence are NaN."""
    Tq, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    u = U[q.dtype]
    out = torch.full((Tq, Hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, Tq), math.nan, dtype=torch.float64, device=q.device)
    tol_o, tol_l = out.clone(), lse.clone()
    for b in range(len(q_offsets) - 1):
        a, e, c, f = q_offsets[b], q_offsets[b + 1], kv_offsets[b], kv_offsets[b + 1]
        n, m = e - a, f - c
        if n == 0:
            continue
        hide = None
        if causal:
            i, j = torch.arange(n, device=q.device), torch.arange(m, device=q.device)
            hide = j[None, :] > (i + m - n)[:, None]
        for h in range(Hq):
            qh, kh, vh = q[a:e, h].double(), k[c:f, h // G].double(), v[c:f, h // G].double()
            s = qh @ kh.T * scale
            big = qh.abs() @ kh.abs().T * scale
            if hide is not None:
                s = s.masked_fill(hide, -math.inf)
                big = big.masked_fill(hide, 0.0)
            o, l, A = softmax_row(s, vh)
            out[a:e, h], lse[h, a:e] = o, l
            es = (d + 16) * 2.0 ** -23 * (big.amax(1) if m else torch.zeros(n, dtype=torch.float64, device=q.device))
            es = torch.nan_to_num(es, 0, 0, 0)
            rel = u + 2 * es + (m + 16) * 2.0 ** -23
            tol_o[a:e, h] = u * o.abs() + rel[:, None] * A
            tol_l[h, a:e] = es + (m + 16) * 2.0 ** -23 + 2.0 ** -22 * l.abs()
    return out, lse, tol_o, tol_l


def close(got, want, tol, what=""):
    """Every finite value within its tolerance (half of the smallest subnormal of fp16 besides), the others alike."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN where there should be none, or the reverse"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities differ"
    if fine.any():
        over = (got[fine] - want[fine]).abs() - tol[fine] - 2.0 ** -25
        assert float(over.max()) <= 0, (f"{what}: {float(over.max()):.3e} over the tolerance; worst error "
                                        f"{float((got[fine] - want[fine]).abs().max()):.3e}")


def e4m3(x):
    """Nearest E4M3 value, ties to even, saturating, of a double tensor (NaN stays)."""
    ax = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.frexp(torch.nan_to_num(ax, 1.0, 1e300))[1].double() - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exponent(top):
    """Smallest e in [-127, 127] with top <= 448 2^e (double tensor; 0 gives -127)."""
    m, e = torch.frexp(top / 448)
    return torch.where(top > 0, e - (m == 0.5).int(), torch.full_like(e, -127)).clamp(-127, 127).double()


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def store(x, codes, exps, table, offsets, held):
    """-> values [pages, Hkv, page, d] (double), exponent bytes after storing; lists for table, offsets and held."""
    page = codes.shape[2]
    val, exps, x = values(codes), exps.clone(), x.double()
    for b in range(len(held)):
        pos, end, src = held[b], held[b] + offsets[b + 1] - offsets[b], offsets[b]
        while pos < end:
            n = min(end, (pos // page + 1) * page) - pos
            pg, slot = table[b][pos // page], pos % page
            new = x[src:src + n].transpose(0, 1)
            top = torch.nan_to_num(new.abs(), 0.0).amax((1, 2))
            e = exponent(top)
            if slot:
                old = exps[pg].double() - 127
                e = torch.maximum(e, old)
                val[pg, :, :slot] = torch.where((e > old)[:, None, None],
                                                e4m3(val[pg, :, :slot] * torch.exp2(old - e)[:, None, None]),
                                                val[pg, :, :slot])
            val[pg, :, slot:slot + n] = e4m3(new * torch.exp2(-e)[:, None, None])
            exps[pg] = (e + 127).to(torch.uint8)
            pos, src = pos + n, src + n
    return val, exps


def cached(val, exps, pages, n):
    """Keys or values [Hkv, n, d] of a sequence from page values and exponent bytes."""
    x = val[pages] * torch.exp2(exps[pages].double() - 127)[:, :, None, None]
    return x.transpose(0, 1).reshape(val.shape[1], -1, val.shape[3])[:, :n]


def attend(q, k_codes, v_codes, k_exps, v_exps, table, lens, scale=None):
    """-> out, lse, tolerances.  P' = p 2^(ev - EV) 32 (p relative to a base no more than 2^3 below the maximum, EV the
    largest exponent so far) as three E4M3 parts, each rest scaled by 16: relative error 2^-4 a part, 2^-12 in all, and
    half of E4M3's subnormal step, 2^-10, of the third part's unit, 2^-8 / 32: 2^-23 of a weight of 1 at the scale 2^EV.
    Q: two (bf16) or three (fp16) parts of q scaled so that the largest element lies in (224, 448]: 8 and 11 significant
    bits fit; smaller elements have 2^-10 of 224: 2^-17 of the row's largest."""
    B, Hq, d = q.shape
    Hkv, page = k_codes.shape[1], k_codes.shape[2]
    G, u = Hq // Hkv, U[q.dtype]
    u_p = 2.0 ** -12
    scale = scale or 1.0 / math.sqrt(d)
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    kv, vv = values(k_codes), values(v_codes)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        pages = torch.as_tensor(table[b][:-(-n // page)], dtype=torch.long, device=q.device)
        k, v = cached(kv, k_exps, pages, n), cached(vv, v_exps, pages, n)
        ev = v_exps[pages].double()  # [pages, Hkv]
        up = torch.exp2(ev.amax(0)[None, :] - ev).repeat_interleave(page, 0)[:n].T  # [Hkv, n]: 2^(EV - ev)
        for h in range(Hq):
            g = h // G
            qh = q[b, h].double()
            s = (qh @ k[g].T) * scale
            o, l, A = softmax_row(s[None], v[g])
            S = float((qh.abs() @ k[g].abs().T).max()) * scale
            es = (2 * d + 16) * 2.0 ** -23 * S + 2.0 ** -17 * float(qh.abs().max()) * float(k[g].abs().sum(1).max()) * scale
            top = float(torch.exp(s.max() - l[0]))  # the weight that p = 1 stands for
            lost = 2.0 ** -23 * top * (up[g][:, None] * v[g].abs()).sum(0)
            out[b, h], lse[b, h] = o[0], l[0]
            tol_o[b, h] = u * o[0].abs() + (u_p + 2 * es + (n + 64) * 2.0 ** -23) * A[0] + lost
            tol_l[b, h] = es + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * l[0].abs()
    return out, lse, tol_o, tol_l
