"""Performance cases of the serving operators: attention over packed prompts, storing
keys and values in the 8-bit paged cache, and single-token attention over that cache.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU, `run()` one
pass: with `own` set through the library's entry points, otherwise through the plain
form below (elementary torch operations in 32 bits).  `exact()` is the operators'
definition in 64 bits, `work()` what one pass cannot do without.

Definitions.  A prompt batch packs B sequences along the token axis, sequence b's
queries at q_offsets[b] .. q_offsets[b + 1] and its keys at kv_offsets[b] ..; query i of
n sees key j of m when (causal) j <= i + m - n; head h reads key head h // (Hq / Hkv).

The cache holds E4M3 codes [pages, Hkv, page, d] and one exponent byte e + 127 for each
(page, key head): a value is code * 2^e with e the smallest integer whose 448 * 2^e
reaches the largest magnitude stored in that page and head.  Storing tokens behind
others of a page keeps the page's exponent or raises it; raised, the codes that are
there are rounded again to the new exponent.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One short question to a chat model: a call where latency counts.
        dict(name="prompt_short", op="prompt", q_lens="77", kv_lens="", Hq=8, Hkv=8, d=64, dtype="bf16", causal=True, pad=0),
        # A prefill batch of a serving loop: ragged prompts packed together, rows left over behind the last.
        dict(name="prompt_packed", op="prompt", q_lens="1300,1,517,2048,129,33,900,64,1777,255,800,5", kv_lens="", Hq=32, Hkv=8,
             d=128, dtype="bf16", causal=True, pad=43),
        # One long document, 40 heads of 128 (the video transformer's heads and length, here causal and grouped).
        dict(name="prompt_long", op="prompt", q_lens="32760", kv_lens="", Hq=40, Hkv=8, d=128, dtype="bf16", causal=True, pad=0),
        # Prefill in chunks: the queries are the newest 512 (or fewer) tokens of longer contexts.
        dict(name="prompt_chunk", op="prompt", q_lens="512,512,301,512", kv_lens="8192,4608,301,16000", Hq=32, Hkv=8, d=128,
             dtype="bf16", causal=True, pad=0),
        # Bidirectional attention over ragged sequences, one key head for each query head, 64 channels, fp16.
        dict(name="prompt_fp16_d64", op="prompt", q_lens="4095,1000,2049,63", kv_lens="", Hq=24, Hkv=24, d=64, dtype="fp16",
             causal=False, pad=0),
        # A prefill batch's keys and values stored in the cache.
        dict(name="store_prompts", op="store", q_lens="8192,1,4097,16384,300,3500", held="0,0,77,0,1000,64", Hkv=8, d=128, page=64,
             dtype="bf16"),
        # One decode step of 64 sequences stored: each token joins others in its page.
        dict(name="store_tokens", op="store", q_lens=",".join(["1"] * 64), held=",".join(str(37 * i + 5) for i in range(64)), Hkv=8,
             d=128, page=64, dtype="bf16"),
        # One sequence decoding: latency.
        dict(name="decode_one", op="decode", lens="1000", Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # A serving batch: 64 sequences from a fresh one to long ones.
        dict(name="decode_batch", op="decode", lens=",".join(str(1 + (i * i * 2 + 131 * i) % 8192) for i in range(64)), Hq=32, Hkv=8,
             d=128, page=64, dtype="bf16"),
        # Two long contexts: little to share out by sequence, much along it.
        dict(name="decode_long", op="decode", lens="131071,100003", Hq=64, Hkv=8, d=128, page=128, dtype="bf16"),
        # Ungrouped heads of 64 channels, small pages, fp16.
        dict(name="decode_fp16_d64", op="decode", lens=",".join(str(400 + 97 * i) for i in range(16)), Hq=24, Hkv=24, d=64, page=16,
             dtype="fp16"),
        # A decode step of one layer as a server runs it: store the step's tokens, then attend.
        dict(name="step_batch", op="step", lens=",".join(str(64 + 53 * i) for i in range(48)), Hq=32, Hkv=4, d=128, page=32,
             dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "store", "decode", "step"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 24])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        G = rng.choice([1, 2, 3, 4, 5, 8])
        B = _spread(rng, 1, 12)
        total = _spread(rng, max(16, B), 8000)
        q = [max(1, int(total / B * rng.uniform(0.05, 1.95))) for _ in range(B)]
        kv = ""
        if rng.random() < 0.4:
            kv = ",".join(str(max(1, n + rng.choice([-1, 1, 1, 1]) * _spread(rng, 1, 4000))) for n in q)
        return dict(op=op, q_lens=",".join(map(str, q)), kv_lens=kv, Hq=G * Hkv, Hkv=Hkv, d=d, dtype=dtype,
                    causal=rng.random() < 0.75, pad=rng.choice([0, 0, 19]))
    if op == "store":
        B = _spread(rng, 1, 64)
        total = _spread(rng, B, 30000)
        q = [1] * B if rng.random() < 0.4 else [max(1, int(total / B * rng.uniform(0.05, 1.95))) for _ in range(B)]
        held = [rng.choice([0, _spread(rng, 1, 4000)]) for _ in range(B)]
        return dict(op=op, q_lens=",".join(map(str, q)), held=",".join(map(str, held)), Hkv=Hkv, d=d, page=page, dtype=dtype)
    G = rng.choice([1, 2, 4, 5, 8, 16])
    B = _spread(rng, 1, 64)
    top = _spread(rng, 64, 200000 // B)
    lens = [max(1, int(top * rng.uniform(0.02, 1.0))) for _ in range(B)]
    return dict(op=op, lens=",".join(map(str, lens)), Hq=G * Hkv, Hkv=Hkv, d=d, page=page, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _ints(text):
    return [int(x) for x in text.split(",")]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _keys(g, tokens, Hkv, d, dtype):
    """Keys with the few strong channels that real projections show, values with tokens of different strength."""
    k = torch.randn((tokens, Hkv, d), generator=g, device="cuda")
    k *= 1.0 + 3.0 * (torch.rand((1, Hkv, d), generator=g, device="cuda") < 0.03)
    v = torch.randn((tokens, Hkv, d), generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn((tokens, 1, 1), generator=g, device="cuda"))
    return k.to(dtype), v.to(dtype)


def _pages_of(lens, page, g):
    """A shuffled block table over a pool with a few spare pages; -1 behind a sequence's last page."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pool, table


def _rows_to_pages(lens, page, table):
    """(page, slot) of each token of sequences of these lengths, packed."""
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    return table[seq, pos // page].long(), pos % page


def _cache(g, held, lens, Hkv, d, page, dtype):
    """A cache that holds `held` tokens of sequences whose pages reach to `lens`: codes, exponents, block table.
    Slots that hold no token, and exponents of pages that hold none, are arbitrary bytes."""
    pool, table = _pages_of(lens, page, g)
    shape = (pool, Hkv, page, d)
    kc = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    vc = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    ke = torch.randint(100, 150, (pool, Hkv), generator=g, device="cuda", dtype=torch.uint8)
    ve = torch.randint(100, 150, (pool, Hkv), generator=g, device="cuda", dtype=torch.uint8)
    if sum(held):
        k, v = _keys(g, sum(held), Hkv, d, dtype)
        pg, slot = _rows_to_pages(held, page, table)
        used = torch.zeros(pool, dtype=torch.bool, device="cuda")
        used[pg] = True
        for x, codes, exps in ((k, kc, ke), (v, vc, ve)):
            e = _exponent(torch.zeros((pool, Hkv), device="cuda").index_reduce_(0, pg, x.float().abs().amax(2), "amax"))
            exps[used] = (e[used] + 127).to(torch.uint8)
            codes[pg, :, slot] = _encode(x.float(), e[pg].unsqueeze(2))
    return dict(kc=kc, vc=vc, ke=ke, ve=ve, table=table)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dtype, d, Hkv = DTYPES[case["dtype"]], case["d"], case["Hkv"]
    st = dict(case)
    if case["op"] == "prompt":
        q_lens = _ints(case["q_lens"])
        kv_lens = _ints(case["kv_lens"]) if case["kv_lens"] else q_lens
        Tq, Tkv, pad = sum(q_lens), sum(kv_lens), case["pad"]
        st["q"] = _normal(g, (Tq + pad, case["Hq"], d), dtype, 1.5)
        st["k"], st["v"] = _keys(g, Tkv + pad, Hkv, d, dtype)
        if pad:  # rows that belong to no sequence hold anything
            st["k"][Tkv:] = float("nan")
            st["v"][Tkv:] = float("inf")
        st["q_offsets"], st["kv_offsets"] = _i32(_offsets(q_lens)), _i32(_offsets(kv_lens))
        st["out"] = torch.zeros((Tq + pad, case["Hq"], d), dtype=dtype, device="cuda")
        st["lse"] = torch.zeros((case["Hq"], Tq + pad), dtype=torch.float32, device="cuda")
        return st
    page = case["page"]
    if case["op"] == "store":
        n, held = _ints(case["q_lens"]), _ints(case["held"])
    else:
        total = _ints(case["lens"])
        n = [1] * len(total) if case["op"] == "step" else [0] * len(total)
        held = [t - k for t, k in zip(total, n)]
    lens = [a + b for a, b in zip(held, n)]
    st.update(_cache(g, held, lens, Hkv, d, page, dtype))
    if sum(n):  # the tokens to store behind those
        st["k"], st["v"] = _keys(g, sum(n), Hkv, d, dtype)
        st["offsets"], st["held_lens"] = _i32(_offsets(n)), _i32(held)
    if case["op"] != "store":
        st["q"] = _normal(g, (len(lens), case["Hq"], d), dtype, 1.5)
        st["lens_t"] = _i32(lens)
        st["out"] = torch.zeros((len(lens), case["Hq"], d), dtype=dtype, device="cuda")
        st["lse"] = torch.zeros((len(lens), case["Hq"]), dtype=torch.float32, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["op"]
    if own:
        from mxfp4_microscaled_quantization_b200 import mxattn as mx

        if op == "prompt":
            return mx.mxattn_prompt(st["q"], st["k"], st["v"], st["q_offsets"], st["kv_offsets"], causal=st["causal"],
                                    out=st["out"], lse=st["lse"])
        cache = (st["kc"], st["vc"], st["ke"], st["ve"], st["table"])
        if op in ("store", "step"):
            mx.mxattn_cache_store(st["k"], st["v"], *cache, st["offsets"], st["held_lens"])
        if op in ("decode", "step"):
            o = mx.mxattn_cache_attend(st["q"], *cache, st["lens_t"], out=st["out"], lse=st["lse"])
        if op == "decode":
            return o
        held = [st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn), st["ke"], st["ve"]]
        return held if op == "store" else [*o, *held]
    if op == "prompt":
        return _plain_prompt(st)
    if op in ("store", "step"):
        _plain_store(st, st["k"], st["kc"], st["ke"])
        _plain_store(st, st["v"], st["vc"], st["ve"])
    if op in ("decode", "step"):
        o = _plain_decode(st)
    if op == "decode":
        return o
    held = [st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn), st["ke"], st["ve"]]
    return held if op == "store" else [*o, *held]


# ------------------------------------------------------------------ the plain form

def _plain_prompt(st):
    """Softmax of all scores of the packed batch, those of other sequences and later keys left out.  The scores of a
    few heads at a time where all of them would not fit."""
    q, k, v, qo, ko = st["q"], st["k"], st["v"], st["q_offsets"].long(), st["kv_offsets"].long()
    Hq, Hkv, d = st["Hq"], st["Hkv"], st["d"]
    Tq, Tkv = int(sum(_ints(st["q_lens"]))), int(sum(_ints(st["kv_lens"] or st["q_lens"])))
    qi, kj = torch.arange(Tq, device="cuda"), torch.arange(Tkv, device="cuda")
    qb = torch.searchsorted(qo, qi, right=True) - 1
    kb = torch.searchsorted(ko, kj, right=True) - 1
    seen = qb[:, None] == kb[None, :]
    if st["causal"]:
        seen &= (kj - ko[kb + 1])[None, :] <= (qi - qo[qb + 1])[:, None]
    G, step = Hq // Hkv, max(1, int(2 ** 32 // (max(1, Tq * Tkv) * (Hq // Hkv))))
    for h in range(0, Hkv, step):
        n = min(step, Hkv - h)
        qh = q[:Tq, h * G:(h + n) * G].float().view(Tq, n, G, d).permute(1, 2, 0, 3).reshape(n, G * Tq, d)
        s = (qh @ k[:Tkv, h:h + n].float().permute(1, 2, 0)).view(n, G, Tq, Tkv)
        s *= 1.0 / math.sqrt(d)
        s.masked_fill_(~seen, -math.inf)
        m = s.amax(3, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = s.sub_(m).exp_()
        total = p.sum(3, keepdim=True)
        o = (p.view(n, G * Tq, Tkv) @ v[:Tkv, h:h + n].float().permute(1, 0, 2)).view(n, G, Tq, d)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        st["out"][:Tq, h * G:(h + n) * G] = o.permute(2, 0, 1, 3).reshape(Tq, n * G, d).to(q.dtype)
        st["lse"][h * G:(h + n) * G, :Tq] = (m + total.log()).view(n * G, Tq)
    return st["out"], st["lse"]


def _exponent(amax):
    """The smallest e in [-127, 127] with amax <= 448 * 2^e; -127 where amax is 0."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _encode(x, e):
    return (torch.ldexp(x, -e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_store(st, x, codes, exps):
    page, table = st["page"], st["table"].long()
    off, held = st["offsets"].long(), st["held_lens"].long()
    T = x.shape[0]
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(off, i, right=True) - 1
    pos = held[b] + i - off[b]
    pg, slot = table[b, pos // page], pos % page
    amax = torch.zeros((codes.shape[0], codes.shape[1]), device="cuda").index_reduce_(0, pg, x.float().abs().amax(2), "amax")
    touched = torch.zeros(codes.shape[0], dtype=torch.bool, device="cuda")
    touched[pg] = True
    # the first page of a sequence's new tokens may hold others already, in its slots below held % page
    grown = torch.nonzero((off[1:] > off[:-1]) & (held % page > 0))[:, 0]
    gp = table[grown, held[grown] // page]
    e = _exponent(amax)
    old = exps[gp].int() - 127
    e[gp] = torch.maximum(e[gp], old)
    kept = _encode(_decode(codes[gp]), (e[gp] - old)[:, :, None, None])
    below = torch.arange(page, device="cuda")[None, :] < (held[grown] % page)[:, None]
    codes[gp] = torch.where(below[:, None, :, None], kept, codes[gp])
    codes[pg, :, slot] = _encode(x.float(), e[pg][:, :, None])
    exps[touched] = (e[touched] + 127).to(torch.uint8)


def _plain_decode(st):
    q, table, lens = st["q"], st["table"].long(), st["lens_t"].long()
    B, Hq, d = q.shape
    Hkv, page = st["Hkv"], st["page"]
    L = table.shape[1] * page
    seen = torch.arange(L, device="cuda")[None, :] < lens[:, None]
    at = table.clamp(min=0)

    def rows(codes, exps):
        scale = torch.ldexp(torch.ones((), device="cuda"), exps[at].int() - 127)
        x = _decode(codes[at]).mul_(scale[..., None, None])  # [B, pages, Hkv, page, d]
        x = x.transpose(1, 2).reshape(B, Hkv, L, d)
        return x.masked_fill_(~seen[:, None, :, None], 0.0)

    s = q.float().view(B, Hkv, Hq // Hkv, d) @ rows(st["kc"], st["ke"]).transpose(2, 3)
    s *= 1.0 / math.sqrt(d)
    s.masked_fill_(~seen[:, None, None, :], -math.inf)
    m = s.amax(3, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = (p @ rows(st["vc"], st["ve"])) / total
    st["out"].copy_(o.view(B, Hq, d))
    st["lse"].copy_((m + total.log()).view(B, Hq))
    return st["out"], st["lse"]


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_attention(q, k, v, shift):
    """One head group of one sequence: q [G, n, d], k, v [m, d]; query i sees key j <= i + shift (shift None: all)."""
    outs, lses = [], []
    for at in range(0, q.shape[1], 1024):
        s = (q[:, at:at + 1024] @ k.T) / math.sqrt(q.shape[2])
        if shift is not None:
            i = torch.arange(at, at + s.shape[1], device="cuda")
            s = s.masked_fill(torch.arange(k.shape[0], device="cuda")[None, :] > (i + shift)[:, None], -math.inf)
        lse = torch.logsumexp(s, 2)
        w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, :, None])
        outs.append(w @ v)
        lses.append(lse)
    return torch.cat(outs, 1), torch.cat(lses, 1)


def _exact_store(st, x, codes, exps):
    """Page by page: what the tokens of one sequence in one page make of it.  Values as float64, exponents untouched type."""
    page, table = st["page"], st["table"].cpu().tolist()
    val, exps = codes.view(torch.float8_e4m3fn).double(), exps.clone()
    off, held = st["offsets"].cpu().tolist(), st["held_lens"].cpu().tolist()
    x = x.double()

    def near(y):  # to the nearest E4M3 value, ties to even, by the spacing of the value's binade
        step = torch.exp2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].double() - 4)
        return (torch.round(y / step) * step).clamp(-448, 448)

    for b in range(len(held)):
        pos, end, src = held[b], held[b] + off[b + 1] - off[b], off[b]
        while pos < end:
            n = min(end, (pos // page + 1) * page) - pos
            pg, slot = table[b][pos // page], pos % page
            new = x[src:src + n].transpose(0, 1)  # [Hkv, n, d]
            top = new.abs().amax((1, 2))
            m, e = torch.frexp(top / 448)  # m * 2^e with 0.5 <= m < 1: the power of two that reaches it is 2^e, or 2^(e - 1) itself
            e = torch.where(top > 0, e - (m == 0.5).int(), -127).clamp(-127, 127).double()
            if slot:
                old = exps[pg].double() - 127
                e = torch.maximum(e, old)
                val[pg, :, :slot] = near(val[pg, :, :slot] * torch.exp2(old - e)[:, None, None])
            val[pg, :, slot:slot + n] = near(new * torch.exp2(-e)[:, None, None])
            exps[pg] = (e + 127).to(torch.uint8)
            pos, src = pos + n, src + n
    return val, exps


def exact(case, seed):
    st = prepare(case, seed)
    G = case.get("Hq", case["Hkv"]) // case["Hkv"]
    if case["op"] == "prompt":
        if sum(a * b for a, b in zip(_ints(case["q_lens"]), _ints(case["kv_lens"] or case["q_lens"]))) * case["Hq"] > 5e10:
            return None
        out, lse = st["out"].double(), st["lse"].double()
        qo, ko = st["q_offsets"].tolist(), st["kv_offsets"].tolist()
        for b in range(len(qo) - 1):
            shift = (ko[b + 1] - ko[b]) - (qo[b + 1] - qo[b]) if case["causal"] else None
            for h in range(case["Hkv"]):
                o, l = _exact_attention(st["q"][qo[b]:qo[b + 1], h * G:(h + 1) * G].double().transpose(0, 1),
                                        st["k"][ko[b]:ko[b + 1], h].double(), st["v"][ko[b]:ko[b + 1], h].double(), shift)
                out[qo[b]:qo[b + 1], h * G:(h + 1) * G] = o.transpose(0, 1)
                lse[h * G:(h + 1) * G, qo[b]:qo[b + 1]] = l
        return out, lse
    kv, vv = st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn)
    ke, ve = st["ke"], st["ve"]
    if case["op"] in ("store", "step"):
        kv, ke = _exact_store(st, st["k"], st["kc"], ke)
        vv, ve = _exact_store(st, st["v"], st["vc"], ve)
    if case["op"] == "store":
        return [kv, vv, ke, ve]
    out, lse = st["out"].double(), st["lse"].double()
    table, page = st["table"].long(), case["page"]
    for b, n in enumerate(_ints(case["lens"])):
        at = table[b, :-(-n // page)]

        def rows(val, exps):
            x = val[at].double() * torch.exp2(exps[at].double() - 127)[:, :, None, None]
            return x.transpose(0, 1).reshape(case["Hkv"], -1, case["d"])[:, :n]

        k, v = rows(kv, ke), rows(vv, ve)
        s = st["q"][b].double().view(case["Hkv"], G, -1) @ k.transpose(1, 2) / math.sqrt(case["d"])
        out[b] = (torch.softmax(s, 2) @ v).reshape(case["Hq"], -1)
        lse[b] = torch.logsumexp(s, 2).reshape(-1)
    return [out, lse] if case["op"] == "decode" else [out, lse, kv, vv, ke, ve]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "prompt":
        q = _ints(case["q_lens"])
        kv = _ints(case["kv_lens"]) if case["kv_lens"] else q
        if case["causal"]:
            pairs = sum(sum(max(0, min(m, i + 1 + m - n)) for i in range(n)) for n, m in zip(q, kv))
        else:
            pairs = sum(n * m for n, m in zip(q, kv))
        return {"bytes": sum(q) * case["Hq"] * (4 * d + 4) + sum(kv) * Hkv * 4 * d, "flops": 4 * d * case["Hq"] * pairs}
    page, nbytes, flops = case["page"], 0, 0
    if case["op"] in ("store", "step"):
        n = _ints(case["q_lens"]) if case["op"] == "store" else [1] * len(_ints(case["lens"]))
        tokens = sum(n)
        nbytes += tokens * Hkv * 2 * d * 3 + 2 * Hkv * sum(-(-k // page) for k in n)
        flops += tokens * Hkv * 2 * d * 3
    if case["op"] in ("decode", "step"):
        lens = _ints(case["lens"])
        nbytes += sum(lens) * Hkv * 2 * d + sum(-(-k // page) for k in lens) * (2 * Hkv + 4) + len(lens) * case["Hq"] * (4 * d + 4)
        flops += 4 * d * case["Hq"] * sum(lens)
    return {"bytes": nbytes, "flops": flops}
