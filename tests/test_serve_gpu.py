"""The serving operators on the GPU against their definitions in 64 bits (tests/serve_ref.py, which derives the
tolerances): packed prompts, the 8-bit paged cache, single-token attention, and the three as a server runs them."""
import math
import os
import sys

import pytest
import torch

from mxfp4_microscaled_quantization_b200 import mxattn as mx

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------ prompts

def check_prompt(q, k, v, qo, ko, causal, scale=0.0, cut=True, **kw):
    ws = mx.new_prompt_workspace(k.shape[0] if cut else 0, q.shape[2])
    o, lse = mx.mxattn_prompt(q, k, v, i32(qo), i32(ko), causal, scale, workspace=ws, **kw)
    assert mx.mxattn_workspace_status(ws) == 0
    want, wl, to, tl = ref.prompt(q, k, v, qo, ko, causal, scale or None)
    n = qo[-1]
    ref.close(lse[:, :n], wl[:, :n], tl[:, :n], "lse")
    ref.close(o[:n], want[:n], to[:n], "out")
    return o, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(4, 4, 64, BF), (8, 2, 128, BF), (6, 2, 128, FP), (5, 1, 64, FP), (2, 1, 128, BF)])
@pytest.mark.parametrize("lens", [[1], [2, 1], [77], [127, 128, 129], [0, 5, 0, 300, 0], [257, 64, 1000], [513], [1] * 40])
def test_prompt_packed(lens, Hq, Hkv, d, dtype, causal):
    g, o = gen(sum(lens) + Hq), offsets(lens)
    q, k, v = randn(g, o[-1], Hq, d, dtype=dtype), randn(g, o[-1], Hkv, d, dtype=dtype), randn(g, o[-1], Hkv, d, dtype=dtype)
    check_prompt(q, k, v, o, o, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(8, 2, 128, BF), (3, 3, 64, FP)])
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 128, 300], [5, 1000, 130]), ([3], [0]), ([200, 1], [1, 700]),
                                            ([1, 1, 1], [255, 256, 257]), ([130, 0, 64], [0, 9, 64]), ([384], [140])])
def test_prompt_other_keys_than_queries(q_lens, kv_lens, Hq, Hkv, d, dtype, causal):
    """Later chunks of a prompt (more keys), and rows that see no key (fewer): zeros and -inf."""
    g, qo, ko = gen(7), offsets(q_lens), offsets(kv_lens)
    q = randn(g, qo[-1], Hq, d, dtype=dtype)
    k, v = randn(g, ko[-1], Hkv, d, dtype=dtype), randn(g, ko[-1], Hkv, d, dtype=dtype)
    check_prompt(q, k, v, qo, ko, causal)


@pytest.mark.parametrize("n,Hq,Hkv,d,dtype", [(4100, 4, 1, 128, BF), (2500, 2, 2, 64, FP)])
def test_prompt_long(n, Hq, Hkv, d, dtype):
    g = gen(n)
    q, k, v = randn(g, n, Hq, d, dtype=dtype, scale=2.0), randn(g, n, Hkv, d, dtype=dtype), randn(g, n, Hkv, d, dtype=dtype)
    check_prompt(q, k, v, [0, n], [0, n], True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,d,dtype", [
    ([1], [5000], 2, 1, 128, BF),               # one query: every part of one item
    ([200], [4003], 3, 1, 64, FP),              # an odd number of tiles: the last item has one
    ([17, 64, 3], [2048, 4096, 1000], 8, 2, 128, BF),
    ([300, 2, 40, 0], [9000, 300, 2300, 500], 4, 2, 64, BF),
    ([3000], [2900], 1, 1, 128, FP),            # rows that see no key; parts that only later rows see
    ([129] * 3, [3333] * 3, 5, 1, 128, BF)])
def test_prompt_cut_along_the_keys(q_lens, kv_lens, Hq, Hkv, d, dtype, causal):
    """Few queries on long keys: items cut into parts and joined; the same within rounding as without (a workspace too
    small for parts)."""
    g, qo, ko = gen(40), offsets(q_lens), offsets(kv_lens)
    q = randn(g, qo[-1], Hq, d, dtype=dtype, scale=1.5)
    k, v = randn(g, ko[-1], Hkv, d, dtype=dtype), randn(g, ko[-1], Hkv, d, dtype=dtype)
    check_prompt(q, k, v, qo, ko, causal)
    check_prompt(q, k, v, qo, ko, causal, cut=False)


def test_prompt_cut_with_masked_junk_and_graph():
    """NaN in keys and values that only later rows see, in the last part; then captured, replayed with other lengths."""
    g = gen(41)
    q, k, v = randn(g, 64, 4, 128), randn(g, 4000, 2, 128), randn(g, 4000, 2, 128)
    k[3990], v[3990] = math.nan, math.inf
    o, lse = mx.mxattn_prompt(q, k, v, i32([0, 64]), i32([0, 4000]))
    clean_k, clean_v = k.clone(), v.clone()
    clean_k[3990], clean_v[3990] = 0, 0
    want, wl, to, tl = ref.prompt(q, clean_k, clean_v, [0, 64], [0, 4000], True)
    seen = 64 - 10  # row 54 is the first that sees key 3990
    ref.close(o[:seen], want[:seen], to[:seen])
    ref.close(lse[:, :seen], wl[:, :seen], tl[:, :seen])
    assert torch.isnan(lse[:, seen:]).all() and not torch.isfinite(o[seen:]).any()
    ws, out, ko = mx.new_prompt_workspace(4000, 128), torch.zeros_like(q), i32([0, 4000])
    qo, lse = i32([0, 64]), torch.zeros((4, 64), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxattn_prompt(q, clean_k, clean_v, qo, ko, out=out, lse=lse, workspace=ws)
    for n, m in ((64, 4000), (64, 300), (1, 4000), (40, 2500), (64, 4000)):
        qo.copy_(i32([0, n]))
        ko.copy_(i32([0, m]))
        graph.replay()
        torch.cuda.synchronize()
        want, wl, to, tl = ref.prompt(q[:n], clean_k, clean_v, [0, n], [0, m], True)
        ref.close(out[:n], want, to)
        ref.close(lse[:, :n], wl, tl)
    assert mx.mxattn_workspace_status(ws) == 0


def test_prompt_growing_scores():
    """The row maximum rises over the whole sequence (every tile rescales), then over none; large scores."""
    g, n = gen(3), 1500
    q = randn(g, n, 2, 64).abs()
    up = torch.linspace(0, 20, n, device="cuda")[:, None, None]
    for ramp in (up, up.flip(0)):
        k = (randn(g, n, 2, 64).float() * 0.1 + ramp).to(BF)
        check_prompt(q, k, randn(g, n, 2, 64), [0, n], [0, n], True)
    q, k = randn(g, 300, 2, 128, scale=20.0), randn(g, 300, 2, 128, scale=20.0)
    check_prompt(q, k, randn(g, 300, 2, 128), [0, 300], [0, 300], True)


@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_prompt_scale(scale):
    g = gen(4)
    check_prompt(randn(g, 200, 2, 64), randn(g, 200, 2, 64), randn(g, 200, 2, 64), [0, 200], [0, 200], True, scale)


def test_prompt_strided():
    """Q, K and V as parts of one projection's output, O head-major."""
    g, n, d = gen(5), 301, 128
    qkv = randn(g, n, 8 + 2 + 2, d)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    o = torch.zeros((8, n, d), dtype=BF, device="cuda").transpose(0, 1)
    check_prompt(q, k, v, [0, 100, n], [0, 100, n], True, out=o)
    one, want = randn(g, 1, 8, d), randn(g, 1, 2, d)
    check_prompt(one, want, want, [0, 1], [0, 1], True)
    heads_first = [randn(g, h, n, d).transpose(0, 1) for h in (8, 2, 2)]
    check_prompt(*heads_first, [0, 200, n], [0, 200, n], True)
    wide = [randn(g, n, h, 192)[:, :, 8:8 + d] for h in (8, 2, 2)]  # heads 192 apart
    check_prompt(*wide, [0, 200, n], [0, 200, n], False)


def test_prompt_rows_of_no_sequence_stay():
    g = gen(6)
    q, k, v = randn(g, 300, 4, 64), randn(g, 300, 2, 64), randn(g, 300, 2, 64)
    for x in (q, k, v):
        x[250:] = math.nan
    o, lse = torch.full((300, 4, 64), 7.0, dtype=BF, device="cuda"), torch.full((4, 300), 9.0, device="cuda")
    check_prompt(q, k, v, [0, 100, 250], [0, 100, 250], True, out=o, lse=lse)
    assert (o[250:] == 7).all() and (lse[:, 250:] == 9).all()


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_prompt_masked_places_hold_anything(junk, dtype):
    """NaN and infinities in other sequences and in later keys of the same one change no row that does not see them."""
    g, lens = gen(8), [130, 300, 70]
    o = offsets(lens)
    q, k, v = randn(g, 500, 4, 128, dtype=dtype), randn(g, 500, 2, 128, dtype=dtype), randn(g, 500, 2, 128, dtype=dtype)
    clean, _ = mx.mxattn_prompt(q, k, v, i32(o), causal=True)
    k2, v2 = k.clone(), v.clone()
    k2[o[1] + 210], v2[o[1] + 210] = junk, junk       # seen by the rows 210 .. 299 of sequence 1 only
    v2[o[3] - 1, 1, 5] = junk                          # by the last row of the batch, one channel
    ws = mx.new_prompt_workspace()
    got, lse = mx.mxattn_prompt(q, k2, v2, i32(o), causal=True, workspace=ws)
    assert mx.mxattn_workspace_status(ws) == 0
    want, wl, to, tl = ref.prompt(q, k, v, o, o, True)
    keep = torch.ones(500, dtype=torch.bool, device="cuda")
    keep[o[1] + 210:o[2]] = False
    keep[o[3] - 1] = False
    ref.close(got[keep], want[keep], to[keep], "rows that see none of it")
    ref.close(lse[:, keep], wl[:, keep], tl[:, keep], "their lse")
    assert torch.isfinite(got[keep]).all()
    last = got[o[3] - 1].float()                       # the one channel of the heads of key head 1, nothing else
    assert not torch.isfinite(last[2:, 5]).any()
    last[2:, 5] = 0
    assert torch.isfinite(last).all()


def test_prompt_lowest_values():
    """Keys that give the lowest scores of the type, and -inf, take no weight; a row with nothing else is that of its type."""
    g = gen(9)
    q, k, v = torch.ones((200, 2, 64), dtype=BF, device="cuda"), randn(g, 200, 2, 64), randn(g, 200, 2, 64)
    k[50:60] = torch.finfo(BF).min / 64
    k[3] = torch.finfo(BF).min / 64
    check_prompt(q, k, v, [0, 200], [0, 200], True)


def test_prompt_bad_offsets_are_reported():
    """Offsets that leave the tensors or decrease are brought into range: no access outside, the other rows right."""
    g = gen(10)
    q, k, v = randn(g, 100, 2, 64), randn(g, 100, 2, 64), randn(g, 100, 2, 64)
    for bad in ([0, 40, 101], [0, 40, 1 << 30], [0, 40, -5], [0, 40, 30]):
        ws = mx.new_prompt_workspace()
        o, _ = mx.mxattn_prompt(q, k, v, i32(bad), causal=True, workspace=ws)
        assert mx.mxattn_workspace_status(ws) == 1
        want, _, to, _ = ref.prompt(q, k, v, [0, 40], [0, 40], True)
        ref.close(o[:40], want[:40], to[:40])
    ws.zero_()
    mx.mxattn_prompt(q, k, v, i32([0, 40, 100]), causal=True, workspace=ws)
    assert mx.mxattn_workspace_status(ws) == 0


def test_prompt_many_sequences():
    g, lens = gen(11), [(7 * i) % 23 for i in range(600)]
    o = offsets(lens)
    q, k, v = randn(g, o[-1], 2, 64), randn(g, o[-1], 1, 64), randn(g, o[-1], 1, 64)
    check_prompt(q, k, v, o, o, True)


def test_prompt_nothing_to_do_and_no_lse():
    e = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    o, lse = mx.mxattn_prompt(e, e, e, i32([0, 0]))
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    g = gen(12)
    q = randn(g, 50, 2, 64)
    ws, out = mx.new_prompt_workspace(), torch.zeros_like(q)
    st = mx.lib().mxattn_prompt(q.data_ptr(), q.data_ptr(), q.data_ptr(), 0, i32([0, 50]).data_ptr(), i32([0, 50]).data_ptr(), 1,
                                50, 50, 2, 2, 64, None, 1, 0.0, out.data_ptr(), None, 0, ws.data_ptr(), 256,
                                torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want, _, to, _ = ref.prompt(q, q, q, [0, 50], [0, 50], True)
    ref.close(out, want, to)


def test_prompt_streams_graph_and_repeat():
    """Two calls at once on two streams; a captured call replayed with other offsets and inputs; the same bits each time."""
    g = gen(13)
    a = [randn(g, 700, 4, 128) for _ in range(1)] + [randn(g, 700, 2, 128) for _ in range(2)]
    o1, o2 = i32([0, 300, 700]), i32([0, 650, 700])
    base1, base2 = mx.mxattn_prompt(*a, o1)[0], mx.mxattn_prompt(*a, o2)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros((700, 4, 128), dtype=BF, device="cuda") for _ in range(2)]
    w = [mx.new_prompt_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        mx.mxattn_prompt(*a, o1, out=outs[0], workspace=w[0], stream=s1)
        mx.mxattn_prompt(*a, o2, out=outs[1], workspace=w[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], base1) and torch.equal(outs[1], base2)
    off, out, lse = o1.clone(), torch.zeros_like(outs[0]), torch.zeros((4, 700), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxattn_prompt(*a, off, out=out, lse=lse, workspace=w[0])
    for o, base in ((o1, base1), (o2, base2)):
        off.copy_(o)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base)


# ------------------------------------------------------------------ the cache

def make_cache(g, pool, Hkv, page, d):
    """Pages and exponents of arbitrary bytes."""
    r = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return [r(pool, Hkv, page, d), r(pool, Hkv, page, d), r(pool, Hkv), r(pool, Hkv)]


def make_table(g, lens, page, spare=2, extra=0):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device="cuda").tolist()
    table = [[-1] * (max(need + [1]) + extra) for _ in lens]
    for b, n in enumerate(need):
        for i in range(n):
            table[b][i] = order.pop()
    return sum(need) + spare, table


def check_store(cache, k, v, table, off, held, status_want=0):
    want_k, want_ke = ref.store(k, cache[0], cache[2], table, off, held)
    want_v, want_ve = ref.store(v, cache[1], cache[3], table, off, held)
    status = i32([0])
    mx.mxattn_cache_store(k, v, *cache, i32(table), i32(off), i32(held), status=status)
    assert int(status) == status_want
    for codes, exps, wc, we in ((cache[0], cache[2], want_k, want_ke), (cache[1], cache[3], want_v, want_ve)):
        assert torch.equal(exps, we)
        got = ref.values(codes)
        assert torch.equal(torch.isnan(got), torch.isnan(wc))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(wc))
        assert torch.equal(torch.signbit(got), torch.signbit(wc)) or bool((got[torch.signbit(got) != torch.signbit(wc)].isnan()).all())


@pytest.mark.parametrize("page,Hkv,d,dtype", [(16, 2, 64, BF), (32, 1, 128, FP), (64, 3, 128, BF), (128, 2, 128, BF), (128, 1, 64, FP)])
@pytest.mark.parametrize("n,held", [([1], [0]), ([1, 1, 1, 1], [0, 15, 16, 200]), ([300, 0, 1, 128], [0, 4, 127, 128]),
                                    ([77, 500], [51, 3]), ([1] * 300, list(range(300)))])
def test_store(n, held, page, Hkv, d, dtype):
    """Codes and exponents bit for bit; the magnitudes span binades so that pages grow under earlier tokens."""
    g, off = gen(sum(n) + page), offsets(n)
    pool, table = make_table(g, [a + b for a, b in zip(n, held)], page)
    cache = make_cache(g, pool, Hkv, page, d)
    cache[2].random_(90, 125, generator=g)
    cache[3].random_(90, 125, generator=g)
    size = torch.exp2(torch.randint(-20, 8, (off[-1], Hkv, 1), generator=g, device="cuda").float())
    k = (torch.randn((off[-1], Hkv, d), generator=g, device="cuda") * size).to(dtype)
    v = (torch.randn((off[-1], Hkv, d), generator=g, device="cuda") * size.flip(0)).to(dtype)
    check_store(cache, k, v, table, off, held)


def test_store_every_value_and_boundary():
    """All finite bf16 and fp16 patterns, and page maxima on and next to 448 2^e for every e."""
    for dtype in (BF, FP):
        bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
        x = bits[torch.isfinite(bits.float())]
        for order in (torch.arange(x.numel(), device="cuda"), torch.randperm(x.numel(), generator=gen(1), device="cuda")):
            y = x[order][:x.numel() // 64 * 64].view(-1, 1, 64).contiguous()
            n = y.shape[0]
            pool, table = make_table(gen(2), [n], 16)
            check_store(make_cache(gen(3), pool, 1, 16, 64), y, -y, table, [0, n], [0])
    top = torch.arange(0x7F80, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)  # every page maximum of bf16
    k = torch.zeros((top.numel(), 1, 64), dtype=BF, device="cuda")
    k[:, 0, 17] = top
    k[:, 0, 3] = -top / 3
    table = [[b] for b in range(top.numel())]
    check_store(make_cache(gen(4), top.numel(), 1, 16, 64), k, k, table, list(range(top.numel() + 1)), [0] * top.numel())


def test_store_grows_step_by_step():
    """One token at a time, each a binade up, then small ones again: the page follows, earlier codes rounded each time."""
    g = gen(5)
    pool, table = make_table(g, [40], 32)
    cache = make_cache(g, pool, 2, 32, 64)
    for t in range(40):
        x = randn(g, 1, 2, 64, scale=2.0 ** (t % 20))
        check_store(cache, x, -x, table, [0, 1], [t])


def test_store_nan_inf_and_zero():
    x = torch.zeros((20, 1, 64), dtype=BF, device="cuda")
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7], x[6, 0, 8] = math.nan, math.inf, -math.inf, -0.0
    pool, table = make_table(gen(6), [20], 16)
    cache = make_cache(gen(6), pool, 1, 16, 64)
    mx.mxattn_cache_store(x, torch.zeros_like(x), *cache, i32(table), i32([0, 20]), i32([0]))
    k = ref.values(cache[0])[table[0][0]][0]
    assert torch.isnan(k[3, 5]) and k[4, 6] == 448 and k[5, 7] == -448
    assert (ref.values(cache[1])[table[0][:2]][:, 0].reshape(32, 64)[:20] == 0).all()
    assert cache[3][table[0][0], 0] == 0 and cache[3][table[0][1], 0] == 0


def test_store_strided():
    g = gen(7)
    qkv = randn(g, 100, 8, 128)
    pool, table = make_table(g, [100], 64)
    check_store(make_cache(g, pool, 2, 64, 128), qkv[:, 4:6], qkv[:, 6:], table, [0, 100], [0])


def test_store_refuses_bad_pages_and_lengths():
    """A page outside the pool, a length past the table or negative, offsets out of range: reported, nothing else touched."""
    g = gen(8)
    x = randn(g, 40, 2, 64)
    pool, table = make_table(g, [16, 16, 16], 16, extra=0)
    for held, off, tab in (([0, 0, 0], [0, 8, 16, 24], [table[0], [pool], table[2]]),
                           ([0, 0, 0], [0, 8, 16, 24], [table[0], [-1], table[2]]),
                           ([0, 9, 0], [0, 8, 16, 24], table), ([0, -1, 0], [0, 8, 16, 24], table),
                           ([0, 1 << 30, 0], [0, 8, 16, 24], table), ([0, 0, 0], [0, 8, 8, 41], table)):
        cache = make_cache(gen(9), pool, 2, 16, 64)
        before = [c.clone() for c in cache]
        status = i32([0])
        mx.mxattn_cache_store(x, x, *cache, i32(tab), i32(off), i32(held), status=status)
        assert int(status) == 1
        p0 = table[0][0]
        assert not torch.equal(cache[0][p0, :, :8], before[0][p0, :, :8])  # sequence 0 is stored
        bad = table[1][0]
        for c, w in zip(cache, before):
            assert torch.equal(c[bad], w[bad])


def test_store_reports_a_bad_length_anywhere_in_a_large_batch():
    g, B = gen(28), 700
    x = randn(g, B, 1, 64)
    table = [[b] for b in range(B)]
    for bad in (0, 255, 256, 699):
        held = [3] * B
        held[bad] = 16
        cache, status = make_cache(gen(9), B, 1, 16, 64), i32([0])
        before = cache[0].clone()
        mx.mxattn_cache_store(x, x, *cache, i32(table), i32(range(B + 1)), i32(held), status=status)
        assert int(status) == 1
        assert torch.equal(cache[0][bad], before[bad]) and not torch.equal(cache[0][(bad + 1) % B], before[(bad + 1) % B])


def check_attend(q, cache, table, lens, scale=0.0, status=0, **kw):
    ws = mx.new_cache_attend_workspace(q.shape[1], cache[0].shape[1], q.shape[2])
    o, lse = mx.mxattn_cache_attend(q, *cache, i32(table), i32(lens), scale, workspace=ws, **kw)
    assert mx.mxattn_workspace_status(ws) == status
    want, wl, to, tl = ref.attend(q, *cache, table, lens, scale or None)
    ref.close(lse, wl, tl, "lse")
    ref.close(o, want, to, "out")
    return o, lse


def fill(g, lens, Hkv, page, d, dtype, v_spread=0.5, extra=0):
    pool, table = make_table(g, lens, page, extra=extra)
    cache = make_cache(g, pool, Hkv, page, d)
    T = sum(lens)
    k = randn(g, T, Hkv, d, dtype=dtype)
    v = (torch.randn((T, Hkv, d), generator=g, device="cuda") * torch.exp(v_spread * torch.randn((T, 1, 1), generator=g, device="cuda"))).to(dtype)
    mx.mxattn_cache_store(k, v, *cache, i32(table), i32(offsets(lens)), i32([0] * len(lens)))
    return cache, table


@pytest.mark.parametrize("Hq,Hkv,d,page,dtype", [(8, 2, 128, 64, BF), (3, 3, 64, 16, FP), (16, 1, 128, 128, BF), (5, 1, 128, 32, FP),
                                                 (40, 2, 64, 64, BF), (33, 1, 128, 16, BF), (130, 2, 128, 64, FP)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 0], [15, 16, 17, 127, 128, 129], [300], [1000, 3, 0, 517], [5] * 70])
def test_attend(lens, Hq, Hkv, d, page, dtype):
    g = gen(sum(lens) + Hq + page)
    cache, table = fill(g, lens, Hkv, page, d, dtype, extra=1)
    check_attend(randn(g, len(lens), Hq, d, dtype=dtype, scale=1.5), cache, table, lens)


@pytest.mark.parametrize("lens", [[40000], [33000, 1, 20001, 129, 5000], [2000] * 33])
def test_attend_long(lens):
    g = gen(len(lens))
    cache, table = fill(g, lens, 2, 64, 128, BF)
    check_attend(randn(g, len(lens), 8, 128, scale=3.0), cache, table, lens)


def test_attend_scores_rise_and_fall():
    """The maximum moves in every tile, or in the first only; values of very different page exponents."""
    g, n = gen(20), 3000
    for ramp in (torch.linspace(0, 12, n, device="cuda"), torch.linspace(12, 0, n, device="cuda")):
        pool, table = make_table(g, [n], 16)
        cache = make_cache(g, pool, 1, 16, 64)
        k = (randn(g, n, 1, 64).float() * 0.1 + ramp[:, None, None]).to(BF)
        v = (randn(g, n, 1, 64).float() * torch.exp2(ramp[:, None, None] * 2 - 12)).to(BF)
        mx.mxattn_cache_store(k, v, *cache, i32(table), i32([0, n]), i32([0]))
        check_attend(randn(g, 1, 4, 64).abs(), cache, table, [n])


def test_attend_empty_values_and_extreme_exponents():
    """Pages of zeros (exponent -127) beside others, and exponents at both ends of what is reachable."""
    g = gen(21)
    pool, table = make_table(g, [96], 32)
    cache = make_cache(g, pool, 1, 32, 128)
    k, v = randn(g, 96, 1, 128), randn(g, 96, 1, 128)
    v[32:64] = 0
    k[64:] = 0
    mx.mxattn_cache_store(k, v, *cache, i32(table), i32([0, 96]), i32([0]))
    check_attend(randn(g, 1, 4, 128), cache, table, [96])
    v[:] = 0
    mx.mxattn_cache_store(k, v, *cache, i32(table), i32([0, 96]), i32([0]))
    o, _ = check_attend(randn(g, 1, 4, 128), cache, table, [96])
    assert (o == 0).all()
    for size in (2.0 ** -100, 2.0 ** 100):
        v = (torch.randn((96, 1, 128), generator=g, device="cuda") * size).to(BF)
        mx.mxattn_cache_store(k, v, *cache, i32(table), i32([0, 96]), i32([0]))
        check_attend(randn(g, 1, 4, 128), cache, table, [96])


def test_attend_query_sizes():
    """Queries of zeros, tiny and large ones, and a few strong channels."""
    g = gen(22)
    cache, table = fill(g, [200] * 4, 1, 64, 128, BF)
    q = randn(g, 4, 8, 128)
    q[0] = 0
    q[1] *= 2.0 ** -40
    q[2] *= 16
    q[3, :, 7] *= 64
    check_attend(q, cache, table, [200] * 4)
    cache, table = fill(g, [200], 1, 64, 64, FP)
    check_attend(randn(g, 1, 4, 64, dtype=FP, scale=2.0 ** -12), cache, table, [200])


def test_attend_nan_queries_and_keys():
    """What a sequence sees and is NaN or infinite makes its own rows NaN, no others."""
    g = gen(27)
    cache, table = fill(g, [200] * 4, 1, 64, 128, BF)
    q = randn(g, 4, 8, 128)
    want, _, to, _ = ref.attend(q, *cache, table, [200] * 4)
    q[1, 2, 5], q[2, 3, 6] = math.nan, math.inf
    cache[1][table[3][3], 0, 199 % 64, 9] = 0x7F
    o, lse = mx.mxattn_cache_attend(q, *cache, i32(table), i32([200] * 4))
    assert torch.isnan(o[1, 2]).all() and torch.isnan(o[2, 3]).all() and torch.isnan(lse[1, 2]) and torch.isnan(o[3, :, 9]).all()
    for x in (o, want):
        x[1, 2], x[2, 3], x[3, :, 9] = 0, 0, 0
    ref.close(o, want, to)


def test_attend_many_sequences():
    """More sequences than threads of a block, most of them short or empty, one long among them."""
    g = gen(29)
    lens = [(5 * i) % 40 for i in range(900)]
    lens[617] = 3000
    cache, table = fill(g, lens, 1, 16, 64, BF)
    check_attend(randn(g, 900, 4, 64), cache, table, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads", [1, 3, 4, 5, 8, 9, 15, 16, 17])
def test_attend_every_number_of_heads(heads, dtype, d):
    """The parts of queries and weights share the columns of a product with the heads, up to 16 of them a block."""
    g, lens = gen(heads + d), [129, 1, 0, 700, 64, 2100]
    cache, table = fill(g, lens, 2, 32, d, dtype)
    check_attend(randn(g, len(lens), 2 * heads, d, dtype=dtype, scale=2.0), cache, table, lens)


@pytest.mark.parametrize("Hkv,d,page,dtype", [(24, 64, 16, FP), (8, 128, 64, BF)])
def test_attend_blocks_of_many_one_tile_pieces(Hkv, d, page, dtype):
    """Queries, products and weights change hands at every tile, over and over: no wait may miss its phase."""
    g, lens = gen(31), [1 + 3 * (i % 5) for i in range(128)]
    cache, table = fill(g, lens, Hkv, page, d, dtype)
    q = randn(g, 128, Hkv, d, dtype=dtype)
    o, lse = check_attend(q, cache, table, lens)
    ws = mx.new_cache_attend_workspace(Hkv, Hkv, d)
    for _ in range(200):
        o2, lse2 = mx.mxattn_cache_attend(q, *cache, i32(table), i32(lens), workspace=ws)
    assert mx.mxattn_workspace_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attend_nothing_cached():
    q = randn(gen(1), 3, 4, 64)
    empty = [torch.zeros((0, 2, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    empty += [torch.zeros((0, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    o, lse = mx.mxattn_cache_attend(q, *empty, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), i32([0, 0, 0]))
    assert (o == 0).all() and torch.isneginf(lse).all()
    ws = mx.new_cache_attend_workspace(4, 2, 64)
    o, lse = mx.mxattn_cache_attend(q, *empty, i32([[0], [1], [2]]), i32([16, 3, 0]), workspace=ws)
    assert (o == 0).all() and torch.isneginf(lse).all() and mx.mxattn_workspace_status(ws) == 1


def test_attend_shared_pages_and_strides():
    g = gen(23)
    cache, table = fill(g, [640], 2, 64, 128, BF)
    rows = [table[0], table[0], table[0][:3] + [-1] * (len(table[0]) - 3)]
    x = randn(g, 3, 20, 128)
    o = torch.zeros((8, 3, 128), dtype=BF, device="cuda").transpose(0, 1)
    check_attend(x[:, 5:13], cache, rows, [640, 129, 190], out=o)


def test_attend_bad_pages_and_lengths():
    """Tokens of a page outside the pool are left out, lengths brought into range, both reported."""
    g = gen(24)
    cache, table = fill(g, [128, 128], 2, 64, 64, BF)
    q = randn(g, 2, 4, 64)
    for bad in (-1, cache[0].shape[0], 1 << 30):
        rows = [list(table[0]), [table[1][0], bad]]
        ws = mx.new_cache_attend_workspace(4, 2, 64)
        o, lse = mx.mxattn_cache_attend(q, *cache, i32(rows), i32([128, 128]), workspace=ws)
        assert mx.mxattn_workspace_status(ws) == 1
        want, wl, to, tl = ref.attend(q, *cache, table, [128, 64])
        ref.close(o, want, to)
        ref.close(lse, wl, tl)
    rows = [[-1, -1], table[1]]
    o, lse = mx.mxattn_cache_attend(q, *cache, i32(rows), i32([128, 128]))
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    for given, taken in (([-3, 128], [0, 128]), ([129, 1 << 30], [128, 128])):
        ws = mx.new_cache_attend_workspace(4, 2, 64)
        o, lse = mx.mxattn_cache_attend(q, *cache, i32(table), i32(given), workspace=ws)
        assert mx.mxattn_workspace_status(ws) == 1
        want, wl, to, tl = ref.attend(q, *cache, table, taken)
        ref.close(o, want, to)
        ref.close(lse, wl, tl)


def test_attend_streams_graph_and_repeat():
    g, lens = gen(25), [3000, 1, 700, 0, 64]
    cache, table = fill(g, lens, 2, 64, 128, BF)
    q, t = randn(g, 5, 8, 128), i32(table)
    other = [1500, 1, 699, 0, 5]
    base, base2 = (mx.mxattn_cache_attend(q, *cache, t, i32(x))[0] for x in (lens, other))
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    w = [mx.new_cache_attend_workspace(8, 2, 128) for _ in range(2)]
    outs, ln = [torch.zeros_like(base), torch.zeros_like(base)], [i32(lens), i32(other)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            mx.mxattn_cache_attend(q, *cache, t, ln[i], out=outs[i], workspace=w[i], stream=s[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], base) and torch.equal(outs[1], base2)
    cur, out, lse = ln[0].clone(), torch.zeros_like(base), torch.zeros((5, 8), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxattn_cache_attend(q, *cache, t, cur, out=out, lse=lse, workspace=w[0])
    for x, want in ((ln[1], base2), (ln[0], base), (ln[1], base2)):
        cur.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_beyond_32_bits():
    """A pool whose codes pass 2^32 bytes: the last pages are stored and read where they are."""
    page, Hkv, d = 128, 8, 128
    pool = (1 << 32) // (page * Hkv * d) + 40
    if torch.cuda.mem_get_info()[0] < 3 * pool * page * Hkv * d:
        pytest.skip("not enough free memory")
    g = gen(26)
    cache = [torch.empty((pool, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros((pool, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pages = [pool - 1, 0, pool - 3, pool // 2 + 17]
    k, v, q = randn(g, 400, Hkv, d), randn(g, 400, Hkv, d), randn(g, 1, Hkv, d)
    mx.mxattn_cache_store(k, v, *cache, i32([pages]), i32([0, 400]), i32([0]))
    at = torch.tensor(pages, device="cuda")
    small = [c[at].contiguous() for c in cache]
    assert mx.mxattn_cache_attend(q, *cache, i32([pages]), i32([400]))[0].equal(
        mx.mxattn_cache_attend(q, *small, i32([[0, 1, 2, 3]]), i32([400]))[0])
    check_attend(q, small, [[0, 1, 2, 3]], [400])


def test_tensors_made_by_a_call_on_another_stream():
    """Outputs and workspace that a call makes belong to the stream it is given: work queued on the current stream neither
    delays nor overwrites them."""
    g = gen(31)
    cache, table = fill(g, [700, 30], 2, 64, 128, BF)
    q, k, v = randn(g, 200, 8, 128), randn(g, 3000, 2, 128), randn(g, 3000, 2, 128)
    t, n, qo, ko = i32(table), i32([700, 30]), i32([0, 150, 200]), i32([0, 2500, 3000])
    want = [*mx.mxattn_prompt(q, k, v, qo, ko), *mx.mxattn_cache_attend(q[:2], *cache, t, n)]
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        torch.cuda._sleep(200_000_000)  # about 0.1 s on the current stream
        got = [*mx.mxattn_prompt(q, k, v, qo, ko, stream=stream)]
        got += mx.mxattn_cache_attend(q[:2], *cache, t, n, stream=stream)
        junk = [torch.full_like(x, 5) for x in got for _ in range(3)]  # takes freed memory, on the current stream
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        del junk


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("d,page,dtype", [(128, 64, BF), (64, 16, FP)])
def test_prompt_then_decode(d, page, dtype):
    """A server's run: prompts attended and stored, then steps that store one token each and attend, captured in one graph
    and replayed; checked against attention over the cache's values, and loosely against the unquantized keys."""
    g, lens, steps, Hq, Hkv = gen(30), [130, 1, 64, 333], 5, 8, 2
    o = offsets(lens)
    full = [n + steps for n in lens]
    pool, table = make_table(g, full, page)
    cache, t = make_cache(g, pool, Hkv, page, d), i32(table)
    q, k, v = (randn(g, o[-1], h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    check_prompt(q, k, v, o, o, True)
    status = i32([0])
    mx.mxattn_cache_store(k, v, *cache, t, i32(o), i32([0] * 4), status=status)
    held, total, ones = i32(lens), i32([n + 1 for n in lens]), i32(range(5))
    q1, k1, v1 = (torch.zeros((4, h, d), dtype=dtype, device="cuda") for h in (Hq, Hkv, Hkv))
    out, lse, ws = torch.zeros_like(q1), torch.zeros((4, Hq), device="cuda"), mx.new_cache_attend_workspace(Hq, Hkv, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxattn_cache_store(k1, v1, *cache, t, ones, held, status=status)
        mx.mxattn_cache_attend(q1, *cache, t, total, out=out, lse=lse, workspace=ws)
        held.add_(1)
        total.add_(1)
    keys = [k[o[b]:o[b + 1]] for b in range(4)]
    vals = [v[o[b]:o[b + 1]] for b in range(4)]
    for i in range(steps):
        for x in (q1, k1, v1):
            x.copy_(randn(g, *x.shape, dtype=dtype))
        graph.replay()
        torch.cuda.synchronize()
        now = [n + i + 1 for n in lens]
        want, wl, to, tl = ref.attend(q1, *cache, table, now)
        ref.close(out, want, to)
        ref.close(lse, wl, tl)
        keys = [torch.cat([a, k1[b:b + 1]]) for b, a in enumerate(keys)]
        vals = [torch.cat([a, v1[b:b + 1]]) for b, a in enumerate(vals)]
        for b in range(4):
            kk, vv = keys[b].double().repeat_interleave(Hq // Hkv, 1), vals[b].double().repeat_interleave(Hq // Hkv, 1)
            s = torch.einsum("hd,nhd->hn", q1[b].double(), kk) / math.sqrt(d)
            near = torch.einsum("hn,nhd->hd", torch.softmax(s, 1), vv)
            # E4M3 keys and values: 2^-4 each at most; typically a few hundredths of the output's size
            assert float((out[b].double() - near).norm() / near.norm()) < 0.125
    assert int(status) == 0 and mx.mxattn_workspace_status(ws) == 0
