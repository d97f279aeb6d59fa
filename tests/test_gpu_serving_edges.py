"""Single-token serving on the GPU at its edges.  References and tolerances as
in serving_reference.py."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_reduce_b200 as fp4
import serving_reference as ref
from test_gpu_serving import (BF, F32, MX, NV, check_attention, gen, host, make_cache, randn, sequences, tables,
                              test_write_and_read_are_the_oracle_bit_for_bit as oracle_bits)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- attention: the range --

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("key,query,scale", [
    (105, 0, -111), (118, 0, -123), (118, -60, -64), (110, -110, -5), (118, -112, -8),
    (-120, 0, 114), (-110, 110, -5), (-120, 120, -5), (-60, -60, 114), (60, 60, -126)])
def test_attention_mxfp4_keys_of_every_size(key, query, scale, dtype):
    """Block scales of the keys round 2^key, queries round 2^query: the factors leave fp32's range, the scores do not."""
    g = gen(key + query)
    c = make_cache(g, 4, 2, 128, 32, MX)
    c.k_scales.copy_(torch.randint(123 + key, 128 + key, c.k_scales.shape, generator=g, dtype=torch.uint8))
    table = tables(g, 1, 4, 4)
    q = (randn(g, 1, 2, 8, 128, dtype=F32) * 2.0 ** query).to(dtype)
    check_attention(c, q, table, [111], 2.0 ** scale, 0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("key,query,scale,lo,hi", [(-126, 126, -13, 96, 127), (-126, 125, -12, 96, 127), (110, -120, 19, 1, 8), (115, -123, 14, 1, 8),
                                                   (-60, -60, 113, 40, 64)])
def test_attention_nvfp4_global_scales_of_every_size(key, query, scale, lo, hi, dtype):
    """Global scales of the keys round 2^key: times softmax_scale they leave fp32's normal numbers, the scores do not."""
    g = gen(key + query + 1000)
    c = make_cache(g, 4, 2, 64, 32, NV)
    c.k_global_scale.copy_(torch.tensor([1.0, 1.25]) * 2.0 ** key)
    c.k_scales.copy_(torch.randint(lo, hi, c.k_scales.shape, generator=g, dtype=torch.uint8))
    table = tables(g, 1, 4, 4)
    q = (randn(g, 1, 2, 8, 64, dtype=F32).clamp(-3, 3) * 2.0 ** query).to(dtype)
    check_attention(c, q, table, [111], 2.0 ** scale, 0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [111, 3000])
@pytest.mark.parametrize("fmt,size", [(NV, -126), (NV, -110), (NV, 108), (MX, -116), (MX, 118)])
def test_attention_values_of_every_size(fmt, size, n, dtype):
    """Values round 2^size, compared relative to it (no absolute allowance but the spacing of numbers below the smallest normal one)."""
    g = gen(size + n)
    c = make_cache(g, 50, 2, 64, 64, fmt)
    if fmt == NV:
        c.v_global_scale.copy_(torch.tensor([1.0, 1.25]) * 2.0 ** size)
    else:
        c.v_scales.copy_(torch.randint(124 + size, 128 + size, c.v_scales.shape, generator=g, dtype=torch.uint8))
    table = tables(g, 1, 47, 50)
    q = randn(g, 1, 1, 8, 64, dtype=dtype)
    out, lse = fp4.kv_attention(q, c, table, torch.tensor([n], dtype=torch.int32).cuda(), scale=0.003)
    c.check()
    want, _, tol, _ = ref.attention(q, *sequences(c, table, [n]), [n], 0.003, 0, fmt == MX)
    tol = tol + ref.HALF[dtype] * np.abs(want) + {BF: 2.0 ** -134, F32: 2.0 ** -150}[dtype]
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), np.max(err / tol)


# ------------------------------------------------ attention: NaN out of sight --

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("n,new,window,group,dim,bad", [
    (100, 4, 0, 2, 64, 99), (100, 4, 0, 2, 128, 97), (100, 4, 40, 2, 64, 57), (33, 3, 0, 1, 256, 32), (1300, 2, 900, 3, 64, 399),
    (2600, 4, 0, 4, 128, 2598)])
def test_a_token_s_nan_reaches_the_tokens_that_see_it_and_no_others(n, new, window, group, dim, bad, fmt, dtype):
    """NaN scale bytes of the key, of the value or of both at a position that some of the new tokens see and others do not."""
    g = gen(n + bad)
    c = make_cache(g, 45, 2, dim, 64, fmt)
    table = torch.randperm(45, generator=g)[:-(-n // 64)][None].int().cuda()
    if n > 1024:  # a table wide enough for the tokens to be shared out
        table = torch.cat((table, torch.full((1, 4), -1, dtype=torch.int32, device="cuda")), 1)
    q = randn(g, 1, new, 2 * group, dim, dtype=dtype)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    want = fp4.kv_attention(q, c, table, lens, scale=0.01, window=window)
    pos = n - new + np.arange(new)
    sees = (bad <= pos) & ((bad > pos - window) if window else True)
    assert sees.any() and not sees.all()
    page, off = int(table[0, bad // 64]), bad % 64
    for names in (("k",), ("v",), ("k", "v")):
        kept = {name: getattr(c, name + "_scales")[page, 1, off].clone() for name in names}
        for name in names:
            getattr(c, name + "_scales")[page, 1, off, -1] = 0x7F if fmt == NV else 0xFF
        out, lse = fp4.kv_attention(q, c, table, lens, scale=0.01, window=window)
        c.check()
        for name in names:
            getattr(c, name + "_scales")[page, 1, off] = kept[name]
        for i in range(new):
            if sees[i]:
                assert torch.equal(out[0, i, :group], want[0][0, i, :group])  # the other KV head's
                if fmt == NV or "k" in names:
                    assert out[0, i, group:].isnan().any(-1).all() and lse[0, i, group:].isnan().all()
            else:
                assert torch.equal(out[0, i], want[0][0, i]) and torch.equal(lse[0, i], want[1][0, i])


# --------------------------------------------------------- linear: the handle --

@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_a_weight_laid_out_on_a_given_stream_belongs_to_it(handle):
    """The current stream held up: layout and status word are ordered with the given stream's calls."""
    g = gen(77)
    q = fp4.nvfp4_quantize(randn(g, 300, 2048, scale=0.02))
    x = randn(g, 20, 2048)
    want = fp4.linear(x, fp4.linear_weight(q))
    bad = x.clone()
    bad[3, 5] = float("inf")
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    w = fp4.linear_weight(q, stream=given)
    got = fp4.linear(x, w, stream=given)
    fp4.linear(bad, w, stream=given)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert int(w.status.item()) == fp4.ERR_NONFINITE  # not wiped out by a zero-fill that came late


# ------------------------------------------- the cache: rounds of its token loop --

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt,T,H,D,page,skip", [
    # two tokens a CTA: 592 CTAs write 2368 a round, 740 read 2960, the last round ending in the first token of a thread and in the second
    (NV, 8195, 8, 128, 64, 3), (NV, 8900, 8, 128, 48, 0),
    # 512 units a row: two CTAs side by side; 256 (MXFP4): one token a CTA
    (NV, 5003, 16, 256, 64, 3), (MX, 5003, 16, 256, 64, 3)])
def test_write_and_read_of_many_rounds_a_thread(fmt, T, H, D, page, skip, dtype):
    oracle_bits(T, H, D, page, skip, dtype, fmt, 0)


# ------------------------------------------- attention: long shares of a CTA --

NEEDLES = 30


def needle_cache(g, heads, dim, page, fmt, background=40):
    """`background` pages of noise and NEEDLES pages more with one token each (in their first, last or a middle slot) that
    scores far above it for a query along base [heads, dim]."""
    c = fp4.kv_cache(background + NEEDLES, heads, dim, page, fmt)
    slots = torch.arange(c.num_pages * page)
    k, v = randn(g, len(slots), heads, dim), randn(g, len(slots), heads, dim)
    base = (torch.randint(0, 2, (heads, dim), generator=g) * 2 - 1).to(BF).cuda()
    for i in range(NEEDLES):
        k[(background + i) * page + (0, page - 1, (7 * i) % page)[i % 3]] = base * 2.25
    fp4.kv_write(c, k, v, slots.cuda())
    c.check()
    return c, base


def needle_table(g, lens, width, page, background=40):
    """Noise pages in any order, and every needle page once a sequence: round multiples of 2048 tokens, at the ends, and anywhere."""
    table = torch.randint(0, background, (len(lens), width), generator=g, dtype=torch.int32)
    for b, n in enumerate(lens):
        whole = n // page
        if whole < NEEDLES:
            continue
        at = {0, whole - 1} | {m * 2048 // page + d for m in range(1, n // 2048, max(1, n // 2048 // 6)) for d in (-1, 0)}
        at = sorted(at)[:NEEDLES - 8]
        rest = [p for p in torch.randperm(whole, generator=g).tolist() if p not in at][:NEEDLES - len(at)]
        for i, p in enumerate(at + rest):
            table[b, p] = background + i
        table[b, -(-n // page):] = -1
    return table.cuda()


LONG = [  # lens, new, heads, group, dim, page, window: more than 16 rounds of 128 tokens for each of 740, 592 or 444 CTAs
    ([60001, 20480, 49999, 33333, 55000], 1, 8, 1, 64, 64, 0),
    ([60000, 41000, 33, 63333], 1, 8, 1, 128, 48, 0),
    ([60000, 41000, 33333, 47000], 4, 8, 3, 64, 64, 40001),
]


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("lens,new,heads,group,dim,page,window", LONG)
def test_attention_of_long_shares(lens, new, heads, group, dim, page, window, fmt):
    g = gen(sum(lens))
    c, base = needle_cache(g, heads, dim, page, fmt)
    table = needle_table(g, lens, -(-max(lens) // page) + 1, page)
    q = base[:, None].expand(heads, group, dim) * (1 + 0.05 * torch.rand(len(lens), new, heads, group, 1, generator=g).cuda())
    q = q.flatten(2, 3).to(BF)
    # a needle's score is 7.2 (ln 1340) over a background of e^s, s of deviation 0.4: 1 to 4 % of a sum
    check_attention(c, q, table, lens, 7.2 / 2.25 / dim, window)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("lens,new,heads,group,dim,page,window", LONG + [([5200, 4097, 2049, 1300] + [i % 40 for i in range(750)], 1, 8, 1, 64, 64, 0)])
def test_attention_counts_every_token_once(lens, new, heads, group, dim, page, window, fmt, dtype):
    """Queries of zero: every weight is exactly one, and lse the logarithm of the number of visible tokens.  A single token
    of 63333 lost or taken twice moves it by 1.6e-5; log2f and the product with ln 2 by 2^-22 of it, 3e-6."""
    g = gen(sum(lens) + 1)
    c = make_cache(g, 50, heads, dim, page, fmt)
    table = torch.randint(0, 50, (len(lens), -(-max(lens) // page) + 1), generator=g, dtype=torch.int32).cuda()
    q = torch.zeros(len(lens), new, heads * group, dim, dtype=dtype, device="cuda")
    _, lse = fp4.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32).cuda(), window=window)
    c.check()
    pos = np.array(lens)[:, None] - new + np.arange(new)
    count = np.maximum(0, np.minimum(pos + 1, window) if window else pos + 1)
    with np.errstate(divide="ignore"):
        want = np.log(count)[:, :, None].repeat(heads * group, 2)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    seen = ~np.isneginf(want)
    assert (np.abs(got[seen] - want[seen]) <= 2.0 ** -22 * np.abs(want[seen]) + 2.0 ** -20).all()


def test_attention_of_a_long_sequence_that_one_cta_takes():
    """8 units a CTA slot and more under a table of 6400 tokens: a unit is a CTA's, however long it is."""
    g = gen(79)
    lens = [5200, 4097, 2049] + [int(i) for i in torch.randint(0, 40, (760,), generator=g)]
    c, base = needle_cache(g, 8, 64, 64, NV)
    table = needle_table(g, lens, 100, 64)
    q = base[None, None].expand(len(lens), 1, 8, 64).contiguous()
    check_attention(c, q, table, lens, 7.2 / 2.25 / 64, 0)


def test_the_helpers_refuse_words_and_workspaces_that_are_not_what_they_seem():
    """A status that is no int32 word, and a workspace of fewer bytes than elements times their size."""
    g = gen(80)
    w = fp4.linear_weight(fp4.nvfp4_quantize(randn(g, 70, 64)))
    x, slots = randn(g, 3, 64), torch.tensor([1, 2, 3]).cuda()
    c = make_cache(g, 4, 2, 64, 16, NV)
    k, table, lens, q = randn(g, 3, 2, 64), tables(g, 1, 4, 4), torch.tensor([60], dtype=torch.int32).cuda(), randn(g, 1, 1, 4, 64)
    need = fp4.kv_attention_workspace(q, c, table).numel(), fp4.linear_workspace(3, w).numel()
    one = torch.zeros(16, dtype=torch.uint8, device="cuda")
    for status in (torch.zeros(1, dtype=torch.uint8, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
        for bad in (lambda: fp4.kv_write(c, k, k, slots, status=status), lambda: fp4.kv_read(c, slots, status=status),
                    lambda: fp4.kv_attention(q, c, table, lens, status=status), lambda: fp4.linear(x, w, status=status),
                    lambda: fp4.KVCache(NV, c.k_packed, c.k_scales, c.v_packed, c.v_scales, c.k_global_scale, c.v_global_scale, status),
                    lambda: fp4.LinearWeight(NV, w.packed, w.scales_mma, w.global_scale, 70, 64, status)):
            with pytest.raises((TypeError, ValueError), match="status"):
                bad()
    for bad in (lambda: fp4.kv_attention(q, c, table, lens, workspace=one[:1].expand(need[0])),
                lambda: fp4.linear(x, w, workspace=one[:1].expand(need[1]))):
        with pytest.raises(ValueError, match="workspace"):
            bad()
    torch.cuda.synchronize()
    c.check()
    w.check()
