"""Single-token serving on the GPU: the paged FP4 cache (write and read
back, bit for bit against the oracle), attention over it and the product of a
few rows with an FP4 weight (against 64-bit references, tolerances in
serving_reference.py)."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_reduce_b200 as fp4
import serving_reference as ref

pytestmark = pytest.mark.gpu

NV, MX = fp4.NVFP4, fp4.MXFP4
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def make_cache(g, pages, heads, dim, page, fmt):
    """A cache full of noise (codes and scale bytes of every kind but NaN)."""
    kg = (torch.rand(heads, generator=g) + 0.5) / 64
    vg = (torch.rand(heads, generator=g) + 0.5) / 64
    c = fp4.kv_cache(pages, heads, dim, page, fmt, kg.cuda(), vg.cuda())
    for name in ("k", "v"):
        getattr(c, name + "_packed").copy_(torch.randint(0, 256, c.k_packed.shape, generator=g, dtype=torch.uint8))
        lo, hi = (0, 127) if fmt == NV else (117, 132)
        getattr(c, name + "_scales").copy_(torch.randint(lo, hi, c.k_scales.shape, generator=g, dtype=torch.uint8))
    return c


def host(c):
    """Decoded keys and values of the whole cache, [pages, heads, page, D] in 64 bits."""
    out = []
    for n in ("k", "v"):
        s = getattr(c, n + "_global_scale")
        gs = s.cpu().double().numpy()[None, :, None, None] if c.fmt == NV else 1.0
        out.append(ref.decode(getattr(c, n + "_packed").cpu().numpy(), getattr(c, n + "_scales").cpu().numpy(), c.fmt == NV, gs))
    return out


def tables(g, batch, width, pages):
    t = torch.stack([torch.randperm(pages, generator=g)[:width] for _ in range(batch)]) if width else torch.zeros(batch, 0)
    return t.int().cuda()


def sequences(c, table, lens):
    k, v = host(c)
    pick = lambda x, b: x[table[b].cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, c.heads, c.head_dim)[:lens[b]]  # noqa: E731
    return [pick(k, b) for b in range(len(lens))], [pick(v, b) for b in range(len(lens))]


# ---------------------------------------------------------------- the cache --

CACHE = [(1, 1, 32, 16, 0), (5, 3, 64, 48, 0), (64, 8, 128, 64, 0), (131, 2, 96, 16, 3), (37, 5, 256, 32, 2), (3, 40, 128, 16, 0),
         (1000, 1, 1024, 64, 7)]


@pytest.mark.parametrize("fmt,rule", [(NV, 0), (MX, 0), (MX, 1)], ids=["nv", "mx-floor", "mx-ceil"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,page,skip", CACHE)
def test_write_and_read_are_the_oracle_bit_for_bit(T, H, D, page, skip, dtype, fmt, rule):
    g = gen(T * 7 + H)
    pages = -(-T // page) + 2
    c = make_cache(g, pages, H, D, page, fmt)
    before = {n: getattr(c, n).cpu().numpy().copy() for n in ("k_packed", "k_scales", "v_packed", "v_scales")}
    qkv = randn(g, T, 4 * H, D, dtype=dtype)
    k, v = qkv[:, H:2 * H], qkv[:, 3 * H:]
    k[:, :, 5] *= 30
    v[0] = 0
    slots = torch.randperm(pages * page, generator=g)[:T]
    if skip:
        slots[::skip] = -1 - slots[::skip]
    fp4.kv_write(c, k, v, slots.cuda(), rule=rule)
    keep = (slots >= 0).numpy()
    at = slots.numpy()[keep]
    for n, x in (("k", k), ("v", v)):
        gs = getattr(c, n + "_global_scale")
        packed, scales = ref.quantize_rows(x, fmt == NV, gs.cpu() if gs is not None else None, rule)
        for name, want in ((n + "_packed", packed), (n + "_scales", scales)):
            full = before[name]
            full[at // page, :, at % page] = want[keep]
            assert np.array_equal(getattr(c, name).cpu().numpy(), full), name  # the rest of the cache as it was
    for out_dtype in (BF, F32):
        kr, vr = fp4.kv_read(c, slots.cuda(), out_dtype)
        for n, got in (("k", kr), ("v", vr)):
            q = fp4.Quantized(fmt, getattr(c, n + "_packed")[at // page, :, at % page].contiguous(),
                              getattr(c, n + "_scales")[at // page, :, at % page].contiguous(), None, c.status, len(at), D)
            for h in range(H):
                one = fp4.Quantized(fmt, q.packed[:, h].contiguous(), q.scales[:, h].contiguous(),
                                    getattr(c, n + "_global_scale")[h:h + 1].contiguous() if fmt == NV else None, c.status, len(at), D)
                if len(at):
                    assert torch.equal(got[torch.from_numpy(keep), h], fp4.dequantize(one, out_dtype))
            assert not got[torch.from_numpy(~keep)].any()
    c.check()


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_write_and_read_where_places_are_formed_with_64_bits(dtype, fmt):
    """Pages of 2^20 tokens: the 32-bit division by the page size does not reach."""
    test_write_and_read_are_the_oracle_bit_for_bit(1000, 1, 32, 1 << 20, 7, dtype, fmt, 0)


def test_read_into_a_strided_view_leaves_its_neighbours():
    g = gen(3)
    c = make_cache(g, 3, 2, 64, 16, NV)
    slots = torch.tensor([5, -1, 47, 16]).cuda()
    buf = torch.full((4, 6, 64), 7.0, dtype=BF, device="cuda")
    k, v = fp4.kv_read(c, slots)
    fp4.kv_read(c, slots, k=buf[:, 1:3], v=buf[:, 4:])
    assert torch.equal(buf[:, 1:3], k) and torch.equal(buf[:, 4:], v)
    assert (buf[:, 0] == 7).all() and (buf[:, 3] == 7).all()


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_bad_slots_and_non_finite_values_set_the_status_and_nothing_else_breaks(fmt):
    g = gen(4)
    c = fp4.kv_cache(2, 2, 64, 16, fmt)
    k, v = randn(g, 4, 2, 64), randn(g, 4, 2, 64)
    slots = torch.tensor([3, 32, 9, 1 << 50]).cuda()  # 32 slots: the second and fourth are past them
    fp4.kv_write(c, k, v, slots)
    assert int(c.status.item()) == fp4.ERR_INDEX
    c.status.zero_()
    kr, _ = fp4.kv_read(c, slots)
    assert int(c.status.item()) == fp4.ERR_INDEX
    assert not kr[1].any() and not kr[3].any() and kr[0].any() and kr[2].any()
    c.status.zero_()
    k[1, 1, 7] = float("nan")
    v[2, 0, 0] = float("inf")
    want = fp4.kv_read(c, torch.tensor([3]).cuda())[0]
    fp4.kv_write(c, k, v, torch.tensor([3, 4, 5, -1]).cuda())
    assert int(c.status.item()) == fp4.ERR_NONFINITE
    c.status.zero_()
    assert torch.equal(fp4.kv_read(c, torch.tensor([3]).cuda())[0], want)
    with pytest.raises(fp4.FP4Error):
        c.status.fill_(fp4.ERR_INDEX)
        c.check()


def test_a_global_scale_that_is_no_normal_number_is_an_error():
    g = gen(5)
    for bad in (0.0, 1e-40, float("nan"), float("inf"), -1.0, 2e35):
        kg = torch.tensor([1 / 64, bad])
        c = fp4.kv_cache(1, 2, 64, 16, NV, kg, 1 / 64)
        fp4.kv_write(c, randn(g, 1, 2, 64), randn(g, 1, 2, 64), torch.tensor([0]).cuda())
        assert int(c.status.item()) == fp4.ERR_RANGE
        assert c.k_packed[0, 0, 0].any() and not c.k_packed[0, 1].any()


# ---------------------------------------------------------------- attention --

def check_attention(c, q, table, lens, scale, window, got=None):
    out, lse = got if got is not None else fp4.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale, window=window)
    c.check()
    k, v = sequences(c, table, lens)
    o, s, tol, ltol = ref.attention(q, k, v, lens, scale, window, c.fmt == MX)
    tol = tol + ref.HALF[q.dtype] * np.abs(o) + 1e-30
    err = np.abs(out.double().cpu().numpy() - o)
    assert (err <= tol).all(), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
    got_s = lse.double().cpu().numpy()
    empty = np.isinf(s)
    assert np.array_equal(np.isneginf(got_s), empty)
    assert (np.abs(got_s[~empty] - s[~empty]) <= ltol[~empty]).all(), np.max(np.abs(got_s[~empty] - s[~empty]) / ltol[~empty])
    return out, lse


ATTN = [  # lens, new tokens, kv heads, group, D, page, window
    ([1], 1, 1, 1, 64, 16, 0),
    ([17, 0, 33], 1, 2, 1, 128, 16, 0),
    ([137], 1, 8, 4, 128, 64, 0),
    ([31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 1, 2, 64, 48, 0),
    ([1000, 1, 257], 1, 2, 8, 128, 16, 0),
    ([300, 2, 0, 5], 4, 2, 3, 64, 32, 0),
    ([511], 7, 1, 5, 256, 64, 0),
    ([90, 400], 1, 4, 16, 128, 32, 0),
    ([90, 200], 2, 1, 24, 64, 32, 0),
    ([700, 3, 40], 2, 2, 4, 128, 80, 33),
    ([400, 77], 5, 1, 6, 64, 16, 1),
    ([2500], 1, 1, 4, 256, 128, 999),
    ([4097], 3, 1, 7, 128, 16, 0),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("lens,new,heads,group,dim,page,window", ATTN)
def test_attention(lens, new, heads, group, dim, page, window, fmt, dtype):
    g = gen(sum(lens) + new)
    width = -(-max(lens) // page) + 1
    c = make_cache(g, max(width, 1) + 3, heads, dim, page, fmt)
    table = tables(g, len(lens), width, c.num_pages)
    q = randn(g, len(lens), new, heads * group, dim, dtype=dtype)
    check_attention(c, q, table, lens, 1 / np.sqrt(dim) / 40, window)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_attention_with_sharp_scores_and_a_large_offset(fmt):
    """Scores of several hundred, most weights zero: the running maximum must carry them."""
    g = gen(11)
    c = make_cache(g, 9, 2, 128, 64, fmt)
    table = tables(g, 2, 8, 9)
    q = randn(g, 2, 1, 8, 128, scale=4.0)
    check_attention(c, q, table, [500, 77], 0.5, 0)
    check_attention(c, q, table, [500, 77], -0.5, 0)
    check_attention(c, q, table, [500, 77], 0.0, 0)


def test_attention_of_queries_of_every_size():
    """A query's magnitude must not matter: rows from 1e-30 to 1e30 beside each other."""
    g = gen(12)
    c = make_cache(g, 5, 1, 64, 32, NV)
    table = tables(g, 1, 4, 5)
    q = randn(g, 1, 1, 8, 64)
    sizes = torch.tensor([1e-38, 1e-30, 1e-8, 1.0, 1e4, 0.0, 300.0, 1e-3], device="cuda").to(BF)
    q = q * sizes[:, None]
    check_attention(c, q, table, [100], 1e-3, 0)
    check_attention(c, q.float(), table, [100], 1e-3, 0)


def test_attention_mxfp4_scales_over_the_whole_range():
    """Keys and values whose block scales lie far from one: tokens from 2^-60 to 2^60."""
    g = gen(13)
    c = make_cache(g, 4, 2, 128, 32, MX)
    table = tables(g, 1, 4, 4)
    for shift in (-60, 0, 60):
        c.v_scales.copy_(torch.randint(120 + shift, 131 + shift, c.v_scales.shape, generator=g, dtype=torch.uint8))
        c.k_scales.copy_(torch.randint(120 + shift, 131 + shift, c.k_scales.shape, generator=g, dtype=torch.uint8))
        check_attention(c, randn(g, 1, 2, 4, 128), table, [111], 2.0 ** -shift / 64, 0)
    # tokens of very different size next to each other
    tok = torch.randint(0, 60, (4, 1, 32, 1), generator=g, dtype=torch.uint8)
    c.v_scales.copy_((100 + tok + torch.randint(0, 8, c.v_scales.shape, generator=g, dtype=torch.uint8)))
    c.k_scales.fill_(120)
    check_attention(c, randn(g, 1, 1, 4, 128), table, [128], 0.01, 0)


def test_attention_zero_codes_and_zero_scales():
    g = gen(14)
    for fmt in (NV, MX):
        c = make_cache(g, 4, 1, 64, 16, fmt)
        c.k_scales.zero_()
        c.v_packed[1].zero_()
        table = tables(g, 1, 4, 4)
        check_attention(c, randn(g, 1, 1, 2, 64), table, [50], 0.125, 0)


def test_what_lies_behind_a_sequence_is_never_used():
    """NaN scale bytes in every slot past the end, and a page table whose unused entries name no page."""
    g = gen(15)
    for fmt in (NV, MX):
        c = make_cache(g, 8, 2, 128, 48, fmt)
        table = tables(g, 2, 4, 8)
        table[1] = torch.tensor([x for x in range(8) if x not in table[0].tolist()][:4], dtype=torch.int32)
        lens = [100, 35]
        q = randn(g, 2, 1, 4, 128)
        want = fp4.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32).cuda())
        for b, n in enumerate(lens):
            for j in range(n, 4 * 48):
                page = int(table[b, j // 48])
                c.k_scales[page, :, j % 48] = 0xFF
                c.v_scales[page, :, j % 48] = 0xFF
            table[b, -(-n // 48):] = -77 - b
        got = fp4.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32).cuda())
        c.check()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_and_lengths_set_the_status_and_spare_the_other_sequences():
    g = gen(16)
    c = make_cache(g, 6, 2, 64, 16, NV)
    table = tables(g, 3, 4, 6)
    q = randn(g, 3, 1, 4, 64)
    good = [64, 50, 20]
    want = fp4.kv_attention(q, c, table, torch.tensor(good, dtype=torch.int32).cuda())
    for page in (6, -1, 1 << 30, -(1 << 31)):
        bad = table.clone()
        bad[1, 2] = page
        got = fp4.kv_attention(q, c, bad, torch.tensor(good, dtype=torch.int32).cuda())
        assert int(c.status.item()) == fp4.ERR_INDEX
        c.status.zero_()
        for b in (0, 2):
            assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])
    for n in (65, -1, (1 << 31) - 1, -(1 << 31)):
        got = fp4.kv_attention(q, c, table, torch.tensor([64, n, 20], dtype=torch.int32).cuda())
        assert int(c.status.item()) == fp4.ERR_INDEX
        c.status.zero_()
        for b in (0, 2):
            assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])
    q[1, 0, 2, 5] = float("nan")
    got = fp4.kv_attention(q, c, table, torch.tensor(good, dtype=torch.int32).cuda())
    assert int(c.status.item()) == fp4.ERR_NONFINITE
    c.status.zero_()
    for b in (0, 2):
        assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])


def test_attention_of_a_fused_projection_s_view_and_without_lse():
    g = gen(17)
    c = make_cache(g, 4, 2, 64, 32, NV)
    table = tables(g, 2, 3, 4)
    qkv = randn(g, 2, 3, 12, 64)
    lens = torch.tensor([90, 60], dtype=torch.int32).cuda()
    want, lse = fp4.kv_attention(qkv[:, :, :8].contiguous(), c, table, lens)
    got, _ = fp4.kv_attention(qkv[:, :, :8], c, table, lens)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    ws = fp4.kv_attention_workspace(qkv[:, :, :8], c, table)
    assert fp4.lib().fp4_kv_attention(c._ref, qkv.data_ptr(), fp4.BF16, 2, 3, 8, 12 * 64, table.data_ptr(), 3, lens.data_ptr(),
                                      0.125, 0, out.data_ptr(), None, ws.data_ptr(), ws.numel(), c.status.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == fp4.OK
    assert torch.equal(out, want)
    none = fp4.kv_attention(qkv[:0, :, :8], c, table[:0], lens[:0])
    assert none[0].shape == (0, 3, 8, 64)
    empty = fp4.kv_attention(qkv[:, :, :8], c, table[:, :0].contiguous(), torch.zeros(2, dtype=torch.int32).cuda())
    assert not empty[0].any() and torch.isneginf(empty[1]).all()


def test_attention_repeats_bit_for_bit_and_its_workspace_serves_smaller_calls():
    g = gen(18)
    c = make_cache(g, 80, 2, 128, 64, NV)
    table = tables(g, 3, 70, 80)
    q = randn(g, 3, 2, 8, 128)
    lens = torch.tensor([4400, 100, 2000], dtype=torch.int32).cuda()
    ws = fp4.kv_attention_workspace(q, c, table)
    first = fp4.kv_attention(q, c, table, lens, workspace=ws)
    for _ in range(5):
        fp4.kv_attention(q[:1], c, table[:1], lens[:1], workspace=ws)
        fp4.kv_attention(q[:, :1].contiguous(), c, table, lens, workspace=ws)
        again = fp4.kv_attention(q, c, table, lens, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    check_attention(c, q, table, [4400, 100, 2000], 128 ** -0.5, 0)


@pytest.mark.parametrize("B,longest,heads,group", [(40, 900, 2, 3), (150, 700, 1, 2), (300, 300, 1, 1)])
def test_attention_of_many_sequences(B, longest, heads, group):
    """Batches beyond a warp's and beyond a CTA's scan of the lengths; sequences share pages."""
    g = gen(B)
    c = make_cache(g, 30, heads, 64, 32, NV)
    width = -(-longest // 32)
    table = torch.randint(0, 30, (B, width), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    lens[3], lens[B - 1] = 0, longest
    check_attention(c, randn(g, B, 1, heads * group, 64), table, lens, 0.003, 0)


def test_attention_of_more_units_than_the_gpu_holds_at_once():
    g = gen(41)
    B, heads = 1600, 4
    c = make_cache(g, 9, heads, 64, 16, NV)
    table = torch.randint(0, 9, (B, 20), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, 24, (B,), generator=g).tolist()
    lens[1111] = 320
    check_attention(c, randn(g, B, 1, heads, 64), table, lens, 0.003, 0)


WIDE = [  # lens, new, heads, group, dim, window: tables for 1500 tokens, whatever is there of them
    ([0, 1, 15, 16, 17, 0, 127, 128, 129, 300, 1500], 1, 2, 3, 64, 0),
    ([1], 1, 1, 1, 128, 0),
    ([130], 1, 8, 4, 128, 0),
    ([257, 1499, 3], 4, 3, 5, 128, 0),
    ([0, 0, 0], 2, 2, 2, 64, 0),
    ([1500, 700, 20], 1, 2, 8, 256, 0),
    ([1500, 700, 20], 2, 1, 9, 128, 1100),
    ([0] * 60 + [1500] + [2] * 40, 1, 4, 2, 64, 0),
    ([129] * 90, 1, 2, 1, 128, 0),
    ([1 + 11 * i for i in range(130)], 1, 3, 1, 64, 0),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("lens,new,heads,group,dim,window", WIDE)
def test_attention_of_short_sequences_under_a_wide_table(lens, new, heads, group, dim, window, fmt, dtype):
    """The tokens are shared out over all CTAs: shares that end inside a unit's start, cross many units, or are a part of one."""
    g = gen(len(lens) + dim + new)
    c = make_cache(g, 40, heads, dim, 48, fmt)
    table = torch.randint(0, 40, (len(lens), 32), generator=g, dtype=torch.int32).cuda()
    for b, n in enumerate(lens):
        table[b, -(-n // 48):] = -1
    check_attention(c, randn(g, len(lens), new, heads * group, dim, dtype=dtype), table, lens, 1 / np.sqrt(dim) / 40, window)
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("n,new,group,window", [(12900, 1, 1, 0), (60001, 1, 2, 0), (9000, 3, 7, 0), (70000, 1, 1, 40000)])
def test_attention_of_one_sequence_in_many_pieces(n, new, group, window, fmt):
    """One sequence and head over the whole GPU: dozens to hundreds of pieces to join."""
    g = gen(n)
    c = make_cache(g, 50, 1, 64, 64, fmt)
    table = torch.randint(0, 50, (1, -(-n // 64)), generator=g, dtype=torch.int32).cuda()
    check_attention(c, randn(g, 1, new, group, 64), table, [n], 0.003, window)


def test_attention_calls_of_different_shapes_take_turns_on_one_workspace():
    g = gen(43)
    c = make_cache(g, 60, 2, 128, 64, NV)
    big, small = tables(g, 4, 50, 60), tables(g, 1, 50, 60)
    qb, qs = randn(g, 4, 2, 16, 128), randn(g, 1, 1, 4, 128)
    lb = torch.tensor([3200, 64, 1999, 0], dtype=torch.int32).cuda()
    ls = torch.tensor([3111], dtype=torch.int32).cuda()
    want_b, want_s = fp4.kv_attention(qb, c, big, lb), fp4.kv_attention(qs, c, small, ls)
    want_f = fp4.kv_attention(qs.float(), c, small, ls)
    ws = fp4.kv_attention_workspace(qb, c, big)
    for _ in range(4):
        for args, want in (((qs, c, small, ls), want_s), ((qb, c, big, lb), want_b), ((qs.float(), c, small, ls), want_f)):
            got = fp4.kv_attention(*args, workspace=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_captured_once_follows_growing_lengths():
    g = gen(44)
    c = make_cache(g, 70, 2, 64, 16, NV)
    table = tables(g, 2, 60, 70)
    q = randn(g, 2, 1, 6, 64)
    lens = torch.tensor([5, 0], dtype=torch.int32).cuda()
    ws = fp4.kv_attention_workspace(q, c, table)
    fp4.kv_attention(q, c, table, lens, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fp4.kv_attention(q, c, table, lens, workspace=ws)
    for n in ([5, 0], [300, 17], [960, 959], [1, 513]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(c, q, table, n, 0.125, 0, got=(out, lse))
    del graph


def test_attention_captured_once_follows_growing_lengths_under_a_wide_table():
    """The tokens are shared out anew by every replay."""
    g = gen(46)
    c = make_cache(g, 70, 2, 64, 64, NV)
    table = torch.randint(0, 70, (3, 80), generator=g, dtype=torch.int32).cuda()
    q = randn(g, 3, 2, 6, 64)
    lens = torch.tensor([5, 0, 1], dtype=torch.int32).cuda()
    ws = fp4.kv_attention_workspace(q, c, table)
    fp4.kv_attention(q, c, table, lens, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fp4.kv_attention(q, c, table, lens, workspace=ws)
    for n in ([5, 0, 1], [300, 17, 5120], [5120, 5119, 2], [0, 0, 0], [1, 1300, 129]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(c, q, table, n, 0.125, 0, got=(out, lse))  # 64 ** -0.5, the default
    del graph


# ------------------------------------------------------------------- linear --

def make_weight(g, n, k, fmt, dtype=BF):
    w = randn(g, n, k, dtype=dtype, scale=0.02)
    if n and k:
        w[0, 0] = 1.5
    q = fp4.nvfp4_quantize_padded(w) if fmt == NV else fp4.mxfp4_quantize_padded(w)
    q.check()
    dec = ref.decode(q.packed.cpu().numpy(), q.scales.cpu().numpy(), fmt == NV, q.global_scale.item() if fmt == NV else 1.0)
    return fp4.linear_weight(q), dec[:, :k]


def check_linear(x, w, dec, out_dtype, y=None):
    y = fp4.linear(x, w, out_dtype=out_dtype) if y is None else y
    w.check()
    want, tol = ref.linear(x, dec)
    tol = tol + ref.HALF[out_dtype] * np.abs(want) + 1e-30
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
    return y


LINEAR = [(1, 1, 32), (1, 128, 256), (2, 129, 64), (3, 127, 512), (5, 1001, 1440), (8, 256, 4096), (9, 300, 320), (16, 640, 992),
          (17, 130, 2080), (33, 200, 544), (64, 384, 1024), (65, 100, 288), (131, 77, 256), (1, 4096, 4096)]


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["to-bf16", "to-f32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("rows,n,k", LINEAR)
def test_linear(rows, n, k, fmt, dtype, out_dtype):
    g = gen(rows * n + k)
    w, dec = make_weight(g, n, k, fmt)
    check_linear(randn(g, rows, k, dtype=dtype), w, dec, out_dtype)


@pytest.mark.parametrize("fmt,k", [(NV, 255), (NV, 241), (NV, 31), (MX, 1), (MX, 33), (MX, 255)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_linear_of_a_padded_weight_and_strided_rows(fmt, k, dtype):
    g = gen(k)
    w, dec = make_weight(g, 70, k, fmt)
    x = randn(g, 6, 2 * k + 3, dtype=dtype)
    x[:, k:] = float("nan")  # beside the rows
    check_linear(x[:, :k], w, dec, dtype)
    check_linear(x[::2, :k], w, dec, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
@pytest.mark.parametrize("rows,n,k", [(200, 70, 160), (401, 129, 96), (3, 40, 20000), (2, 20000, 160), (1, 4000, 14464), (90, 1300, 4096), (40, 300, 2080)])
def test_linear_beyond_one_tile(rows, n, k, fmt, dtype):
    """Several tiles of rows, long and short K, more bands than SMs, K shares of unequal length."""
    g = gen(rows + n + k)
    w, dec = make_weight(g, n, k, fmt)
    check_linear(randn(g, rows, k, dtype=dtype), w, dec, F32)


def test_calls_on_a_given_stream():
    g = gen(27)
    w, dec = make_weight(g, 300, 512, NV)
    x = randn(g, 3, 512)
    c = make_cache(g, 4, 2, 64, 16, NV)
    table = tables(g, 1, 4, 4)
    q = randn(g, 1, 1, 2, 64)
    lens = torch.tensor([60], dtype=torch.int32).cuda()
    want = fp4.linear(x, w), fp4.kv_attention(q, c, table, lens)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        y, o = torch.empty_like(want[0]), torch.empty_like(want[1])
        ws = fp4.linear_workspace(3, w), fp4.kv_attention_workspace(q, c, table)
        torch.cuda.synchronize()
        fp4.linear(x, w, out=y, workspace=ws[0], stream=given)
        fp4.kv_attention(q, c, table, lens, out=o, workspace=ws[1], stream=given)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(o, want[1])


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_calls_on_a_given_stream_allocate_for_it(handle):
    """Without workspaces or outputs, the current stream held up: what the calls allocate belongs to the given stream."""
    g = gen(76)
    c = make_cache(g, 80, 2, 64, 32, NV)
    w = fp4.linear_weight(fp4.nvfp4_quantize(randn(g, 300, 2048, scale=0.02)))
    table, lens = tables(g, 2, 64, 80), torch.tensor([2000, 1200], dtype=torch.int32).cuda()
    q, x, slots = randn(g, 2, 1, 8, 64), randn(g, 20, 2048), torch.arange(64).cuda()
    want = [fp4.linear(x, w), *fp4.kv_attention(q, c, table, lens), *fp4.kv_read(c, slots)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = side.cuda_stream if handle else side
    torch.cuda._sleep(20_000_000)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        got = [fp4.linear(x, w, stream=given), *fp4.kv_attention(q, c, table, lens, stream=given), *fp4.kv_read(c, slots, stream=given)]
        del junk[:1]
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    torch.cuda.synchronize()
    c.check()
    w.check()


def test_linear_rows_of_every_size_and_empty_ones():
    g = gen(21)
    for fmt in (NV, MX):
        w, dec = make_weight(g, 150, 512, fmt)
        x = randn(g, 7, 512)
        x *= torch.tensor([1e-38, 1e-20, 1.0, 0.0, 1e20, 3e37, 1e-5], device="cuda").to(BF)[:, None]
        x[2, ::7] *= 1000  # outlier channels
        check_linear(x, w, dec, F32)
        check_linear(x.float() * 1.2345, w, dec, F32)
    assert fp4.linear(x[:0], w).shape == (0, 150)
    assert fp4.linear(x.view(7, 1, 512)[:3], w).shape == (3, 1, 150)
    assert torch.equal(fp4.linear(x.view(7, 1, 512)[:3], w).view(3, 150), fp4.linear(x[:3], w))


def test_linear_mxfp4_scales_over_the_whole_range():
    g = gen(22)
    n, k = 140, 256
    packed = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda()
    for lo, hi in ((0, 30), (60, 190), (230, 245)):
        scales = torch.randint(lo, hi, (n, k // 32), generator=g, dtype=torch.uint8).cuda()
        q = fp4.Quantized(MX, packed, scales, None, fp4.new_status("cuda"), n, k)
        dec = ref.decode(packed.cpu().numpy(), scales.cpu().numpy(), False)
        x = randn(g, 3, k) * 2.0 ** -10
        y = fp4.linear(x, fp4.linear_weight(q), out_dtype=F32)
        want, tol = ref.linear(x, dec)
        err = np.abs(y.double().cpu().numpy() - want)
        # fp32 results below the smallest normal number are spaced 2^-149
        assert (err <= tol + 2.0 ** -24 * np.abs(want) + k * 2.0 ** -149).all()


def test_linear_nvfp4_every_scale_byte_and_code():
    g = gen(23)
    n, k = 127, 16 * 32
    codes = torch.arange(256, dtype=torch.uint8).repeat(n * k // 512).view(n, k // 2).cuda()
    scales = (torch.arange(n * 32) % 127).to(torch.uint8).view(n, 32).cuda()
    q = fp4.Quantized(NV, codes, scales, torch.tensor([0.37]).cuda(), fp4.new_status("cuda"), n, k)
    dec = ref.decode(codes.cpu().numpy(), scales.cpu().numpy(), True, float(np.float32(0.37)))
    for dtype in (BF, F32):
        check_linear(randn(g, 4, k, dtype=dtype), fp4.linear_weight(q), dec, F32)


def test_linear_non_finite_rows_set_the_status_and_spare_the_others():
    g = gen(24)
    for fmt in (NV, MX):
        w, dec = make_weight(g, 200, 320, fmt)
        for rows in (4, 12):
            x = randn(g, rows, 320)
            want = fp4.linear(x, w)
            x[1, 77] = float("inf")
            x[2, 3] = float("nan")
            got = fp4.linear(x, w)
            assert int(w.status.item()) == fp4.ERR_NONFINITE
            w.status.zero_()
            keep = [r for r in range(rows) if r not in (1, 2)]
            assert torch.equal(got[keep], want[keep])


def test_linear_rows_do_not_depend_on_their_batch():
    """A row's result is the same alone and in a batch that takes the same tile."""
    g = gen(25)
    w, dec = make_weight(g, 256, 1024, NV)
    x = randn(g, 8, 1024)
    assert torch.equal(fp4.linear(x, w)[:5], fp4.linear(x[:5], w))


def test_linear_writes_its_output_alone():
    g = gen(26)
    w, dec = make_weight(g, 77, 96, MX)
    buf = torch.full((3 * 77 + 64,), 5.0, dtype=BF, device="cuda")
    fp4.linear(randn(g, 3, 96), w, out=buf[32:32 + 231].view(3, 77))
    assert (buf[:32] == 5).all() and (buf[32 + 231:] == 5).all()


def test_the_helpers_refuse_what_does_not_fit():
    g = gen(28)
    w, _ = make_weight(g, 70, 64, NV)
    x = randn(g, 3, 64)
    for bad in (lambda: fp4.linear(x[:, :32], w), lambda: fp4.linear(x.half(), w), lambda: fp4.linear(x.t().contiguous().t(), w),
                lambda: fp4.linear(x, w, out=torch.empty(3, 71, dtype=BF, device="cuda")), lambda: fp4.linear(x.cpu(), w),
                lambda: fp4.linear(x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")[8:])):
        with pytest.raises((ValueError, TypeError, fp4.FP4Error)):
            bad()
    c = make_cache(g, 4, 2, 64, 16, NV)
    k, slots = randn(g, 3, 2, 64), torch.tensor([1, 2, 3]).cuda()
    table, lens, q = tables(g, 1, 4, 4), torch.tensor([60], dtype=torch.int32).cuda(), randn(g, 1, 1, 4, 64)
    for bad in (lambda: fp4.kv_write(c, k, k.float(), slots), lambda: fp4.kv_write(c, k[:, :1], k[:, :1], slots),
                lambda: fp4.kv_write(c, k, k, slots.int()), lambda: fp4.kv_write(c, k, k, slots.cpu()),
                lambda: fp4.kv_write(c, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots), lambda: fp4.kv_write(c, k, k, slots, rule=5),
                lambda: fp4.kv_read(c, slots, out_dtype=torch.float16), lambda: fp4.kv_attention(q[..., :32], c, table, lens),
                lambda: fp4.kv_attention(q, c, table.long(), lens), lambda: fp4.kv_attention(q, c, table, lens.repeat(2)),
                lambda: fp4.kv_attention(q[:, :, :3], c, table, lens), lambda: fp4.kv_attention(q, c, table, lens, window=-1),
                lambda: fp4.kv_attention(q, c, table, lens, scale=float("nan")), lambda: fp4.kv_attention(q.half(), c, table, lens),
                lambda: fp4.kv_attention(q, c, table, lens, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                lambda: fp4.KVCache(NV, c.k_packed, c.k_scales, c.v_packed, c.v_scales), lambda: fp4.KVCache(MX, c.k_packed, c.k_scales, c.v_packed, c.v_scales),
                lambda: fp4.LinearWeight(NV, w.packed, w.scales_mma[:-1], w.global_scale, 70, 64)):
        with pytest.raises((ValueError, TypeError, fp4.FP4Error)):
            bad()
    c.check()
    w.check()


# ------------------------------------------------------------- all together --

def step(c, wqkv, wout, x, slots, table, lens, heads, group, ws):
    """One decoding step's attention layer: projection, cache write, attention, projection."""
    T, D = x.shape[0], c.head_dim
    qkv = fp4.linear(x, wqkv, workspace=ws["a"]).view(T, heads * (group + 2), D)
    q, k, v = qkv[:, :heads * group], qkv[:, heads * group:heads * (group + 1)], qkv[:, heads * (group + 1):]
    fp4.kv_write(c, k, v, slots)
    out, _ = fp4.kv_attention(q[:, None], c, table, lens, workspace=ws["b"])
    return fp4.linear(out.view(T, -1), wout, workspace=ws["c"])


def setup_step(seed, fmt):
    g = gen(seed)
    heads, group, D, T, width = 2, 4, 64, 3, 5
    c = make_cache(g, 20, heads, D, 16, fmt)
    wqkv, dq = make_weight(g, heads * (group + 2) * D, 256, fmt)
    wout, do = make_weight(g, 256, heads * group * D, fmt)
    table = torch.randperm(20, generator=g)[:T * width].view(T, width).int().cuda()
    lens = torch.tensor([33, 80, 1], dtype=torch.int32).cuda()
    pos = (lens - 1).long()
    slots = table.gather(1, (pos // 16)[:, None]).long()[:, 0] * 16 + pos % 16
    ws = {"a": fp4.linear_workspace(T, wqkv), "c": fp4.linear_workspace(T, wout),
          "b": torch.zeros(fp4.lib().fp4_kv_attention_workspace_bytes(c._ref, T, 1, heads * group, width), dtype=torch.uint8, device="cuda")}
    return g, (c, wqkv, wout), (slots, table, lens, heads, group, ws), (dq, do)


@pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])
def test_a_decoding_step(fmt):
    g, (c, wqkv, wout), rest, (dq, do) = setup_step(31, fmt)
    slots, table, lens, heads, group, ws = rest
    x = randn(g, 3, 256)
    y = step(c, wqkv, wout, x, *rest)
    torch.cuda.synchronize()
    c.check(), wqkv.check(), wout.check()
    # each operator on the values its predecessor gave
    qkv = fp4.linear(x, wqkv)
    check_linear(x, wqkv, dq, BF, qkv)
    qkv = qkv.view(3, heads * (group + 2), 64)
    q = qkv[:, :heads * group][:, None]
    kr, vr = fp4.kv_read(c, slots)
    packed, scales = ref.quantize_rows(qkv[:, heads * group:heads * (group + 1)], fmt == NV, c.k_global_scale.cpu() if fmt == NV else None)
    assert np.array_equal(c.k_packed.cpu().numpy()[slots.cpu() // 16, :, slots.cpu() % 16], packed)
    out, _ = check_attention(c, q.contiguous(), table, lens.tolist(), 0.125, 0)
    check_linear(out.view(3, -1), wout, do, BF, y)


def test_a_decoding_step_captured_and_replayed():
    g, handles, rest, _ = setup_step(32, NV)
    x = randn(g, 3, 256)
    step(*handles, x, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(*handles, x, *rest)
    for seed in (1, 2, 3):
        new = randn(gen(seed), 3, 256)
        x.copy_(new)
        graph.replay()
        got = y.clone()
        want = step(*handles, new, *rest)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    del graph


def test_steps_on_two_streams_with_their_own_workspaces():
    a, b = setup_step(33, NV), setup_step(34, MX)
    xs = [randn(a[0], 3, 256), randn(b[0], 3, 256)]
    want = [step(*s[1], x, *s[2]) for s, x in zip((a, b), xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for s, x, st in zip((a, b), xs, streams):
            with torch.cuda.stream(st):
                got.append(step(*s[1], x, *s[2]))
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
