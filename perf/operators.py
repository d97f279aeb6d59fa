"""The operators of single-token serving in FP4, as cases to measure.

  cache      keys and values quantised as they are written into a paged FP4 cache, and read back
  attention  attention of one or a few new tokens a sequence over that cache
  linear     product of a few rows of unquantised activations with an FP4 weight

`own = False` computes them in their plain form (elementary torch operations in 32 bits, 64 where a value next to a
rounding border decides), `own = True` through block_scaled_fp4_reduce_b200.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = {"nvfp4": 16, "mxfp4": 32}


def listed():
    return [
        # one decoding step of 64 sequences: a token each, latency is all that counts
        dict(name="cache 64 tokens", op="cache", fmt="nvfp4", dtype="bf16", tokens=64, heads=8, dim=128, page=64, fused=1, skip=0),
        # a prompt of 8192 tokens written at once, then read back for the next chunk's dense attention
        dict(name="cache 8192 tokens", op="cache", fmt="nvfp4", dtype="bf16", tokens=8192, heads=8, dim=128, page=64, fused=1, skip=0),
        # fp32 activations, odd counts, small pages, padding tokens in the batch
        dict(name="cache odd f32", op="cache", fmt="mxfp4", dtype="f32", tokens=2051, heads=5, dim=96, page=16, fused=0, skip=3),
        # one short conversation: the latency of a call
        dict(name="attention short", op="attention", fmt="nvfp4", dtype="bf16", batch=1, longest=137, heads=8, group=4, dim=128, page=64, new=1, window=0, ragged=0),
        # a serving batch of ragged lengths
        dict(name="attention batch", op="attention", fmt="nvfp4", dtype="bf16", batch=32, longest=8192, heads=8, group=4, dim=128, page=64, new=1, window=0, ragged=1),
        # two very long contexts: the long axis has to be split
        dict(name="attention long", op="attention", fmt="nvfp4", dtype="bf16", batch=2, longest=131071, heads=8, group=8, dim=128, page=128, new=1, window=0, ragged=0),
        # verification of four drafted tokens, sliding window, odd group, an empty sequence in the batch
        dict(name="attention draft", op="attention", fmt="mxfp4", dtype="bf16", batch=23, longest=4099, heads=4, group=3, dim=64, page=48, new=4, window=1501, ragged=1),
        # fp32 queries and answers
        dict(name="attention f32", op="attention", fmt="nvfp4", dtype="f32", batch=5, longest=3001, heads=2, group=5, dim=256, page=32, new=1, window=0, ragged=1),
        # the square projection of the 7B-class weight set for one token
        dict(name="linear 1 row", op="linear", fmt="nvfp4", dtype="bf16", out="bf16", rows=1, n=4096, k=4096),
        # its up-projection for a batch of 16 tokens, MXFP4
        dict(name="linear 16 rows", op="linear", fmt="mxfp4", dtype="bf16", out="bf16", rows=16, n=14336, k=4096),
        # fp32 in and out, odd rows and an odd number of outputs
        dict(name="linear odd f32", op="linear", fmt="nvfp4", dtype="f32", out="f32", rows=5, n=1001, k=14336),
        # its down-projection for a batch of 64 tokens
        dict(name="linear 64 rows", op="linear", fmt="nvfp4", dtype="bf16", out="bf16", rows=64, n=4096, k=14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attention", "attention", "linear", "linear"])
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "cache":
        heads, dim = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 96, 128, 160, 256])
        return dict(op=op, fmt=fmt, dtype=dtype, tokens=_log(rng, 1, 8 * 1024 * 1024 // (heads * dim)), heads=heads, dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128]), fused=rng.randint(0, 1), skip=rng.choice([0, 0, 3, 7]))
    if op == "attention":
        batch, heads, dim = _log(rng, 1, 48), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        most = min(131072, 64 * 1024 * 1024 // (batch * heads * dim))
        return dict(op=op, fmt=fmt, dtype=dtype, batch=batch, longest=_log(rng, 1, most), heads=heads, group=rng.choice([1, 2, 3, 4, 6, 8, 16]),
                    dim=dim, page=rng.choice([16, 32, 48, 64, 128]), new=rng.choice([1, 1, 1, 2, 4, 7]),
                    window=rng.choice([0, 0, 0, _log(rng, 1, most)]), ragged=rng.randint(0, 1))
    return dict(op=op, fmt=fmt, dtype=dtype, out=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 64), n=_log(rng, 64, 14336),
                k=32 * _log(rng, 2, 448))


# ------------------------------------------------------------------ plain forms --

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e4m3(t):
    """The E4M3 value nearest to t >= 0 (in 64 bits), ties to the even code, at most 448."""
    t = t.clamp(max=448.0)
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t)[1].clamp(min=-5) - 4)
    return torch.round(t / step) * step


def _e2m1(v):
    """E2M1 codes: nearest value, ties to the even code, at most 6, the sign kept."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return c + torch.signbit(v).to(torch.uint8) * 8


def _quantize(x, fmt, g):
    """x [..., D], g broadcast over all but the last axis: packed codes [..., D/2] and scale bytes [..., D/G]."""
    b = x.float().unflatten(-1, (-1, GROUP[fmt]))
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        s = _e4m3(amax.double() / (6.0 * g[..., None].double())).float()
        d = (s * g[..., None])[..., None]
        c = torch.where(s[..., None] > 0, _e2m1(b / torch.where(d > 0, d, 1.0)), 0)
        scale = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
        c = _e2m1(torch.ldexp(b.double(), -e[..., None]).float())
        scale = (e + 127).to(torch.uint8)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale


def _values(packed, scale, fmt, g):
    """The values that codes and scales stand for, in 32 bits."""
    c = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    p = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)[c.int()]
    p = p.unflatten(-1, (-1, GROUP[fmt]))
    if fmt == "nvfp4":
        y = p * scale.view(torch.float8_e4m3fn).float()[..., None] * g[..., None, None]
    else:
        y = torch.ldexp(p, (scale.int() - 127)[..., None])
    return y.flatten(-2)


def _plain_cache(s):
    c, ps = s["cache"], s["page"]
    keep = s["slots"] >= 0
    page, off = (s["slots"].clamp(min=0) // ps), (s["slots"].clamp(min=0) % ps)
    at = (page[keep], slice(None), off[keep])
    kp, ks = _quantize(s["k"], s["fmt"], c["k_global_scale"])
    vp, vs = _quantize(s["v"], s["fmt"], c["v_global_scale"])
    c["k_packed"][at], c["k_scales"][at] = kp[keep], ks[keep]
    c["v_packed"][at], c["v_scales"][at] = vp[keep], vs[keep]
    k = _values(c["k_packed"][page, :, off], c["k_scales"][page, :, off], s["fmt"], c["k_global_scale"])
    v = _values(c["v_packed"][page, :, off], c["v_scales"][page, :, off], s["fmt"], c["v_global_scale"])
    zero = ~keep[:, None, None]
    return {"k": k.masked_fill(zero, 0).to(s["k"].dtype), "v": v.masked_fill(zero, 0).to(s["v"].dtype)}


def _visible(lens, new, longest, window):
    """[batch, new, longest]: which cached tokens each new token sees."""
    pos = (lens[:, None] - new + torch.arange(new, device=lens.device))[..., None]
    j = torch.arange(longest, device=lens.device)
    return (j <= pos) & (j > pos - window) if window else j <= pos


def _plain_attention(s):
    c, q = s["cache"], s["q"].float()
    B, L, HQ, D = q.shape
    H, n = s["heads"], s["longest"]
    table = s["page_table"].long()
    k = _values(c["k_packed"][table], c["k_scales"][table], s["fmt"], c["k_global_scale"][:, None])
    k = k.transpose(2, 3).flatten(1, 2)[:, :n].transpose(1, 2)  # [B, H, n, D]
    qg = q.unflatten(2, (H, HQ // H)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, L * group, D]
    see = _visible(s["seq_lens"], L, n, s["window"])[:, None].repeat_interleave(HQ // H, 2)
    x = torch.where(see, qg @ k.transpose(2, 3) * s["scale"], -math.inf)
    del k
    m = x.amax(-1, keepdim=True)
    p = torch.where(see, torch.exp(x - torch.where(m > -math.inf, m, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    v = _values(c["v_packed"][table], c["v_scales"][table], s["fmt"], c["v_global_scale"][:, None])
    v = v.transpose(2, 3).flatten(1, 2)[:, :n].transpose(1, 2)
    o = p @ v / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    back = lambda t: t.unflatten(2, (L, HQ // H)).transpose(1, 2).flatten(2, 3)  # noqa: E731
    return {"out": back(o).to(s["q"].dtype), "lse": back(lse)}


def _plain_linear(s):
    w = _values(s["packed"], s["scales"], s["fmt"], s["global_scale"])
    return (s["x"].float() @ w.T).to(TYPES[s["out"]])


# ------------------------------------------------------------------- the states --

def _table(gen, pages, batch, width):
    """A page table whose pages lie scattered over the cache."""
    return torch.randperm(pages, generator=gen, device=DEV)[: batch * width].view(batch, width)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    case = dict(case)
    fmt, dtype = case["fmt"], TYPES[case["dtype"]]
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        w = rand(n, k) * 0.02
        w = torch.where(torch.rand(n, k, generator=gen, device=DEV) < 0.0005, w * 30, w).to(torch.bfloat16)
        g = (w.abs().amax().float() / 2688.0).reshape(1)
        packed, scales = _quantize(w, fmt, g)
        # activations with heavy tails: Student-t with three degrees of freedom
        x = (rand(case["rows"], k) / (rand(3, case["rows"], k).square().sum(0) / 3).sqrt() * 0.5).to(dtype)
        nb, kt = scales.shape[1], -(-scales.shape[1] // 4)
        tiles = torch.zeros(-(-n // 128) * 128, kt * 4, dtype=torch.uint8, device=DEV)
        tiles[:n, :nb] = scales  # the tensor cores' scale layout, which a program keeps with its weights
        tiles = tiles.view(-1, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()
        return dict(case, x=x, packed=packed, scales=scales, scales_mma=tiles, global_scale=g)
    H, D, ps = case["heads"], case["dim"], case["page"]
    if case["op"] == "cache":
        T = case["tokens"]
        pages = -(-T // ps) + 3
        fill = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=DEV)  # noqa: E731
        slots = _table(gen, pages, 1, -(-T // ps))[0]
        slots = (slots[:, None] * ps + torch.arange(ps, device=DEV)).flatten()[:T].contiguous()
        if case["skip"]:
            slots[:: case["skip"]] = -1  # padding tokens of the batch
        # keys with a few strong channels, as rotary attention has them
        k, v = rand(T, H, D), rand(T, H, D)
        k[..., :: 31] *= 8
        if case["fused"]:  # views of one projection's output, query heads before them
            qkv = torch.zeros(T, 5 * H, D, dtype=dtype, device=DEV)
            qkv[:, 3 * H: 4 * H], qkv[:, 4 * H:] = k, v
            k, v = qkv[:, 3 * H: 4 * H], qkv[:, 4 * H:]
        else:
            k, v = k.to(dtype), v.to(dtype)
        cache = dict(k_packed=fill(pages, H, ps, D // 2), k_scales=fill(pages, H, ps, D // GROUP[fmt]),
                     v_packed=fill(pages, H, ps, D // 2), v_scales=fill(pages, H, ps, D // GROUP[fmt]),
                     k_global_scale=_calibrated(gen, H, 36.0), v_global_scale=_calibrated(gen, H, 4.5))
        return dict(case, k=k, v=v, slots=slots, cache=cache)
    B, n = case["batch"], case["longest"]
    width = -(-n // ps)
    pages = B * width + 2
    cache = {}
    for name, strong, bound in (("k", 8.0, 36.0), ("v", 1.0, 4.5)):
        x = torch.randn(pages, H, ps, D, generator=gen, device=DEV, dtype=torch.bfloat16)
        x[..., :: 31] *= strong
        g = _calibrated(gen, H, bound)
        cache[name + "_packed"], cache[name + "_scales"] = _quantize(x, fmt, g[:, None])
        cache[name + "_global_scale"] = g
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    if case["ragged"] and B > 1:
        some = torch.randint(0, n + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        some[0], some[1] = n, 0
        lens = some
    q = rand(B, case["new"], H * case["group"], D).to(dtype)
    return dict(case, q=q, cache=cache, page_table=_table(gen, pages, B, width).int(), seq_lens=lens, scale=1.0 / math.sqrt(D))


def _calibrated(gen, heads, bound):
    """A global scale for each head from a bound on its values, as a calibration run gives it: a few values pass it."""
    return bound * (1 + 0.2 * torch.rand(heads, generator=gen, device=DEV)) / 2688.0


# ----------------------------------------------------------------------- passes --

def run(state):
    if not own:
        return {"cache": _plain_cache, "attention": _plain_attention, "linear": _plain_linear}[state["op"]](state)
    import block_scaled_fp4_reduce_b200 as fp4

    if "handle" not in state:  # the handle and the workspace that a serving program keeps
        fmt = fp4.NVFP4 if state["fmt"] == "nvfp4" else fp4.MXFP4
        if state["op"] == "linear":
            state["handle"] = fp4.LinearWeight(fmt, state["packed"], state["scales_mma"], state["global_scale"], state["n"], state["k"])
            state["workspace"] = fp4.linear_workspace(state["rows"], state["handle"])
        else:
            state["handle"] = fp4.KVCache(fmt, **state["cache"])
        if state["op"] == "attention":
            state["workspace"] = fp4.kv_attention_workspace(state["q"], state["handle"], state["page_table"])
    if state["op"] == "linear":
        return fp4.linear(state["x"], state["handle"], out_dtype=TYPES[state["out"]], workspace=state["workspace"])
    if state["op"] == "cache":
        fp4.kv_write(state["handle"], state["k"], state["v"], state["slots"])
        k, v = fp4.kv_read(state["handle"], state["slots"], out_dtype=state["k"].dtype)
        return {"k": k, "v": v}
    out, lse = fp4.kv_attention(state["q"], state["handle"], state["page_table"], state["seq_lens"], scale=state["scale"],
                                window=state["window"], workspace=state["workspace"])
    return {"out": out, "lse": lse}


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear":
        w = c["n"] * c["k"] * (0.5 + 1 / GROUP[c["fmt"]])
        return {"bytes": w + c["rows"] * (c["k"] * size + c["n"] * (2 if c["out"] == "bf16" else 4)), "flops": 2.0 * c["rows"] * c["n"] * c["k"]}
    held = c["heads"] * c["dim"] * (0.5 + 1 / GROUP[c["fmt"]])  # bytes of one token's keys
    if c["op"] == "cache":
        values = c["heads"] * c["dim"]
        kept = c["tokens"] - (-(-c["tokens"] // c["skip"]) if c["skip"] else 0)
        return {"bytes": kept * 2 * (values * size + held) + c["tokens"] * (2 * values * size + 8), "flops": 0}
    # ragged lengths: an even spread over the range, the longest and an empty one among them
    tokens = c["batch"] * c["longest"]
    if c["ragged"] and c["batch"] > 1:
        tokens = c["longest"] * (1 + (c["batch"] - 2) / 2)
    if c["window"]:
        tokens = min(tokens, c["batch"] * (c["window"] + c["new"]))
    rows = c["new"] * c["heads"] * c["group"]
    return {"bytes": tokens * 2 * held + c["batch"] * rows * (2 * c["dim"] * size + 4), "flops": 4.0 * tokens * rows * c["dim"]}


# ------------------------------------------------------------- exact, in 64 bits --

def _grid(fmt):
    """All sixteen E2M1 values and the block scales of every byte, from the bit fields."""
    code = []
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        code.append((-1.0 if c & 8 else 1.0) * (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)))
    scale = []
    for b in range(256):
        if fmt == "mxfp4":
            scale.append(2.0 ** (b - 127) if b < 255 else math.nan)
        else:
            e, m = (b >> 3) & 15, b & 7
            v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            scale.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(code, dtype=torch.float64, device=DEV), torch.tensor(scale, dtype=torch.float64, device=DEV)


def _exact_values(packed, scales, fmt, g):
    code, scale = _grid(fmt)
    out = torch.empty(*packed.shape[:-1], packed.shape[-1] * 2, dtype=torch.float64, device=DEV)
    out[..., 0::2] = code[(packed % 16).long()]
    out[..., 1::2] = code[torch.div(packed, 16, rounding_mode="floor").long()]
    s = scale[scales.long()]
    if fmt == "nvfp4":
        s = s * g.double().reshape(*g.shape, *([1] * (s.dim() - g.dim())))
    return out * s.repeat_interleave(GROUP[fmt], -1)


def _nearest(v, values):
    """Index of the value nearest to v >= 0 in an ascending list, ties to the even index, beyond the last to it."""
    hi = torch.searchsorted(values, v).clamp(1, len(values) - 1)
    lo = hi - 1
    a, b = v - values[lo], values[hi] - v
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _exact_round(x, fmt, g):
    """Quantised and decoded again: x [T, H, D] in 64 bits."""
    code, scale = _grid(fmt)
    b = x.double().reshape(*x.shape[:2], -1, GROUP[fmt])
    top = b.abs().max(-1)[0]
    if fmt == "nvfp4":
        s = scale[:127][_nearest((top / (g.double()[:, None] * 6)).clamp(max=448.0), scale[:127])]
        d = (s * g.double()[:, None]).float().double()  # the block's divisor is rounded to 32 bits, as the quotient is
        v = (b / torch.where(s > 0, d, 1.0)[..., None]).float().double()
        unit = s * g.double()[:, None]
    else:
        unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=1e-45))) - 2).clamp(-127, 127))
        v = b / unit[..., None]
    out = code[:8][_nearest(v.abs().clamp(max=6.0), code[:8])] * torch.sign(v) * unit[..., None]
    return out.reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        return s["x"].double() @ _exact_values(s["packed"], s["scales"], s["fmt"], s["global_scale"]).T
    c = s["cache"]
    if s["op"] == "cache":
        k, v = _exact_round(s["k"], s["fmt"], c["k_global_scale"]), _exact_round(s["v"], s["fmt"], c["v_global_scale"])
        k[s["slots"] < 0], v[s["slots"] < 0] = 0, 0
        return {"k": k, "v": v}
    B, L, HQ, D = s["q"].shape
    H, ps = s["heads"], s["page"]
    out = torch.zeros(B, L, HQ, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, L, HQ), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seq_lens"].tolist()):
        pages = s["page_table"][b, : -(-n // ps)].long()
        for h in range(H if n else 0):
            one = torch.tensor(1.0)
            k, v = (_exact_values(c[t + "_packed"][pages, h], c[t + "_scales"][pages, h], s["fmt"], one.to(DEV)).reshape(-1, D)[:n]
                    * (c[t + "_global_scale"][h].double() if s["fmt"] == "nvfp4" else 1.0) for t in "kv")
            for i in range(L):
                last = n - L + i
                first = max(0, last - s["window"] + 1) if s["window"] else 0
                if last < first:
                    continue
                mine = slice(h * s["group"], (h + 1) * s["group"])
                x = s["q"][b, i, mine].double() @ k[first: last + 1].T * s["scale"]
                lse[b, i, mine] = torch.logsumexp(x, -1)
                out[b, i, mine] = torch.exp(x - lse[b, i, mine, None]) @ v[first: last + 1]
    return {"out": out, "lse": lse}
