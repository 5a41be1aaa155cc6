"""The 4-bit latent cache and dense latent attention, as cases that can be timed and checked.

Five operators: the append of latent rows to a paged 4-bit cache, reading rows of it back (as bf16,
or unpacked into rows of the FP8 cache), sparse attention over selected rows of it, and attention
over every row that a query sees of the 4-bit or the FP8 cache.  Where `own` is false `run` computes
them from elementary torch operations; where it is true it makes the library's calls.

A row of the 4-bit cache stands for scale * [code * 2^(group - 127) (512 values) | rope (64 values)]:
two e2m1 codes a byte (the even value in the low half), a group byte for 32 values, one fp32 scale.
"""
import math

import torch

own = False

LATENT, ROPE, GROUP = 512, 64, 32
TOP = 384.0  # 6 * 2^6: the largest code under the largest group factor
SCALE_MIN = 2.0 ** -60
E_MIN, E_MAX = -5, 6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # sparse attention ---------------------------------------------------------------------
        # one sequence answering: the smallest decode step, where the call's latency counts
        dict(name="sparse_decode_1x20k", op="sparse", B=1, T=1, H=64, S=20000, k=2048, page=64, shared=False, holes=False),
        # a served batch: 32 sequences, one new token each, 200,000 cached tokens
        dict(name="sparse_decode_32x200k", op="sparse", B=32, T=1, H=64, S=200000, k=2048, page=64, shared=False, holes=False),
        # a chunk of a long prompt over its paged cache
        dict(name="sparse_chunk_4k_128k", op="sparse", B=1, T=4096, H=64, S=131072, k=2048, page=64, shared=False, holes=False),
        # a quarter of the heads (heads split over devices), odd sizes, pages that end inside a tile,
        # skipped entries and rows that select nothing
        dict(name="sparse_ragged_16h", op="sparse", B=3, T=37, H=16, S=5001, k=511, page=48, shared=False, holes=True),
        # dense attention ----------------------------------------------------------------------
        # a layer without an indexer, one sequence answering over a long context
        dict(name="dense_decode_1x128k", op="dense", B=1, T=1, H=64, S=131072, page=64, four=True, ragged=False, causal=True),
        # the same for a served batch of sequences of every length, one slot of it empty
        dict(name="dense_decode_32_ragged", op="dense", B=32, T=1, H=64, S=32768, page=64, four=True, ragged=True, causal=True),
        # a chunk of a prompt over what is cached before it and itself
        dict(name="dense_chunk_1k_32k", op="dense", B=1, T=1024, H=64, S=32768, page=64, four=True, ragged=False, causal=True),
        # two chunks of odd lengths over the FP8 cache, a quarter of the heads, pages that end inside a tile
        dict(name="dense_ragged_16h_fp8", op="dense", B=2, T=301, H=16, S=4099, page=48, four=False, ragged=True, causal=True),
        # the cache ----------------------------------------------------------------------------
        # a whole prompt's latent rows appended, and handed on as FP8 rows (which is how they come back whole)
        dict(name="append_prefill_128k", op="append", B=1, n=131072, cap=131072, page=64, inter=True, norm=True),
        # one new token in each of 32 sequences
        dict(name="append_decode_32", op="append", B=32, n=1, cap=2048, page=64, inter=True, norm=True),
        # a cached prompt read back
        dict(name="read_range_128k", op="read", B=1, n=131072, cap=131072, page=64, ranged=True),
        # the selected rows of a decode step read back
        dict(name="read_topk_32x2048", op="read", B=32, n=2048, cap=16384, page=64, ranged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sparse", "sparse", "dense", "dense", "append", "read"])
    page = rng.choice([1, 16, 48, 64, 64, 100, 128, 256])
    B = _log(rng, 1, 32)
    if op == "sparse":
        H = rng.choice([1, 8, 16, 20, 32, 64, 64, 128])
        S = _log(rng, 64, 131072 if B < 9 else 16384)
        k = rng.choice([2048, _log(rng, 1, 4096)])
        T = min(_log(rng, 1, 1024), S, max(1, (1 << 22) // (B * k)), max(1, (1 << 28) // (B * k * H)))
        return dict(op=op, B=B, T=T, H=H, S=S, k=k, page=page, shared=rng.random() < 0.2, holes=rng.random() < 0.3)
    if op == "dense":
        H = rng.choice([1, 8, 16, 20, 32, 64, 64, 128])
        S = min(_log(rng, 1, 131072), (1 << 20) // B)
        T = min(_log(rng, 1, 1024), max(1, (1 << 30) // (B * S * H)))
        return dict(op=op, B=B, T=T, H=H, S=S, page=page, four=rng.random() < 0.7, ragged=rng.random() < 0.6,
                    causal=rng.random() < 0.8)
    n = min(_log(rng, 1, 131072), 131072 // B)
    cap = n + rng.randrange(1 + n)
    if op == "append":
        return dict(op=op, B=B, n=n, cap=cap, page=page, inter=rng.random() < 0.5, norm=rng.random() < 0.8)
    return dict(op=op, B=B, n=n, cap=cap, page=page, ranged=rng.random() < 0.5)


# --- inputs ----------------------------------------------------------------------------------

def _angles(cap, dev):
    """cos and sin of position x frequency, formed in 64 bits: far positions lose their angle in 32."""
    f = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
    a = torch.arange(cap, device=dev, dtype=torch.float64)[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _new_cache(B, cap, page, four, g, dev):
    """An empty paged cache; the pages of the sequences lie in shuffled order, with a few spare."""
    per = -(-cap // page)
    pages = B * per + 3
    table = torch.randperm(pages, generator=g, device=dev)[:B * per].to(torch.int32).reshape(B, per).contiguous()
    cache = dict(scales=torch.ones((pages, page), device=dev),
                 rope=torch.zeros((pages, page, ROPE), device=dev, dtype=torch.bfloat16), block_table=table)
    if four:
        cache["codes"] = torch.zeros((pages, page, LATENT // 2), device=dev, dtype=torch.uint8)
        cache["groups"] = torch.full((pages, page, LATENT // GROUP), 127, device=dev, dtype=torch.uint8)
    else:
        cache["codes"] = torch.zeros((pages, page, LATENT), device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return cache


def _fill_cache(cache, g):
    """Rows as an RMS norm leaves them, quantised; a page block at a time (a cache can be large)."""
    dev = cache["codes"].device
    pages, page = cache["scales"].shape
    gain = 1 + 0.2 * torch.randn(LATENT, generator=g, device=dev)
    four = "groups" in cache
    step = max(1, (1 << 17) // page)
    for p in range(0, pages, step):
        m = min(step, pages - p)
        y = torch.randn((m, page, LATENT), generator=g, device=dev) * gain
        s = y.abs().amax(-1) / (TOP if four else 448.0)
        if four:
            codes, groups = _four_bits(y / s[..., None])
            cache["codes"][p:p + m] = codes
            cache["groups"][p:p + m] = groups
        else:
            cache["codes"][p:p + m] = (y / s[..., None]).to(torch.float8_e4m3fn)
        cache["scales"][p:p + m] = s
        cache["rope"][p:p + m] = (torch.randn((m, page, ROPE), generator=g, device=dev) / s[..., None]).to(torch.bfloat16)


def _selection(B, T, S, k, pos0, holes, g, dev):
    """Index rows as a top-k writes them: ascending positions spread over what the row sees, -1 behind;
    neighbouring rows of a sequence share about 70% of theirs."""
    n = (pos0 + torch.arange(T, device=dev, dtype=torch.int64)).clamp(1, S)[None, :, None].expand(B, T, 1)
    j = torch.arange(k, device=dev, dtype=torch.int64)
    lo, hi = j * n // k, (j + 1) * n // k
    u = torch.where(torch.rand((B, T, k), generator=g, device=dev) < 0.7,
                    torch.rand((B, 1, k), generator=g, device=dev), torch.rand((B, T, k), generator=g, device=dev))
    idx = lo + (u * (hi - lo)).long().clamp(max=(hi - lo - 1).clamp(min=0))
    idx = torch.where(n >= k, idx, torch.where(j < n, j, -1))
    if holes:  # entries skipped anywhere, rows that keep nothing
        idx = torch.where(torch.rand((B, T, k), generator=g, device=dev) < 0.05, -1, idx)
        idx[:, 3::7] = -1
    return idx.to(torch.int32).contiguous()


def _lengths(c):
    """Rows that each sequence holds, longest first: all S, or a ramp down from S with one empty slot."""
    if not c["ragged"]:
        return [c["S"]] * c["B"]
    return [0 if c["B"] > 4 and b == c["B"] // 2 else max(1, c["S"] - b * c["S"] // c["B"]) for b in range(c["B"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    c = dict(case)
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    st = dict(case=c)
    if c["op"] in ("sparse", "dense"):
        st["cache"] = _new_cache(c["B"], c["S"], c["page"], c.get("four", True), g, dev)
        _fill_cache(st["cache"], g)
        temp = torch.exp2(3 * torch.rand(c["H"], generator=g, device=dev) - 1)  # heads flat to peaked
        q = torch.randn((c["B"], c["T"], c["H"], LATENT + ROPE), generator=g, device=dev) * temp[:, None]
        st["q"] = q.to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(LATENT + ROPE)
        if c["op"] == "sparse":
            Ti = 1 if c["shared"] else c["T"]
            st["idx"] = _selection(c["B"], Ti, c["S"], c["k"], c["S"] - Ti + 1, c["holes"], g, dev)
        else:
            lens = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
            st["lens"] = lens[torch.randperm(c["B"], generator=g, device=dev)].contiguous()
        return st
    st["cache"] = _new_cache(c["B"], c["cap"], c["page"], True, g, dev)
    if c["op"] == "append":
        x = torch.randn((c["B"], c["n"], LATENT + ROPE), generator=g, device=dev)
        st["x"] = (x * torch.exp2(2 * torch.rand((c["B"], c["n"], 1), generator=g, device=dev))).to(torch.bfloat16)
        st["weight"] = 1 + 0.2 * torch.randn(LATENT, generator=g, device=dev) if c["norm"] else None
        st["cos"], st["sin"] = _angles(c["cap"], dev)
        start = torch.randint(0, c["cap"] - c["n"] + 1, (c["B"], 1), generator=g, device=dev)
        st["positions"] = (start + torch.arange(c["n"], device=dev)).contiguous()
        st["idx"] = st["positions"].to(torch.int32)
        return st
    _fill_cache(st["cache"], g)
    if not c["ranged"]:
        st["idx"] = _selection(c["B"], 1, c["cap"], c["n"], c["cap"], False, g, dev)[:, 0].contiguous()
    return st


# --- plain forms -----------------------------------------------------------------------------

def _four_bits(z):
    """(two e2m1 codes a byte, a group byte for 32 values) of z [..., 512]: the least power of two that brings a
    group's largest magnitude to 6, then the nearest code, ties to the even one."""
    g = z.abs().unflatten(-1, (-1, GROUP)).amax(-1)
    m, e = torch.frexp(g / 6.0)  # in [0.5, 1) x 2^e
    e = torch.where(6.0 * torch.ldexp(torch.ones_like(g), e - 1) >= g, e - 1, e)
    e = torch.where(g > 0, e, E_MIN).clamp(E_MIN, E_MAX)
    q = torch.ldexp(z.unflatten(-1, (-1, GROUP)), -e[..., None]).flatten(-2)
    a = q.abs()
    code = sum((a > t).to(torch.uint8) for t in (0.25, 1.25, 2.5, 5.0)) + sum((a >= t).to(torch.uint8) for t in (0.75, 1.75, 3.5))
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8)


def _values(codes, groups):
    """What codes [..., 256] under group bytes [..., 16] stand for, 32 bits, [..., 512]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    f = torch.exp2(groups.float() - 127.0)
    return (v.unflatten(-1, (-1, GROUP)) * f[..., None]).flatten(-2)


def _cache_row(cache, b, pos):
    """Flat cache row of position pos[...] of sequence b[...]."""
    page = cache["scales"].shape[1]
    return cache["block_table"][b, pos // page].long() * page + pos % page


def _codes_of(cache, r):
    """The latent values of flat cache rows r before their scale."""
    if "groups" in cache:
        return _values(cache["codes"].reshape(-1, LATENT // 2)[r], cache["groups"].reshape(-1, LATENT // GROUP)[r])
    return cache["codes"].view(torch.uint8).reshape(-1, LATENT)[r].view(torch.float8_e4m3fn).float()


def _rows(cache, b, pos):
    """What the cache rows stand for, 32 bits, [..., 576]."""
    r = _cache_row(cache, b, pos)
    s = cache["scales"].reshape(-1)[r][..., None]
    return torch.cat((_codes_of(cache, r) * s, cache["rope"].reshape(-1, ROPE)[r].float() * s), -1)


def _rotated(x, cos, sin, inter):
    a, c = (x[..., 0::2], x[..., 1::2]) if inter else x.chunk(2, -1)
    u, v = a * cos - c * sin, c * cos + a * sin
    return torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)


def _append_plain(st, c):
    x = st["x"].float()
    y, r = x[..., :LATENT], x[..., LATENT:]
    if c["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * st["weight"]
    r = _rotated(r, st["cos"][st["positions"]], st["sin"][st["positions"]], c["inter"])
    s = (y.abs().amax(-1) / TOP).clamp(min=SCALE_MIN)
    codes, groups = _four_bits(y / s[..., None])
    cache = st["cache"]
    at = _cache_row(cache, torch.arange(c["B"], device=y.device)[:, None], st["positions"])
    cache["codes"].view(-1, LATENT // 2)[at] = codes
    cache["groups"].view(-1, LATENT // GROUP)[at] = groups
    cache["scales"].view(-1)[at] = s
    cache["rope"].view(-1, ROPE)[at] = (r / s[..., None]).to(torch.bfloat16)
    values = _values(cache["codes"].view(-1, LATENT // 2)[at], cache["groups"].view(-1, LATENT // GROUP)[at])
    return dict(codes=values.to(torch.float8_e4m3fn), scales=cache["scales"].view(-1)[at], rope=cache["rope"].view(-1, ROPE)[at])


def _read_plain(st, c):
    dev = st["cache"]["scales"].device
    b = torch.arange(c["B"], device=dev)[:, None]
    if c["ranged"]:
        return _rows(st["cache"], b, torch.arange(c["n"], device=dev).expand(c["B"], -1)).to(torch.bfloat16)
    idx = st["idx"].long()
    y = _rows(st["cache"], b, idx.clamp(min=0))
    return torch.where((idx >= 0)[..., None], y, 0.0).to(torch.bfloat16)


def _softmax_plain(s, rows):
    """(bf16 sums of rows weighted by the softmax of s, its log sum); a row of s that is -inf throughout gives zeros."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[..., :LATENT]) / torch.where(l > 0, l, 1.0)
    return out.to(torch.bfloat16), (m + torch.log(l))[..., 0]


def _sparse_plain(st, c):
    q, idx = st["q"].float(), st["idx"].long()
    b = torch.arange(c["B"], device=q.device)[:, None, None]
    rows = _rows(st["cache"], b, idx.clamp(min=0))  # [B, T or 1, k, 576]
    s = torch.matmul(q, rows.transpose(-1, -2)) * st["scale"]
    return _softmax_plain(torch.where((idx >= 0)[:, :, None], s, -math.inf), rows)


def _dense_plain(st, c):
    B, T, H, S = c["B"], c["T"], c["H"], c["S"]
    dev = st["q"].device
    pos = torch.arange(S, device=dev)
    rows = _rows(st["cache"], torch.arange(B, device=dev)[:, None], pos.expand(B, -1))  # [B, S, 576]
    s = torch.matmul(st["q"].float().reshape(B, T * H, -1), rows.transpose(-1, -2)) * st["scale"]
    sees = st["lens"].long()[:, None] - ((T - 1) - torch.arange(T, device=dev) if c["causal"] else torch.zeros(T, device=dev, dtype=torch.int64))
    s = s.view(B, T, H, S).masked_fill_(pos >= sees[:, :, None, None], -math.inf)
    out, lse = _softmax_plain(s.view(B, T * H, S), rows)
    return out.view(B, T, H, LATENT), lse.view(B, T, H)


# --- one pass --------------------------------------------------------------------------------

def run(st):
    c = st["case"]
    if not own:
        return {"sparse": _sparse_plain, "dense": _dense_plain, "append": _append_plain, "read": _read_plain}[c["op"]](st, c)
    import long_context_sparse_tcgen05_gb300 as dsa
    if c["op"] == "sparse":
        return dsa.dsa_latent4_attn(dict(q=st["q"], cache=st["cache"], scale=st["scale"], S=c["S"]), st["idx"])
    if c["op"] == "dense":
        call = dsa.dsa_latent4_attn_dense if c["four"] else dsa.dsa_latent_attn_dense
        return call(dict(q=st["q"], cache=st["cache"], scale=st["scale"], S=c["S"]), st["lens"], causal=c["causal"])
    if c["op"] == "read":
        if c["ranged"]:
            return dsa.dsa_latent4_read(st["cache"], n=c["n"])
        return dsa.dsa_latent4_read(st["cache"], idx=st["idx"])
    dsa.dsa_latent4_append(st["x"], st["cache"], weight=st["weight"], cos=st["cos"], sin=st["sin"], interleaved=c["inter"],
                           positions=st["positions"])
    rows = dsa.dsa_latent4_unpack(st["cache"], idx=st["idx"])
    return dict(codes=rows["codes"], scales=rows["scales"], rope=rows["rope"])


def work(case):
    c = case
    if c["op"] == "sparse":
        rows, Ti = c["B"] * c["T"], 1 if c["shared"] else c["T"]
        keys = min(c["k"], c["S"])
        union = c["B"] * min(c["S"], Ti * keys)  # each selected cache row once
        return {"bytes": rows * c["H"] * (2 * 576 + 2 * 512 + 4) + 4 * c["B"] * Ti * c["k"] + union * 404,
                "flops": 2 * rows * c["H"] * keys * (576 + 512)}
    if c["op"] == "dense":
        lens, T = _lengths(c), c["T"]
        pairs = sum(sum(max(0, n - T + 1 + t) for t in range(T)) if c["causal"] else n * T for n in lens)
        return {"bytes": c["B"] * T * c["H"] * (2 * 576 + 2 * 512 + 4) + 4 * c["B"] + sum(lens) * (404 if c["four"] else 644),
                "flops": 2 * c["H"] * pairs * (576 + 512)}
    tok = c["B"] * c["n"]
    if c["op"] == "append":  # the rows in, into the cache, and out of it again as FP8 rows
        return {"bytes": tok * (1152 + 8 + 404 + 404 + 4 + 644) + 4 * ROPE * min(tok, c["cap"]), "flops": tok * 576 * 10}
    return {"bytes": tok * (404 + 1152 + (0 if c["ranged"] else 4)), "flops": tok * 576}


# --- the definitions in 64 bits --------------------------------------------------------------

def _exact_latent(cache, p, o):
    """Latent values before the scale of rows o of pages p (1-d), 64 bits."""
    if "groups" not in cache:
        return cache["codes"].view(torch.uint8)[p, o].view(torch.float8_e4m3fn).double()
    packed, groups = cache["codes"][p, o].long(), cache["groups"][p, o].double()
    nibbles = torch.empty((packed.shape[0], LATENT), device=packed.device, dtype=torch.int64)
    nibbles[:, 0::2] = packed % 16
    nibbles[:, 1::2] = packed // 16
    half_steps = nibbles % 8  # exponent in the two upper bits, one bit of fraction
    ex, fr = half_steps // 2, (half_steps % 2).double()
    v = torch.where(ex == 0, fr / 2, (1 + fr / 2) * 2.0 ** (ex - 1).double())
    v = torch.where(nibbles >= 8, -v, v)
    return v * torch.repeat_interleave(2.0 ** (groups - 127), GROUP, dim=1)


def _exact_rows(cache, b, pos):
    page = cache["scales"].shape[1]
    p = cache["block_table"][b].long()[torch.div(pos, page, rounding_mode="floor")]
    o = torch.remainder(pos, page)
    return torch.cat((_exact_latent(cache, p, o), cache["rope"][p, o].double()), 1) * cache["scales"][p, o].double()[:, None]


def _exact_spin(v, angle_cos, angle_sin, inter):
    """Rotation as a product of complex numbers."""
    h = v.shape[-1] // 2
    z = torch.view_as_complex(v.unflatten(-1, (h, 2)).contiguous() if inter else torch.stack((v[..., :h], v[..., h:]), -1).contiguous())
    z = z * torch.complex(angle_cos.double(), angle_sin.double())
    return torch.stack((z.real, z.imag), -1).flatten(-2) if inter else torch.cat((z.real, z.imag), -1)


def _exact_quantised(z):
    """The e2m1 value under its group's power of two that is nearest to each value of z [n, 512], 64 bits."""
    grid = torch.tensor(E2M1, device=z.device, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(z)
    for i in range(LATENT // GROUP):
        part = z[:, i * GROUP:(i + 1) * GROUP]
        f = torch.full((z.shape[0],), 2.0 ** E_MIN, device=z.device, dtype=torch.float64)
        for e in range(E_MIN, E_MAX):
            f = torch.where(part.abs().max(1).values > 6 * 2.0 ** e, 2.0 ** (e + 1), f)
        a = (part / f[:, None]).abs()
        lower, upper = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # apart on a tie alone
        out[:, i * GROUP:(i + 1) * GROUP] = torch.sign(part) * grid[torch.where(lower % 2 == 0, lower, upper)] * f[:, None]
    return out


def _exact_attention(q, rows, limit, scale):
    """Softmax of scale * q . row over the first limit[i] rows for queries q [m, 576]: (values, log sums)."""
    s = (q @ rows.T) * scale
    s.masked_fill_(torch.arange(rows.shape[0], device=q.device) >= limit[:, None], -math.inf)
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return w @ rows[:, :LATENT], lse


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    dev = torch.device("cuda")
    if c["op"] in ("sparse", "dense"):
        B, T, H = c["B"], c["T"], c["H"]
        if c["op"] == "sparse" and B * T > 8192:  # row by row below: longer than 20 seconds
            return None
        out = torch.zeros((B, T, H, LATENT), device=dev, dtype=torch.float64)
        lse = torch.full((B, T, H), -math.inf, device=dev, dtype=torch.float64)
        for b in range(B):
            if c["op"] == "sparse":
                for t in range(T):
                    sel = st["idx"][b, 0 if c["shared"] else t]
                    sel = sel[sel >= 0].long()
                    if sel.numel():
                        rows = _exact_rows(st["cache"], b, sel)
                        logits = (st["q"][b, t].double() @ rows.T) * st["scale"]
                        out[b, t] = torch.softmax(logits, -1) @ rows[:, :LATENT]
                        lse[b, t] = torch.logsumexp(logits, -1)
                continue
            n = int(st["lens"][b])
            if n == 0:
                continue
            rows = _exact_rows(st["cache"], b, torch.arange(n, device=dev))
            step = max(1, 2048 // H)
            for t in range(0, T, step):
                m = min(step, T - t)
                limit = torch.arange(n - T + 1 + t, n - T + 1 + t + m, device=dev) if c["causal"] else torch.full((m,), n, device=dev)
                o, l = _exact_attention(st["q"][b, t:t + m].double().reshape(m * H, -1), rows, limit.repeat_interleave(H), st["scale"])
                out[b, t:t + m], lse[b, t:t + m] = o.view(m, H, LATENT), l.view(m, H)
        return out, lse
    if c["op"] == "read":
        y = torch.zeros((c["B"], c["n"], LATENT + ROPE), device=dev, dtype=torch.float64)
        for b in range(c["B"]):
            pos = torch.arange(c["n"], device=dev) if c["ranged"] else st["idx"][b].long()
            ok = pos >= 0
            y[b, ok] = _exact_rows(st["cache"], b, pos[ok])
        return y
    y, pos = st["x"].double(), st["positions"]
    lat, r = y[..., :LATENT], y[..., LATENT:]
    if c["norm"]:
        lat = lat / ((lat * lat).sum(-1, keepdim=True) / LATENT + 1e-6).sqrt() * st["weight"].double()
    r = _exact_spin(r, st["cos"][pos], st["sin"][pos], c["inter"])
    s = torch.clamp(lat.abs().max(-1).values / TOP, min=SCALE_MIN)
    codes = torch.stack([_exact_quantised(lat[b] / s[b][:, None]) for b in range(c["B"])])
    return dict(codes=codes, scales=s, rope=r / s[..., None])
