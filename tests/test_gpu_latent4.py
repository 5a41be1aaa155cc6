"""The 4-bit latent cache (append, read, unpack, sparse attention) and attention over every row that a query
sees, against plain 64-bit implementations.  A row of the 4-bit cache is exactly a row of the FP8 cache under
the same scale, so sparse attention over it has to give the bits that the FP8 cache's gives over the unpacked
rows.  Tolerances count roundings: a bf16 result is off by at most 2^-8 of its value, and fp32 work by a few
2^-24 of the largest term (2^-18 covers sums of up to 1,024 terms)."""
import math

import pytest
import torch

import long_context_sparse_tcgen05_gb300 as dsa

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn
BF16_STEP, FP32_WORK = 2.0 ** -8, 2.0 ** -18
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_tcgen05_gb300 import build
    build.build()
    dsa.load_library()
    dsa.read_device_flags(DEV)
    yield


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _angles(rows, seed=0):
    a = torch.rand((rows, 32), generator=_gen(900 + seed), device=DEV, dtype=torch.float64) * 2000 - 1000
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _cache(B, cap, page, four=True, seed=0, spread=0.0):
    """A paged cache (page 0: no table) with shuffled pages; every row, used or not, holds data: of the 4-bit one
    every code under every group byte."""
    g = _gen(seed + 31)
    if page:
        per = -(-cap // page)
        pages = B * per + 2
        table = torch.randperm(pages, generator=g, device=DEV)[:B * per].int().reshape(B, per).contiguous()
    else:
        pages, page, table = B, cap, None
    cache = dict(scales=torch.exp2(torch.randn((pages, page), generator=g, device=DEV) * spread) * 0.01,
                 rope=torch.randn((pages, page, 64), generator=g, device=DEV).mul(100).bfloat16(), block_table=table)
    if four:
        cache["codes"] = torch.randint(0, 256, (pages, page, 256), generator=g, device=DEV).to(torch.uint8)
        cache["groups"] = torch.randint(122, 134, (pages, page, 16), generator=g, device=DEV).to(torch.uint8)
    else:
        cache["codes"] = (torch.randn((pages, page, 512), generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)
    return cache


def _flat(cache, b, pos):
    page = cache["scales"].shape[1]
    if cache["block_table"] is None:
        return b * page + pos
    return cache["block_table"][b, pos // page].long() * page + pos % page


def _factor(groups):
    """The powers of two of group bytes, from a table: torch's power of 2 is not exact in 64 bits on the device."""
    return torch.tensor([2.0 ** (b - 127) for b in range(256)], device=DEV, dtype=torch.float64)[groups.int()]


def _latent64(cache, r):
    """What the codes of flat rows r stand for, before the scale."""
    if "groups" not in cache:
        return cache["codes"].view(torch.uint8).reshape(-1, 512)[r].view(E4M3).double()
    packed = cache["codes"].reshape(-1, 256)[r].int()
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV, dtype=torch.float64)
    v = grid[torch.stack((packed % 16, packed // 16), -1).flatten(-2)]
    return v * _factor(cache["groups"].reshape(-1, 16)[r]).repeat_interleave(32, -1)


def _rows64(cache, b, pos):
    r = _flat(cache, b, pos)
    return torch.cat((_latent64(cache, r), cache["rope"].reshape(-1, 64)[r].double()), -1) * cache["scales"].reshape(-1)[r].double()[..., None]


def _q(B, T, H, mul=2.0, seed=0):
    g = _gen(seed + 5)
    temp = torch.exp2(4 * torch.rand((H, 1), generator=g, device=DEV) - 2)
    return (torch.randn((B, T, H, 576), generator=g, device=DEV) * temp * mul).bfloat16()


def _idx(B, T, S, k, seed=0):
    g = _gen(seed + 77)
    n = min(k, S)
    idx = torch.full((B, T, k), -1, device=DEV, dtype=torch.int32)
    idx[..., :n] = torch.rand((B, T, S), generator=g, device=DEV).topk(n, -1).indices.sort(-1).values.int()
    return torch.where(torch.rand((B, T, k), generator=g, device=DEV) < 0.1, -1, idx).contiguous()


def _same(a, b):
    return all(torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32), y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32)) for x, y in zip(a, b))


# --- the cache ---------------------------------------------------------------------------------

def _quantised32(lat):
    """(scales, group exponents, codes 0-15) of lat [..., 512] fp32, as the append defines them."""
    top = lat.abs().amax(-1)
    s = (top / torch.full_like(top, 384)).clamp(min=2.0 ** -60)  # (by a Python number torch multiplies by its reciprocal)
    z = (lat / s[..., None]).unflatten(-1, (16, 32))
    m = z.abs().amax(-1)
    e = torch.full_like(m, -5.0)
    for k in range(-5, 6):
        e = torch.where(m > 6 * 2.0 ** k, k + 1.0, e)
    a = (z * torch.exp2(-e)[..., None]).flatten(-2)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    lower, upper = torch.bucketize(a.abs(), mid), torch.bucketize(a.abs(), mid, right=True)
    code = torch.where(lower % 2 == 0, lower, upper)  # a tie goes to the even code
    return s, e, code + 8 * torch.signbit(a)


@pytest.mark.parametrize("B,n,cap,page", [(1, 1, 1, 1), (1, 1, 40, 0), (3, 5, 40, 16), (2, 37, 100, 48), (2, 9, 30, 7),
                                          (4, 300, 300, 64), (1, 70, 90, 1), (2, 33, 64, 0)])
@pytest.mark.parametrize("inter,rope", [(True, True), (False, True), (True, False)])
def test_append_without_norm_is_the_definition_bit_for_bit(B, n, cap, page, inter, rope):
    """fp32 quotients rounded as IEEE division rounds leave nothing open: every code, group and scale."""
    g = _gen(n + cap)
    cache = _cache(B, cap, page)
    before = {k: v.clone() for k, v in cache.items() if v is not None}
    x = torch.randn((B, n, 576), generator=g, device=DEV) * torch.exp2(4 * torch.rand((B, n, 1), generator=g, device=DEV) - 2)
    x[..., :512] *= torch.exp2(-3 * torch.rand((B, n, 16), generator=g, device=DEV) ** 3 * 4).repeat_interleave(32, -1)
    x = x.bfloat16()
    cos, sin = _angles(cap) if rope else (None, None)
    pos = torch.stack([torch.randperm(cap, generator=g, device=DEV)[:n] for _ in range(B)])
    dsa.dsa_latent4_append(x, cache, cos=cos, sin=sin, interleaved=inter, positions=pos)
    assert dsa.read_device_flags(DEV) == 0
    s, e, code = _quantised32(x[..., :512].float())
    at = _flat(cache, torch.arange(B, device=DEV)[:, None], pos)
    assert torch.equal(cache["scales"].reshape(-1)[at], s)
    assert torch.equal(cache["groups"].reshape(-1, 16)[at].float() - 127, e)
    packed = cache["codes"].reshape(-1, 256)[at].int()
    assert torch.equal(torch.stack((packed % 16, packed // 16), -1).flatten(-2), code.int())
    r = x[..., 512:].double()
    if rope:
        c, d = cos[pos].double(), sin[pos].double()
        u, v = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :32], r[..., 32:])
        u, v = u * c - v * d, v * c + u * d
        r = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    ref = r / s.double()[..., None]
    off = (cache["rope"].reshape(-1, 64)[at].double() - ref).abs()
    assert bool((off <= BF16_STEP * ref.abs() + FP32_WORK * ref.abs().amax(-1, keepdim=True)).all())
    keep = torch.ones(cache["scales"].numel(), dtype=torch.bool, device=DEV)
    keep[at.reshape(-1)] = False
    for name, width in (("codes", 256), ("groups", 16), ("scales", 1), ("rope", 64)):
        assert torch.equal(cache[name].reshape(-1, width)[keep], before[name].reshape(-1, width)[keep]), f"{name}: another row changed"


@pytest.mark.parametrize("inter", [True, False])
def test_append_with_norm_matches_64_bits(inter):
    """The normed values are fp32 with an error of 2^-18 of the largest at most: a stored value is the nearest of its
    grid to a value that far from the 64-bit one, and groups differ where their largest is that near a border."""
    B, n, cap = 2, 400, 500
    g = _gen(3)
    cache = _cache(B, cap, 48)
    x = (torch.randn((B, n, 576), generator=g, device=DEV) * 3).bfloat16()
    w = 1 + 0.3 * torch.randn(512, generator=g, device=DEV)
    cos, sin = _angles(cap)
    dsa.dsa_latent4_append(x, cache, weight=w, eps=1e-5, cos=cos, sin=sin, interleaved=inter, pos0=17)
    lat = x[..., :512].double()
    lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + 1e-5) * w.double()
    at = _flat(cache, torch.arange(B, device=DEV)[:, None], torch.arange(17, 17 + n, device=DEV).expand(B, n))
    s = cache["scales"].reshape(-1)[at].double()
    ref_s = lat.abs().amax(-1) / 384
    assert bool(((s - ref_s).abs() <= FP32_WORK * ref_s).all())
    z = (lat / ref_s[..., None]).unflatten(-1, (16, 32))
    f = _factor(cache["groups"].reshape(-1, 16)[at])
    slack = 384 * 2 * FP32_WORK
    top = z.abs().amax(-1)
    assert bool((top <= 6 * f + slack).all()) and bool(((top >= 3 * f - slack) | (f == 2.0 ** -5)).all())
    v = _latent64(cache, at).unflatten(-1, (16, 32)) / f[..., None]
    a = z / f[..., None]
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    assert bool(((v - a).abs() <= step / 2 + slack / f[..., None]).all())
    assert dsa.read_device_flags(DEV) == 0


def test_append_strides_padding_and_bad_positions():
    B, n, cap = 2, 6, 50
    x = torch.randn((B, n + 1, 640), generator=_gen(2), device=DEV).bfloat16()[:, :n, 64:]
    cos, sin = _angles(cap)
    a, b = _cache(B, cap, 16), _cache(B, cap, 16)
    dsa.dsa_latent4_append(x, a, cos=cos, sin=sin, pos0=11)
    dsa.dsa_latent4_append(x.contiguous(), b, cos=cos, sin=sin, positions=(11 + torch.arange(n, device=DEV)).expand(B, n).contiguous())
    for k in ("codes", "groups", "scales", "rope"):
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))
    pos = torch.tensor([[0, -1, 49, 50, 4, 5], [-1, -1, 3, -2, 2 ** 40, 6]], device=DEV)
    c = _cache(B, cap, 16)
    c["block_table"][1, 0] = 99  # positions 0..15 of sequence 1 have no page
    old = c["scales"].clone()
    dsa.dsa_latent4_append(x, c, cos=cos, sin=sin, positions=pos)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    hit = _flat(c, torch.zeros(4, dtype=torch.long, device=DEV), torch.tensor([0, 49, 4, 5], device=DEV))
    assert sorted((c["scales"] != old).reshape(-1).nonzero().flatten().tolist()) == sorted(hit.tolist())


def test_append_zero_tiny_flat_and_non_finite_rows():
    cache = _cache(1, 8, 4)
    x = torch.zeros((1, 6, 576), device=DEV, dtype=torch.bfloat16)
    x[0, :, 512:] = 1.0
    x[0, 1, :512] = 2.0 ** -100
    x[0, 2, 7] = math.nan
    x[0, 3, 9] = -math.inf
    x[0, 4, :512] = 3.0
    x[0, 5, 0], x[0, 5, 32] = 384.0, 2.0 ** -20  # a group far below the row's largest value
    dsa.dsa_latent4_append(x, cache)
    y = dsa.dsa_latent4_read(cache, n=6)
    at = _flat(cache, torch.zeros(6, dtype=torch.long, device=DEV), torch.arange(6, device=DEV))
    s, groups = cache["scales"].reshape(-1)[at], cache["groups"].reshape(-1, 16)[at]
    assert float(s[0]) == 2.0 ** -60 and float(s[1]) == 2.0 ** -60
    assert bool((y[0, :2, :512] == 0).all()) and bool((y[0, :2, 512:] == 1).all())
    assert bool((groups[0] == 122).all()) and bool((groups[4] == 133).all())
    assert bool(s[2].isnan()) and bool(y[0, 2].isnan().all()) and bool(s[3].isnan()) and bool(y[0, 3].isnan().all())
    assert bool((y[0, 4, :512] == 3).all())
    assert float(y[0, 5, 0]) == 384.0 and float(y[0, 5, 32]) == 0.0 and int(groups[5, 1]) == 122


@pytest.mark.parametrize("B,n,cap,page", [(1, 1, 1, 1), (3, 70, 100, 16), (2, 129, 200, 48), (2, 20, 33, 0), (1, 2048, 5000, 64)])
def test_read_and_unpack_are_the_stored_values(B, n, cap, page):
    cache = _cache(B, cap, page, spread=3.0)
    idx = torch.randint(-1, cap, (B, n), generator=_gen(n), device=DEV).int()
    b = torch.arange(B, device=DEV)[:, None]
    none = (idx < 0)[..., None]
    rows = torch.where(none, 0.0, _rows64(cache, b, idx.clamp(min=0).long()))
    y = dsa.dsa_latent4_read(cache, idx)
    # code * 2^e is exact, times the scale one fp32 rounding, then bf16
    assert bool(((y.double() - rows).abs() <= BF16_STEP * rows.abs() + 2.0 ** -23 * rows.abs()).all())
    u = dsa.dsa_latent4_unpack(cache, idx)
    r = _flat(cache, b, idx.clamp(min=0).long())
    assert u["codes"].dtype == E4M3 and u["block_table"] is None
    assert torch.equal(u["codes"].double(), torch.where(none, 0.0, _latent64(cache, r)))
    assert torch.equal(u["scales"], torch.where(none[..., 0], 1.0, cache["scales"].reshape(-1)[r]))
    assert torch.equal(u["rope"].view(torch.int16), torch.where(none, 0, cache["rope"].reshape(-1, 64)[r].view(torch.int16)))
    assert torch.equal(dsa.dsa_latent_read(u, n=n), y)  # the FP8 cache's own read
    lo = min(3, cap - 1)
    m = min(n, cap - lo)
    p = torch.arange(lo, lo + m, device=DEV).int().expand(B, m).contiguous()
    assert torch.equal(dsa.dsa_latent4_read(cache, n=m, pos0=lo), dsa.dsa_latent4_read(cache, p))
    assert torch.equal(dsa.dsa_latent4_unpack(cache, n=m, pos0=lo)["codes"].view(torch.uint8), dsa.dsa_latent4_unpack(cache, p)["codes"].view(torch.uint8))
    assert dsa.read_device_flags(DEV) == 0


def test_read_and_unpack_bad_positions_and_pages():
    cache = _cache(2, 40, 16)
    cache["block_table"][1, 1] = -5
    idx = torch.tensor([[0, 48, -2, 39], [15, 16, 31, -1]], device=DEV).int()
    y = dsa.dsa_latent4_read(cache, idx)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    u = dsa.dsa_latent4_unpack(cache, idx)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    for b, i in ((0, 1), (0, 2), (1, 1), (1, 2), (1, 3)):
        assert not bool(y[b, i].any()) and float(u["scales"][b, i]) == 1.0 and not bool(u["codes"][b, i].view(torch.uint8).any())
    assert bool(y[0, 0].any()) and bool(y[0, 3].any()) and bool(y[1, 0].any())
    assert dsa.dsa_latent4_read(cache, n=0).shape == (2, 0, 576) and dsa.dsa_latent4_unpack(cache, n=0)["codes"].shape == (2, 0, 512)


# --- sparse attention over the 4-bit cache -------------------------------------------------------

@pytest.mark.parametrize("B,T,H,S,k,page", [
    (1, 1, 64, 5000, 2048, 64), (1, 1, 1, 1, 1, 1), (2, 3, 8, 40, 31, 16), (1, 4, 16, 100, 32, 48), (2, 5, 20, 100, 33, 7),
    (1, 3, 63, 200, 63, 64), (1, 3, 64, 200, 64, 64), (3, 2, 65, 200, 65, 64), (1, 2, 128, 700, 511, 100),
    (4, 1, 64, 3000, 2048, 64), (2, 90, 64, 400, 129, 64), (2, 200, 16, 400, 300, 0), (1, 7, 32, 30, 100, 16),
    (1, 1, 64, 9000, 8999, 64), (1, 600, 64, 3000, 1500, 64),
])
def test_sparse_attention_gives_the_bits_of_the_unpacked_rows(B, T, H, S, k, page):
    cache = _cache(B, S, page, seed=k, spread=1.0)
    idx = _idx(B, T, S, k, seed=H)
    idx[:, T // 2, : k // 2] = -1  # (a row whose first blocks are empty)
    if T > 4:
        idx[:, 3] = -1
    at = dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=S)
    got = dsa.dsa_latent4_attn(at, idx)
    want = dsa.dsa_latent_attn(dict(at, cache=dsa.dsa_latent4_unpack(cache, n=S)), idx)
    assert _same(got, want) and dsa.read_device_flags(DEV) == 0
    if T > 4:
        assert not bool(got[0][:, 3].any()) and bool((got[1][:, 3] == -math.inf).all())


def test_sparse_attention_bad_indices_pages_and_what_is_not_selected():
    cache = _cache(1, 100, 16)
    at = dict(q=_q(1, 170, 64), cache=cache, scale=0.05, S=90)
    good = _idx(1, 170, 90, 64)
    bad = good.clone()
    bad[0, 0, 5], bad[0, 0, 6], bad[0, 1, 63] = 90, -2, 2 ** 31 - 1
    masked = good.clone()
    masked[0, 0, 5], masked[0, 0, 6], masked[0, 1, 63] = -1, -1, -1
    got = dsa.dsa_latent4_attn(at, bad)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    want = dsa.dsa_latent4_attn(at, masked)
    assert _same(got, want) and dsa.read_device_flags(DEV) == 0
    table = cache["block_table"].clone()
    table[0, 2] = cache["scales"].shape[0]  # positions 32..47
    got = dsa.dsa_latent4_attn(dict(at, cache=dict(cache, block_table=table)), good)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    few = torch.where((good >= 32) & (good < 48), -1, good)
    assert _same(got, dsa.dsa_latent4_attn(at, few))
    few = torch.where(few >= 48, -1, few).contiguous()  # rows from 32 on: infinite and NaN, selected by nothing
    dirty = {k: v.clone() for k, v in cache.items()}
    used = torch.zeros(cache["scales"].numel(), dtype=torch.bool, device=DEV)
    used[_flat(cache, torch.zeros(32, dtype=torch.long, device=DEV), torch.arange(32, device=DEV))] = True
    dirty["codes"].view(-1, 256)[~used] = 0xFF
    dirty["groups"].view(-1, 16)[~used] = 0xFF
    dirty["scales"].view(-1)[~used] = math.nan
    dirty["rope"].view(-1, 64)[~used] = -math.inf
    assert _same(dsa.dsa_latent4_attn(dict(at, cache=dirty), few), dsa.dsa_latent4_attn(at, few))


def test_sparse_attention_nan_rows_strided_queries_and_shared_index_rows():
    B, T, H = 2, 4, 24
    cache = _cache(B, 400, 64)
    wide = torch.randn((B, T + 1, H + 2, 576), generator=_gen(4), device=DEV).bfloat16()
    q = wide[:, 1:, 1:H + 1]
    idx = _idx(B, 1, 400, 200)
    want = dsa.dsa_latent4_attn(dict(q=q.contiguous(), cache=cache, scale=0.05), idx.expand(B, T, 200).contiguous())
    assert _same(dsa.dsa_latent4_attn(dict(q=q, cache=cache, scale=0.05), idx), want)
    o, l = dsa.dsa_latent4_attn(dict(q=q, cache=cache, scale=0.05), idx, lse=False)
    assert l is None and _same([o], want[:1])
    hit = int(idx[1, 0][idx[1, 0] >= 0][7])
    cache["scales"].view(-1)[_flat(cache, torch.ones(1, dtype=torch.long, device=DEV), torch.tensor([hit], device=DEV))] = math.nan
    o, l = dsa.dsa_latent4_attn(dict(q=q, cache=cache, scale=0.05), idx)
    assert _same([o[0], l[0]], [want[0][0], want[1][0]]) and bool(o[1].isnan().all())


@pytest.mark.parametrize("B,T,H,k", [(1, 200, 1, 70), (2, 400, 5, 33), (1, 300, 16, 2048), (3, 130, 40, 64), (2, 100, 64, 100), (1, 90, 128, 65),
                                     (1, 153, 63, 1), (1, 77, 65, 300), (1, 5000, 3, 20)])
def test_sparse_attention_of_many_tokens_of_one_index_row(B, T, H, k):
    """Tokens of one index row share tiles where their queries lie side by side; the bits are those of an index row each."""
    S = 2100
    cache, q, idx = _cache(B, S, 64, seed=k), _q(B, T, H), _idx(B, 1, S, k, seed=H)
    q[0, T // 2] *= 40.0  # (a token whose maximum moves where its neighbours' do not)
    q[0, T // 3, 0, 3] = math.nan
    each = idx.expand(B, T, k).contiguous()
    apart = torch.empty((B, T, H + 1, 576), device=DEV, dtype=torch.bfloat16)[:, :, :H]
    apart.copy_(q)
    for call, c in ((dsa.dsa_latent4_attn, cache), (dsa.dsa_latent_attn, dsa.dsa_latent4_unpack(cache, n=S))):
        at = dict(q=q, cache=c, scale=0.05, S=S)
        want = call(at, each)
        assert _same(call(at, idx), want) and _same(call(dict(at, q=apart), idx), want)
        assert bool(want[0][0, T // 3, 0].isnan().all()) and not bool(want[0][0, 0].isnan().any())
        assert not bool(call(at, torch.full_like(idx, -1))[0].any()) and dsa.read_device_flags(DEV) == 0


# --- attention over every row --------------------------------------------------------------------

def _call(cache):
    return dsa.dsa_latent4_attn_dense if "groups" in cache else dsa.dsa_latent_attn_dense


def _check_dense(at, lens, causal=True, some=None, **kw):
    """Against 64 bits (of `some` (b, t) alone).  A weight is held to 2^-8 of itself and to 2^-14 of the row's largest
    scaled weight; a result is then rounded to bf16."""
    q, cache = at["q"], at["cache"]
    B, T, H, _ = q.shape
    o, l = _call(cache)(at, torch.tensor(lens, dtype=torch.int32, device=DEV), causal=causal, **kw)
    for b in range(B):
        n = lens[b]
        if n:
            pos = torch.arange(n, device=DEV)
            rows, r = _rows64(cache, torch.full_like(pos, b), pos), _flat(cache, torch.full_like(pos, b), pos)
            s = cache["scales"].reshape(-1)[r].double()
        for t in range(T):
            if some is not None and (b, t) not in some:
                continue
            sees = n - (T - 1 - t) if causal else n
            if sees <= 0:
                assert not bool(o[b, t].any()) and bool((l[b, t] == -math.inf).all()), (b, t)
                continue
            v = rows[:sees, :512]
            sc = (q[b, t].double() @ rows[:sees].T) * at["scale"]
            p = torch.softmax(sc, -1)
            ref, lse = p @ v, torch.logsumexp(sc, -1)
            unit = (v / s[:sees, None]).abs().sum(0)
            tol = BF16_STEP * (ref.abs() + p @ v.abs()) + 2.0 ** -14 * (p * s[:sees]).amax(-1, keepdim=True) * unit
            bad = (o[b, t].double() - ref).abs() > tol
            assert not bool(bad.any()), f"({b}, {t}): {int(bad.sum())} of {bad.numel()} values off"
            # (scores are fp32 sums of 576 products: 2^-14 as for the sparse calls)
            assert bool(((l[b, t].double() - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all()), (b, t)
    return o, l


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("B,T,H,S,page,lens", [
    (1, 1, 64, 1, 1, [1]),                        # one token of one row
    (1, 1, 1, 70, 16, [70]),
    (3, 1, 64, 700, 64, [700, 0, 65]),            # a batch with an empty slot
    (2, 5, 20, 300, 48, [300, 3]),                # more tokens than a sequence holds: three a tile
    (1, 130, 1, 200, 64, [200]),                  # one head: 64 tokens a tile
    (2, 33, 16, 150, 7, [150, 33]),
    (1, 9, 128, 500, 100, [500]),                 # two groups of heads
    (2, 3, 65, 400, 64, [400, 399]),
    (1, 3, 33, 128, 64, [127]),                   # a token a tile, half empty
    (2, 40, 64, 130, 0, [130, 40]),               # no block table
    (5, 1, 64, 9000, 64, [9000, 1, 4097, 0, 64]),
    (1, 2, 64, 40000, 64, [39999]),               # parts of a row on every SM
    (40, 1, 8, 640, 64, [16 * i for i in range(40)]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_dense_attention_matches_64_bits(B, T, H, S, page, lens, four, causal):
    cache = _cache(B, S, page, four, seed=S, spread=0.5)
    _check_dense(dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=S), lens, causal)
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("T,H,S,n", [(3000, 8, 3000, 3000), (700, 64, 2000, 1999), (333, 128, 1200, 1100), (4096, 1, 4096, 4090)])
def test_dense_attention_of_long_chunks(T, H, S, n, four):
    """Many tiles a CTA, parts at both ends of its run: sampled tokens against 64 bits, the whole against a second run."""
    cache = _cache(1, S, 64, four)
    at = dict(q=_q(1, T, H), cache=cache, scale=1 / 24)
    some = {(0, t) for t in list(range(0, T, 97)) + [1, 2, T - 2, T - 1]}
    got = _check_dense(at, [n], some=some)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    assert _same(got, _call(cache)(at, lens)) and dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("n", [63, 64, 65, 255, 256, 257, 511, 513, 4096, 9727, 9728, 9729, 20000])
def test_dense_attention_around_the_lengths_that_are_divided(n):
    cache = _cache(1, 20000, 64)
    at = dict(q=_q(1, 1, 64, seed=n), cache=cache, scale=1 / 24, S=20000)
    _check_dense(at, [n])


def test_dense_attention_flat_peaked_rising_and_infinite_scores():
    S = 3000
    cache = _cache(1, S, 64, four=False)
    for mul in (1e-3, 8.0, 40.0):
        _check_dense(dict(q=_q(1, 2, 64, mul), cache=cache, scale=1 / 24), [S])
    cache["scales"].fill_(0.01)
    cache["rope"].zero_()
    flat, pos = cache["rope"].view(-1, 64), torch.arange(S, device=DEV)
    at = _flat(cache, torch.zeros_like(pos), pos)
    q = _q(1, 20, 16, 1.0)
    q[..., 512] = 8.0
    for sign in (1, -1):  # every block's scores above (below) the last one's: references move in each part
        flat[at, 0] = ((pos // 32) * 16.0 * sign / 0.01).bfloat16()
        _check_dense(dict(q=q, cache=cache, scale=1 / 24), [S])
    flat[at, 0] = -math.inf  # every score is minus infinity: empty
    o, l = dsa.dsa_latent_attn_dense(dict(q=q, cache=cache, scale=1 / 24), torch.tensor([S], dtype=torch.int32, device=DEV))
    assert not bool(o.any()) and bool((l == -math.inf).all())


def test_dense_attention_bad_lengths_and_pages_and_rows_behind_the_end():
    B, T, S = 3, 4, 300
    cache = _cache(B, S, 48)
    at = dict(q=_q(B, T, 64), cache=cache, scale=0.05, S=290)
    lens = torch.tensor([290, 100, 0], dtype=torch.int32, device=DEV)
    want = dsa.dsa_latent4_attn_dense(at, lens)
    assert dsa.read_device_flags(DEV) == 0
    got = dsa.dsa_latent4_attn_dense(at, torch.tensor([2 ** 31 - 1, 100, -7], dtype=torch.int32, device=DEV))
    assert _same(got, want) and dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    used = torch.zeros(cache["scales"].numel(), dtype=torch.bool, device=DEV)
    for b, n in ((0, 290), (1, 100)):
        used[_flat(cache, torch.full((n,), b, device=DEV), torch.arange(n, device=DEV))] = True
    dirty = {k: v.clone() for k, v in cache.items()}
    dirty["codes"].view(-1, 256)[~used] = 0xFF
    dirty["scales"].view(-1)[~used] = math.nan
    dirty["rope"].view(-1, 64)[~used] = math.inf
    dirty["block_table"][1, 3:] = 10 ** 6  # pages behind sequence 1's rows are not looked at
    dirty["block_table"][2] = -1
    assert _same(dsa.dsa_latent4_attn_dense(dict(at, cache=dirty), lens), want) and dsa.read_device_flags(DEV) == 0
    dirty["block_table"][0, 2] = -3  # positions 96..143
    o, l = dsa.dsa_latent4_attn_dense(dict(at, cache=dirty), lens)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    idx = torch.arange(290, device=DEV).int().expand(1, 1, 290).contiguous()
    idx = torch.where((idx >= 96) & (idx < 144), -1, idx).contiguous()
    one = {k: v for k, v in cache.items()}
    one["block_table"] = cache["block_table"][:1].contiguous()
    o2, l2 = dsa.dsa_latent4_attn(dict(q=at["q"][:1, 3:], cache=one, scale=0.05), idx)
    top = o2.double().abs().amax()
    assert bool(((o[:1, 3:].double() - o2.double()).abs() <= 4 * BF16_STEP * top).all()) and bool(((l[:1, 3:] - l2).abs() <= 1e-4).all())
    assert _same([o[1:], l[1:]], [want[0][1:], want[1][1:]])


def test_dense_attention_nan_reaches_only_its_head():
    cache = _cache(2, 500, 64)
    q = _q(2, 7, 16)
    lens = torch.tensor([500, 90], dtype=torch.int32, device=DEV)
    want = dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=0.05), lens)
    q2 = q.clone()
    q2[0, 3, 5, 100] = math.nan
    o, l = dsa.dsa_latent4_attn_dense(dict(q=q2, cache=cache, scale=0.05), lens)
    assert bool(o[0, 3, 5].isnan().all()) and bool(l[0, 3, 5].isnan())
    o[0, 3, 5], l[0, 3, 5] = want[0][0, 3, 5], want[1][0, 3, 5]
    assert _same([o, l], want)


def test_dense_attention_strides_outputs_and_workspace():
    B, T, H = 2, 6, 24
    cache = _cache(B, 400, 64)
    wide = torch.randn((B, T + 1, H + 2, 576), generator=_gen(4), device=DEV).bfloat16()
    q = wide[:, 1:, 1:H + 1]
    lens = torch.tensor([400, 77], dtype=torch.int32, device=DEV)
    want = dsa.dsa_latent4_attn_dense(dict(q=q.contiguous(), cache=cache, scale=0.05), lens)
    assert _same(dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=0.05), lens), want)
    out = torch.full((B, T, H, 512), 7.0, device=DEV, dtype=torch.bfloat16)
    ws = torch.zeros(dsa.latent_dense_workspace_size(B, T, 448, H), dtype=torch.uint8, device=DEV)
    o, l = dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=0.05), lens, out=out, lse=False, ws=ws)
    assert l is None and o.data_ptr() == out.data_ptr() and _same([o], want[:1])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=0.05), lens, ws=ws[:-16])


def test_dense_attention_on_two_streams_and_in_two_graphs():
    """Each call has scratch of its own: calls in flight together, and replayed graphs whose lengths and queries
    change in place, give what single calls give."""
    calls = []
    for s in (1, 2):
        cache = _cache(4, 9000, 64, seed=s)
        calls.append((dict(q=_q(4, 1, 64, seed=s), cache=cache, scale=1 / 24), torch.tensor([9000, 100 * s, 0, 5000], dtype=torch.int32, device=DEV)))
    want = [dsa.dsa_latent4_attn_dense(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(dsa.dsa_latent4_attn_dense(*calls[i]))
    torch.cuda.synchronize()
    assert all(_same(g, want[i]) for i in (0, 1) for g in got[i])
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dsa.dsa_latent4_attn_dense(*c))
        graphs.append(g)
    for i, c in enumerate(calls):
        c[0]["q"].copy_(_q(4, 1, 64, seed=30 + i))
        c[1].copy_(torch.tensor([64, 9000, 4321, 1 + i]))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, o in zip(calls, outs):
        assert _same(o, dsa.dsa_latent4_attn_dense(*c))


@pytest.mark.parametrize("B,T,H,S", [(1, 400, 64, 2000), (2, 1, 128, 9000), (1, 900, 16, 3000)])
def test_waits_that_run_out(B, T, H, S):
    """A limit of one cycle: every wait that is not complete at the first look gives up, the kernel ends what it has in
    flight and raises the flag; the same call with the default limit is right."""
    cache = _cache(B, S, 64)
    at = dict(q=_q(B, T, H), cache=cache, scale=1 / 24)
    lens, idx = torch.full((B,), S, dtype=torch.int32, device=DEV), _idx(B, T, S, 512)
    for call, arg in ((dsa.dsa_latent4_attn_dense, lens), (dsa.dsa_latent4_attn, idx)):
        want = call(at, arg)
        assert dsa.read_device_flags(DEV) == 0
        raised = False
        for _ in range(3):
            try:
                dsa.set_wait_limit(1)
                call(at, arg)
                torch.cuda.synchronize()
            finally:
                dsa.set_wait_limit(0)
            flags = dsa.read_device_flags(DEV)  # read, and cleared, after every call
            raised = raised or bool(flags & dsa.FLAG_TIMEOUT)
        assert raised
        assert _same(call(at, arg), want) and dsa.read_device_flags(DEV) == 0


# --- the operators together ----------------------------------------------------------------------

def test_serving_chain_over_the_4_bit_cache():
    """A prompt's latent rows appended to a 4-bit cache in two chunks with norm and rotation, each chunk attended
    densely; then single new tokens, each attended densely (a layer without an indexer) and over an index row; a
    finished sequence's rows handed on to the FP8 cache."""
    B, S, H, new = 2, 300, 64, 3
    cap = S + new
    g = _gen(42)
    cos, sin = _angles(cap)
    x = torch.randn((B, cap, 576), generator=g, device=DEV).bfloat16()
    w = 1 + 0.2 * torch.randn(512, generator=g, device=DEV)
    cache = _cache(B, cap, 48)

    def append(lo, hi):
        dsa.dsa_latent4_append(x[:, lo:hi], cache, weight=w, cos=cos, sin=sin, interleaved=True, pos0=lo)

    def queries(lo, hi):
        q = torch.randn((B, hi - lo, H, 576), generator=g, device=DEV).bfloat16()
        dsa.dsa_norm_rope(q[..., 512:], cos=cos, sin=sin, interleaved=True, pos0=lo, out=q[..., 512:])
        return q

    for lo, hi in ((0, 170), (170, S)):
        append(lo, hi)
        _check_dense(dict(q=queries(lo, hi), cache=cache, scale=1 / 24), [hi] * B, some={(0, 0), (0, 77), (1, hi - lo - 1)})
    for t in range(S, S + new):
        append(t, t + 1)
        q = queries(t, t + 1)
        o, l = _check_dense(dict(q=q, cache=cache, scale=1 / 24), [t + 1] * B)
        # every position as an index row: the same sums in another division
        idx = torch.arange(t + 1, device=DEV).int().expand(B, 1, t + 1).contiguous()
        o2, l2 = dsa.dsa_latent4_attn(dict(q=q, cache=cache, scale=1 / 24), idx)
        assert bool(((o.double() - o2.double()).abs() <= 4 * BF16_STEP * o2.double().abs().amax()).all()) and bool(((l - l2).abs() <= 1e-4).all())
    fp8 = dsa.dsa_latent4_unpack(cache, n=cap)
    assert _same(dsa.dsa_latent_attn(dict(q=q, cache=fp8, scale=1 / 24), idx), (o2, l2))
    lat = x[..., :512].double()
    lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + 1e-6) * w.double()
    y = dsa.dsa_latent4_read(cache, n=cap)[..., :512].double()
    # a value is off by half a step, the largest step being a third of the group's largest value (6 after 4), of which
    # the group factor may be twice what it needs, and by bf16's rounding
    top = lat.unflatten(-1, (16, 32)).abs().amax(-1).repeat_interleave(32, -1)
    low = lat.abs().amax(-1, keepdim=True) * 2.0 ** -6 / 384 * 0.5
    assert bool(((y - lat).abs() <= top / 3 + BF16_STEP * lat.abs() + low).all())
    assert dsa.read_device_flags(DEV) == 0


def test_cache_past_32_bit_offsets():
    """Rows whose codes, and rope values, lie past 4 GiB: written, read, unpacked and attended."""
    rows = (1 << 24) + 40000
    if torch.cuda.mem_get_info(DEV)[0] < rows * 420:
        pytest.skip("not enough memory")
    cache = dict(codes=torch.zeros((1, rows, 256), dtype=torch.uint8, device=DEV), groups=torch.full((1, rows, 16), 127, dtype=torch.uint8, device=DEV),
                 scales=torch.ones((1, rows), device=DEV), rope=torch.zeros((1, rows, 64), dtype=torch.bfloat16, device=DEV), block_table=None)
    n = 300
    x = torch.randn((1, n, 576), generator=_gen(1), device=DEV).bfloat16()
    small = _cache(1, n, 0)
    dsa.dsa_latent4_append(x, cache, pos0=rows - n)
    dsa.dsa_latent4_append(x, small, pos0=0)
    far = torch.arange(rows - n, rows, device=DEV).int().reshape(1, n)
    near = torch.arange(n, device=DEV).int().reshape(1, n)
    assert torch.equal(dsa.dsa_latent4_read(cache, far), dsa.dsa_latent4_read(small, near))
    u, v = dsa.dsa_latent4_unpack(cache, far), dsa.dsa_latent4_unpack(small, near)
    assert torch.equal(u["codes"].view(torch.uint8), v["codes"].view(torch.uint8)) and torch.equal(u["scales"], v["scales"])
    q = _q(1, 1, 64)
    got = dsa.dsa_latent4_attn(dict(q=q, cache=cache, scale=1 / 24), far[None].contiguous())
    assert _same(got, dsa.dsa_latent4_attn(dict(q=q, cache=small, scale=1 / 24), near[None].contiguous()))
    # all rows: the zeros before them weigh in, too
    lens = torch.tensor([rows], dtype=torch.int32, device=DEV)
    o, l = dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=1 / 24), lens)
    rows64 = _rows64(small, torch.zeros(n, dtype=torch.long, device=DEV), near[0].long())
    v, s = rows64[:, :512], small["scales"].reshape(-1).double()
    sc = (q[0, 0].double() @ rows64.T) / 24
    lse = torch.logsumexp(torch.cat((sc, torch.full((64, 1), math.log(rows - n), device=DEV, dtype=torch.float64)), 1), 1)
    assert bool(((l[0, 0].double() - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all())
    p = torch.exp(sc - lse[:, None])
    ref = p @ v
    # as in _check_dense: the largest scaled weight is that of a row of zeros (scale 1), or one of the others'
    top = torch.maximum(torch.exp(-lse), (p * s).amax(-1))[:, None]
    tol = BF16_STEP * (ref.abs() + p @ v.abs()) + 2.0 ** -14 * top * (v / s[:, None]).abs().sum(0)
    assert bool(((o[0, 0].double() - ref).abs() <= tol).all())
    del cache
    torch.cuda.empty_cache()
    assert dsa.read_device_flags(DEV) == 0


def test_trace_names_the_kernels():
    cache = _cache(1, 700, 16)
    x = torch.randn((1, 4, 576), generator=_gen(1), device=DEV).bfloat16()
    at = dict(q=_q(1, 1, 8), cache=cache, scale=0.05)
    dsa.trace_enable(64)
    try:
        dsa.dsa_latent4_append(x, cache)
        dsa.dsa_latent4_read(cache, n=4)
        dsa.dsa_latent4_unpack(cache, n=4)
        dsa.dsa_latent4_attn(at, _idx(1, 1, 700, 64))
        before = dsa.launch_count()
        dsa.dsa_latent4_attn_dense(at, torch.tensor([700], dtype=torch.int32, device=DEV))
        assert dsa.launch_count() == before + 2  # (attention, and the join of its parts)
        kinds = [r[0] for r in dsa.trace_read()]
    finally:
        dsa.trace_disable()
    assert kinds == ["cache"] * 3 + ["attention"] * 2


def test_captured_decode_steps_advance_in_place():
    """A decode step in a graph, of an append and dense attention: positions and lengths advance between replays."""
    B, cap = 3, 500
    cos, sin = _angles(cap)
    x = torch.randn((B, 1, 576), generator=_gen(1), device=DEV).bfloat16()
    q = _q(B, 1, 64)
    pos = torch.full((B, 1), 200, device=DEV, dtype=torch.int64)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    a, b = _cache(B, cap, 16), _cache(B, cap, 16)

    def work(c):
        lens.copy_(pos[:, 0] + 1)
        dsa.dsa_latent4_append(x, c, cos=cos, sin=sin, positions=pos)
        return dsa.dsa_latent4_attn_dense(dict(q=q, cache=c, scale=0.05), lens) + (dsa.dsa_latent4_read(c, pos.int()),)

    work(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = work(a)
    for t in range(5):
        pos.fill_(200 + 60 * t)
        x.normal_(generator=_gen(t))
        g.replay()
        assert _same(y, work(b))
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("B,T,H", [(152, 1, 64), (153, 1, 64), (76, 1, 128), (77, 1, 100), (30, 20, 16), (200, 3, 20)])
def test_dense_attention_of_about_as_many_tiles_as_sms(B, T, H):
    """Cut into equal parts, or divided into equal runs: short and long sequences, empty ones among them."""
    S = 900
    cache = _cache(B, S, 64, seed=B)
    g = torch.Generator()
    g.manual_seed(B)
    for top in (40, 900):
        lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
        _check_dense(dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=S), lens, some={(b, t) for b in range(0, B, 7) for t in (0, T - 1)})
    assert dsa.read_device_flags(DEV) == 0


def test_operands_of_other_kinds_are_refused():
    four, eight = _cache(2, 64, 16), _cache(2, 64, 16, four=False)
    q, lens = _q(2, 1, 64), torch.tensor([5, 6], dtype=torch.int32, device=DEV)
    idx = _idx(2, 1, 64, 32)
    x = torch.zeros((2, 1, 576), device=DEV, dtype=torch.bfloat16)
    at4, at8 = dict(q=q, cache=four, scale=0.05), dict(q=q, cache=eight, scale=0.05)
    for call in (lambda: dsa.dsa_latent_attn(at4, idx), lambda: dsa.dsa_latent_append(x, four), lambda: dsa.dsa_latent_read(four, n=3),
                 lambda: dsa.dsa_latent_attn_dense(at4, lens), lambda: dsa.dsa_latent4_attn_dense(at4, lens.long()),
                 lambda: dsa.dsa_latent4_attn_dense(at4, lens[:1]), lambda: dsa.dsa_latent4_attn_dense(at4, lens.cpu()),
                 lambda: dsa.dsa_latent4_attn_dense(at4, None), lambda: dsa.dsa_latent4_attn_dense(dict(at4, S=0), lens),
                 lambda: dsa.dsa_latent4_attn(at4, idx.long()), lambda: dsa.dsa_latent4_attn(dict(at4, q=q.expand(2, 3, 64, 576)), idx),
                 lambda: dsa.dsa_latent4_attn(dict(at4, cache=dict(four, groups=four["groups"][:1])), idx),
                 lambda: dsa.dsa_latent4_attn(dict(at4, cache=dict(four, rope=four["rope"].float())), idx),
                 lambda: dsa.dsa_latent4_append(x.float(), four), lambda: dsa.dsa_latent4_read(four), lambda: dsa.dsa_latent4_unpack(four, idx, n=3)):
        with pytest.raises(AssertionError):
            call()
    for call in (lambda: dsa.dsa_latent4_attn(at8, idx), lambda: dsa.dsa_latent4_append(x, eight), lambda: dsa.dsa_latent4_read(eight, n=3)):
        with pytest.raises(KeyError):  # (no groups)
            call()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_latent4_attn_dense(dict(at4, S=65), lens)
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("B,T,H,top", [(1, 1500, 64, 1500), (3, 400, 64, 500), (2, 2000, 12, 2000), (400, 1, 64, 700), (1, 900, 128, 3000)])
def test_dense_attention_of_prompts_from_their_start(B, T, H, top):
    """Tiles of one block and of many in one call, more tiles than SMs: runs that end in any of them."""
    cache = _cache(B, top, 64, seed=T)
    g = torch.Generator()
    g.manual_seed(T)
    lens = [top] + torch.randint(0, top + 1, (B - 1,), generator=g).tolist()
    some = {(b, t) for b in range(0, B, max(1, B // 4)) for t in {0, 1, 63, 64, 65, T // 2, T - 2, T - 1} if 0 <= t < T}
    got = _check_dense(dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=top), lens, some=some)
    # every token of a sequence that holds as many rows as there are tokens sees itself: no empty row there
    assert bool(torch.isfinite(got[1][0]).all()) and dsa.read_device_flags(DEV) == 0


def test_dense_attention_sums_of_millions_of_rows_of_the_least_scale_stay_finite():
    """2^22 rows of zeros (their scale is the append's least, 2^-60) behind a block whose weights are 2^39 below theirs, in
    one CTA each: a row sum of weights over scales is 2^(22 + 68) under a reference that may not stay 2^39 below."""
    n, T = 1 << 22, 160
    cache = dict(codes=torch.zeros((1, n, 256), dtype=torch.uint8, device=DEV), groups=torch.full((1, n, 16), 122, dtype=torch.uint8, device=DEV),
                 scales=torch.full((1, n), 2.0 ** -60, device=DEV), rope=torch.zeros((1, n, 64), dtype=torch.bfloat16, device=DEV), block_table=None)
    cache["scales"][0, :64] = 1.0
    cache["rope"][0, :64, 0] = -1.0
    q = torch.zeros((1, T, 64, 576), dtype=torch.bfloat16, device=DEV)
    q[..., 512] = 99 * math.log(2)  # y = -99 in base 2, the zeros' -60
    o, l = dsa.dsa_latent4_attn_dense(dict(q=q, cache=cache, scale=1.0), torch.tensor([n], dtype=torch.int32, device=DEV), causal=False)
    assert not bool(o.any()) and dsa.read_device_flags(DEV) == 0
    want = math.log(n - 64)  # (the first block adds e^-68)
    # (the sums over blocks keep what they lose: as in _check_dense)
    assert bool(((l.double() - want).abs() <= 2.0 ** -14 * (1 + want)).all())
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("B,T,H,S", [(1, 70, 1, 300), (2, 40, 16, 300), (1, 33, 21, 129), (2, 7, 32, 5000), (1, 9, 33, 200), (1, 600, 16, 600), (1, 5, 64, 300)])
@pytest.mark.parametrize("back", [1, 4, 66])
def test_dense_attention_what_is_not_finite_reaches_only_the_tokens_that_see_it(B, T, H, S, back, four):
    """A row that is not finite, `back` positions before a sequence's end: tokens before it keep their bits, whether
    their heads share a tile with tokens that see it or not."""
    at_row = S - back
    cache = _cache(B, S, 48, four, seed=S)
    at = dict(q=_q(B, T, H), cache=cache, scale=0.05, S=S)
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    want = _call(cache)(at, lens)
    first = max(0, T - back)  # the first token of sequence 0 that sees the row
    assert dsa.read_device_flags(DEV) == 0 and bool(torch.isfinite(want[0]).all())
    r = int(_flat(cache, torch.zeros(1, dtype=torch.long, device=DEV), torch.tensor([at_row], device=DEV)))
    append = dsa.dsa_latent4_append if four else dsa.dsa_latent_append
    for kind in ("nan", "inf", "scale", "rope nan", "rope inf") + (() if four else ("code", "code inside")):
        c = {k: v.clone() for k, v in cache.items()}
        if kind in ("nan", "inf"):
            x = torch.randn((B, 1, 576), generator=_gen(back), device=DEV).bfloat16()
            x[0, 0, 300] = math.nan if kind == "nan" else -math.inf
            append(x, c, positions=torch.tensor([[at_row]] + [[-1]] * (B - 1), device=DEV))
            assert not math.isfinite(float(c["scales"].view(-1)[r]))
        elif kind == "scale":
            c["scales"].view(-1)[r] = math.nan
        elif kind.startswith("rope"):
            c["rope"].view(-1, 64)[r, 5] = math.nan if kind == "rope nan" else math.inf
        else:  # an e4m3 NaN under a finite scale
            c["codes"].view(torch.uint8).view(-1, 512)[r, 0 if kind == "code" else 499] = 0xFF if kind == "code" else 0x7F
        o, l = _call(cache)(dict(at, cache=c), lens)
        assert _same([o[0, :first], l[0, :first]], [want[0][0, :first], want[1][0, :first]]), kind
        assert _same([o[1:], l[1:]], [want[0][1:], want[1][1:]]), kind
        if kind != "rope inf":  # (which may be a score of minus infinity)
            assert bool(o[0, first:].isnan().all()) and bool(l[0, first:].isnan().all()), kind
    assert dsa.read_device_flags(DEV) == 0


# --- rows that one accumulation does not hold ------------------------------------------------------

def _long_cache(n, four, seed, page=8192):
    """n positions over one page of rows of one sign: their mean is the result of equal weights."""
    g = _gen(seed)
    cache = dict(scales=torch.full((1, page), 255 / 128, device=DEV), rope=torch.zeros((1, page, 64), dtype=torch.bfloat16, device=DEV),
                 block_table=torch.zeros((1, n // page), dtype=torch.int32, device=DEV))
    if four:
        cache["codes"] = torch.randint(1, 8, (1, page, 512), generator=g, device=DEV).to(torch.uint8)
        cache["codes"] = cache["codes"][..., 0::2] + 16 * cache["codes"][..., 1::2]
        cache["groups"] = torch.full((1, page, 16), 127, dtype=torch.uint8, device=DEV)
    else:
        cache["codes"] = (1 + torch.rand((1, page, 512), generator=g, device=DEV) * 15).to(E4M3)
    return cache


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("lg", [16, 18, 20, 22])
@pytest.mark.parametrize("equal", [True, False])
def test_dense_attention_sums_of_values_over_long_rows(lg, equal, four):
    """Equal weights over 2^lg rows, more tiles than SMs: a CTA walks whole tiles.  Weights times scales are 255 = 256 - 1, two e4m3
    terms exactly, so what is off beside bf16's rounding is the sum alone.  Of 2^18 rows at a time it takes 2^14
    additions (four a block of 64), each of which may lose a last place, 2^-23 of a sum that is at most the last: 2^-9; up to
    16 of those are added with at most 2^-24 each, and the weights' own sums are fp32, too: 2^-18 covers both."""
    n, T = 1 << lg, 160
    cache = _long_cache(n, four, lg)
    if equal:
        cache["codes"] = cache["codes"].view(torch.uint8)[:, :1].expand(-1, 8192, -1).contiguous().view(cache["codes"].dtype)
    rows = _latent64(cache, torch.arange(8192, device=DEV)) * 255 / 128
    want = rows.mean(0)
    q = torch.zeros((1, T, 64, 576), dtype=torch.bfloat16, device=DEV)
    o, l = _call(cache)(dict(q=q, cache=cache, scale=1.0), torch.tensor([n], dtype=torch.int32, device=DEV), causal=False)
    off = ((o.double() - want).abs() / want).amax()
    assert float(off) <= BF16_STEP + 2.0 ** (min(lg, 18) - 4 - 23) + FP32_WORK, float(off)
    assert bool(((l.double() - math.log(n)).abs() <= 2.0 ** -14 * (1 + math.log(n))).all())
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("B,T,H,S,lens", [
    (1, 160, 64, 270000, [270000]),                  # two items a tile, and runs that end in either
    (1, 700, 8, 560000, [559990]),                   # 64 / 8 tokens a tile, fewer tiles than SMs
    (1, 640, 16, 262200, [262200]),                  # tiles that end with the second item's first block, or before it
    (200, 1, 64, 530000, [530000 - 2600 * b for b in range(200)]),
    (2, 90, 128, 540000, [540000, 262144]),
    (2, 3, 64, 530000, [530000, 524289]),            # (parts on every SM: one item each)
])
@pytest.mark.parametrize("causal", [True, False])
def test_dense_attention_of_tiles_in_several_items(B, T, H, S, lens, causal, four):
    g = _gen(S)
    cache = _cache(1, S, 64, four, seed=S, spread=0.5)
    if B > 1:  # (the sequences' pages are the same ones, in other orders)
        table = cache["block_table"][0]
        cache["block_table"] = torch.stack([table[torch.randperm(table.numel(), generator=g, device=DEV)] for _ in range(B)]).contiguous()
    some = {(b, t) for b in {0, B // 2, B - 1} for t in {0, 1, T // 2, T - 1}}
    at = dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=S)
    got = _check_dense(at, lens, causal, some=some)
    assert _same(got, _call(cache)(at, torch.tensor(lens, dtype=torch.int32, device=DEV), causal=causal))
    assert dsa.read_device_flags(DEV) == 0


def test_dense_attention_references_that_move_between_items():
    """Scores that rise, or fall, by more than a reference keeps from one item of a tile to the next; empty items first; a
    NaN in the second item reaches the heads of the tokens that see it, all others keep their bits."""
    S, T, H = 800000, 300, 32
    cache = _cache(1, S, 64, four=False)
    cache["scales"].fill_(0.01)
    cache["rope"].zero_()
    flat, pos = cache["rope"].view(-1, 64), torch.arange(S, device=DEV)
    at = _flat(cache, torch.zeros_like(pos), pos)
    q = _q(1, T, H, 0.05)
    q[..., 512] = 8.0
    some = {(0, t) for t in (0, 1, 150, T - 2, T - 1)}
    for step in (131072, 262144, 400000):
        for sign in (1, -1):
            flat[at, 0] = ((pos // step) * 100.0 * sign / 0.01).bfloat16()
            got = _check_dense(dict(q=q, cache=cache, scale=1 / 24), [S], some=some)
    c = dict(cache, codes=cache["codes"].clone())
    c["codes"].view(torch.uint8).view(-1, 512)[at[S - 2], 77] = 0x7F
    o, l = dsa.dsa_latent_attn_dense(dict(q=q, cache=c, scale=1 / 24), torch.tensor([S], dtype=torch.int32, device=DEV))
    assert _same([o[0, :T - 2], l[0, :T - 2]], [got[0][0, :T - 2], got[1][0, :T - 2]])
    assert bool(o[0, T - 2:].isnan().all()) and bool(l[0, T - 2:].isnan().all())
    flat[at, 0] = torch.where(pos < 600000, -math.inf, 0.0).bfloat16()  # nothing but minus infinity in the first items
    _check_dense(dict(q=q, cache=cache, scale=1 / 24), [S], some=some)
    assert dsa.read_device_flags(DEV) == 0


def test_dense_attention_waits_do_not_grow_with_the_rows():
    """2^22 rows, which a CTA walks in 10^8 cycles and more: no wait lasts longer than 4,096 blocks (10^7), so that a limit of 3 * 10^7
    cycles is not met."""
    n, T = 1 << 22, 160
    cache = _long_cache(n, True, 1)
    at = dict(q=_q(1, T, 64, 0.05), cache=cache, scale=1 / 24)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    want = dsa.dsa_latent4_attn_dense(at, lens)
    try:
        dsa.set_wait_limit(30_000_000)
        got = dsa.dsa_latent4_attn_dense(at, lens)
        torch.cuda.synchronize()
    finally:
        dsa.set_wait_limit(0)
    assert dsa.read_device_flags(DEV) == 0 and _same(got, want)


@pytest.mark.parametrize("four,H", [(True, 64), (False, 64), (False, 16)])
def test_dense_attention_lengths_choose_the_kernel(four, H):
    """Room for rows that one accumulation does not hold, whether they are there or not: short sequences give the bits of
    a call that knows they are, and a captured call follows its lengths past 2^18 rows and back."""
    cap, T = 400000, 161 * max(1, 64 // H)
    small = _cache(1, 5000, 64, four, seed=3)
    big = dict(small, block_table=small["block_table"][0].repeat(-(-cap // 64) // small["block_table"].shape[1] + 1)[None, :-(-cap // 64)].contiguous())
    q = _q(1, T, H)
    n = torch.tensor([4900], dtype=torch.int32, device=DEV)
    want = _call(small)(dict(q=q, cache=small, scale=1 / 24, S=5000), n)
    at = dict(q=q, cache=big, scale=1 / 24, S=cap)
    before = dsa.launch_count()
    assert _same(_call(big)(at, n), want)
    assert dsa.launch_count() == before + 3  # (a kernel of which the lengths say that it has nothing to do, too)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _call(big)(at, n)
    some = {(0, 0), (0, T // 2), (0, T - 1)}
    for rows in (4900, 262144, 262145, cap, 0, 4900):
        n.fill_(rows)
        graph.replay()
        assert _same(got, _check_dense(at, [rows], some=some))
    assert _same(got, want) and dsa.read_device_flags(DEV) == 0
