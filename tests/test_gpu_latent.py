"""The serving operators around the sparse attention path against plain 64-bit implementations:
per-head norm and rotation (bf16 and e4m3 out), the paged FP8 latent cache (append, read) and
attention over selected rows of it.  Tolerances count roundings: a bf16 result is off by at most
2^-8 of its value, an e4m3 code by 2^-4 of its value (2^-10 among the subnormals), and the fp32
work before it by a few 2^-24 of the largest term (2^-18 covers sums of up to 1,024 terms)."""
import ctypes
import math
import threading

import pytest
import torch

import long_context_sparse_tcgen05_gb300 as dsa
from long_context_sparse_tcgen05_gb300 import synth

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn
BF16_STEP, E4M3_STEP, FP32_WORK = 2.0 ** -8, 2.0 ** -4, 2.0 ** -18


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


def _angles(rows, angles, seed=0):
    a = torch.rand((rows, angles), generator=_gen(900 + seed), device=DEV, dtype=torch.float64) * 2000 - 1000
    return a.cos().float().contiguous(), a.sin().float().contiguous()


# --- 64-bit forms ----------------------------------------------------------------------------

def _norm64(x, norm, w, b, eps):
    x = x.double()
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    if norm != "none":
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        x = x * w.double()
    return x if b is None else x + b.double()


def _rope64(y, cos, sin, off, inter):
    """cos, sin [..., angles] for the values off .. off + 2 * angles of y's last axis."""
    n = cos.shape[-1]
    y = y.clone()
    r = y[..., off:off + 2 * n]
    a, c = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :n], r[..., n:])
    u, v = a * cos.double() - c * sin.double(), c * cos.double() + a * sin.double()
    y[..., off:off + 2 * n] = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return y


def _norm_rope64(x, norm="none", weight=None, bias=None, eps=1e-6, cos=None, sin=None, rope_off=0, interleaved=False,
                 pos=None):
    y = _norm64(x, norm, weight, bias, eps)
    if cos is not None:
        p = pos.clamp(0, cos.shape[0] - 1)
        y = _rope64(y, cos[p][:, :, None], sin[p][:, :, None], rope_off, interleaved)
    return y


def _assert_bf16(got, ref, what=""):
    top = ref.abs().amax(-1, keepdim=True)
    bad = (got.double() - ref).abs() > BF16_STEP * ref.abs() + FP32_WORK * top
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off"


def _assert_codes(codes, scale, ref, ref_scale, what=""):
    """codes (fp8) against ref / ref_scale, scale against ref_scale."""
    assert bool(((scale.double() - ref_scale).abs() <= FP32_WORK * ref_scale).all()), f"{what}: scales"
    q = ref / ref_scale[..., None]
    bad = (codes.double() - q).abs() > E4M3_STEP * q.abs() + 2.0 ** -10 + 448 * FP32_WORK
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} codes off"


# --- norm and rotation -------------------------------------------------------------------------

NORM_CASES = [
    # B, n, H, d, norm, off, rd, inter
    (1, 1, 1, 8, "none", 0, 8, True),
    (1, 1, 1, 16, "rms", 0, 16, False),
    (2, 3, 5, 24, "layer", 8, 16, False),
    (3, 7, 1, 128, "layer", 0, 64, False),
    (2, 33, 64, 128, "none", 0, 64, False),
    (2, 5, 20, 96, "rms", 32, 64, True),
    (1, 9, 3, 96, "rms", 0, 96, False),
    (2, 4, 7, 64, "rms", 0, 64, True),
    (1, 6, 9, 256, "layer", 192, 64, False),
    (1, 3, 2, 200, "rms", 0, 0, False),
    (1, 5, 4, 576, "none", 512, 64, True),
    (2, 2, 3, 512, "layer", 0, 512, False),
    (1, 3, 2, 1024, "rms", 512, 512, False),
    (1, 2, 1, 1016, "layer", 8, 1008, False),
    (1, 2, 33, 32, "rms", 0, 32, False),
    (1, 400, 1, 40, "layer", 0, 0, False),
]


def _norm_inputs(B, n, H, d, norm, rd, seed, rows=50):
    g = _gen(seed)
    x = (torch.randn((B, n, H, d), generator=g, device=DEV) * 3 + 0.5).bfloat16()
    kw = dict(norm=norm)
    if norm != "none":
        kw["weight"] = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    if norm == "layer":
        kw["bias"] = 0.3 * torch.randn(d, generator=g, device=DEV)
    if rd:
        kw["cos"], kw["sin"] = _angles(rows, rd // 2, seed)
    pos = torch.randint(0, rows, (B, n), generator=g, device=DEV)
    return x, kw, pos


@pytest.mark.parametrize("B,n,H,d,norm,off,rd,inter", NORM_CASES)
def test_norm_rope_matches_64_bits(B, n, H, d, norm, off, rd, inter):
    x, kw, pos = _norm_inputs(B, n, H, d, norm, rd, d + n)
    kw.update(rope_off=off, interleaved=inter)
    y = dsa.dsa_norm_rope(x, positions=pos, **kw)
    _assert_bf16(y, _norm_rope64(x, pos=pos, **kw))
    # consecutive positions known to the host
    y0 = dsa.dsa_norm_rope(x, pos0=3 if n + 3 <= 50 else 0, **kw) if n <= 50 or not rd else None
    if y0 is not None:
        p = (torch.arange(n, device=DEV) + (3 if n + 3 <= 50 else 0)).expand(B, n)
        _assert_bf16(y0, _norm_rope64(x, pos=p, **kw), "pos0")
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_strided_views_and_in_place(inter):
    B, n, H = 2, 5, 6
    g = _gen(3)
    wide = torch.randn((B, n + 2, H + 1, 192), generator=g, device=DEV).bfloat16()
    x = wide[:, 1:n + 1, :H, 128:]
    cos, sin = _angles(9, 32)
    pos = torch.randint(0, 9, (B, n), generator=g, device=DEV)
    dst = torch.full((B, n, H, 576), 7.0, device=DEV, dtype=torch.bfloat16)
    kw = dict(cos=cos, sin=sin, interleaved=inter)
    out = dsa.dsa_norm_rope(x, positions=pos, out=dst[..., 512:], **kw)
    ref = _norm_rope64(x, pos=pos, **kw)
    _assert_bf16(out, ref)
    assert bool((dst[..., :512] == 7).all())
    before = wide.clone()
    dsa.dsa_norm_rope(x, positions=pos, out=x, **kw)  # in place, through the view
    assert torch.equal(x, out)
    before[:, 1:n + 1, :H, 128:] = x
    assert torch.equal(before, wide)


def test_norm_rope_in_place_with_norm_and_wide_heads():
    for d, rd, off in ((1024, 1024, 0), (256, 128, 64), (64, 64, 0), (576, 64, 512)):
        x, kw, pos = _norm_inputs(2, 9, 5, d, "rms", rd, d)
        want = dsa.dsa_norm_rope(x, positions=pos, rope_off=off, **kw)
        dsa.dsa_norm_rope(x, positions=pos, rope_off=off, out=x, **kw)
        assert torch.equal(x, want)


def test_norm_rope_padding_and_bad_positions():
    x, kw, pos = _norm_inputs(2, 6, 5, 64, "rms", 64, 1)
    pos[0, 2], pos[1, 5] = -1, -1
    out = torch.full_like(x, 3.0)
    dsa.dsa_norm_rope(x, positions=pos, out=out, **kw)
    assert dsa.read_device_flags(DEV) == 0
    keep = pos == -1
    assert bool((out[keep] == 3).all())
    _assert_bf16(out[~keep], _norm_rope64(x, pos=pos, **kw)[~keep])
    pos[0, 0], pos[1, 1] = 50, -2  # one past the tables; negative
    out.fill_(3.0)
    dsa.dsa_norm_rope(x, positions=pos, out=out, **kw)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    keep = (pos < 0) | (pos >= 50)
    assert bool((out[keep] == 3).all()) and int(keep.sum()) == 4
    _assert_bf16(out[~keep], _norm_rope64(x, pos=pos, **kw)[~keep])


def test_norm_rope_of_constant_zero_and_non_finite_rows():
    x = torch.zeros((1, 4, 2, 64), device=DEV, dtype=torch.bfloat16)
    x[0, 1] = 5.0
    x[0, 2, 0, 3] = math.nan
    x[0, 3, 1, 0] = math.inf
    for norm in ("rms", "layer"):
        y = dsa.dsa_norm_rope(x, norm=norm)
        assert bool((y[0, 0] == 0).all())
        _assert_bf16(y[0, 1], _norm64(x[0, 1], norm, None, None, 1e-6))
        assert bool(y[0, 2, 0].isnan().all()) and bool((y[0, 2, 1] == 0).all())  # the NaN stays in its head
        assert bool(y[0, 3, 1, 0].isnan()) and bool((y[0, 3, 0] == 0).all())


E4M3_CASES = NORM_CASES + [
    (2, 9, 8, 576, "layer", 512, 64, False),
    (1, 3, 16, 1024, "rms", 0, 64, True),
    (1, 3, 16, 512, "none", 0, 64, False),
    (3, 4, 1, 320, "rms", 0, 64, False),
    (3, 70, 1, 64, "layer", 0, 64, True),
    (2, 5, 2, 128, "none", 64, 64, False),
    (1, 3, 40, 128, "rms", 0, 128, False),
    (1, 2, 128, 128, "none", 0, 64, False),
    (1, 2, 64, 256, "rms", 0, 64, True),
]


@pytest.mark.parametrize("B,n,H,d,norm,off,rd,inter", E4M3_CASES)
@pytest.mark.parametrize("at_position", [False, True])
def test_norm_rope_e4m3_matches_64_bits(B, n, H, d, norm, off, rd, inter, at_position):
    x, kw, pos = _norm_inputs(B, n, H, d, norm, rd, d + n + 7, rows=max(50, n))
    pos = torch.stack([torch.randperm(max(50, n), device=DEV, generator=_gen(b))[:n] for b in range(B)])
    kw.update(rope_off=off, interleaved=inter)
    cap = max(50, n) if at_position else n + 3
    codes = torch.full((B, cap, H * d), 0x11, device=DEV, dtype=torch.uint8)
    scales = torch.full((B, cap), -5.0, device=DEV)
    dsa.dsa_norm_rope_e4m3(x, codes, scales, positions=pos, at_position=at_position, **kw)
    ref = _norm_rope64(x, pos=pos, **kw).flatten(2)
    rows = pos if at_position else torch.arange(n, device=DEV).expand(B, n)
    b = torch.arange(B, device=DEV)[:, None]
    _assert_codes(codes.view(E4M3)[b, rows], scales[b, rows], ref, ref.abs().amax(-1) / 448)
    codes[b, rows], scales[b, rows] = 0x11, -5.0  # and nothing else was written
    assert bool((codes == 0x11).all()) and bool((scales == -5).all())
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("H,d", [(1, 128), (64, 128), (5, 24)])
def test_norm_rope_e4m3_without_norm_equals_the_plain_append(H, d):
    B, n = 3, 11
    x = torch.randn((B, n, H, d), generator=_gen(5), device=DEV).bfloat16()
    x[1, 2] = 0
    want_c, want_s = torch.zeros((B, 40, H * d), device=DEV, dtype=torch.uint8), torch.zeros((B, 40), device=DEV)
    got_c, got_s = want_c.clone(), want_s.clone()
    dsa.dsa_quantize_e4m3_append(x.flatten(2), want_c, want_s, pos0=9)
    dsa.dsa_norm_rope_e4m3(x, got_c, got_s, pos0=9, at_position=True)
    assert torch.equal(got_c, want_c) and torch.equal(got_s, want_s)


def test_norm_rope_e4m3_padding_bad_rows_and_nan():
    x, kw, pos = _norm_inputs(2, 5, 3, 64, "rms", 64, 4)
    pos = torch.tensor([[0, -1, 30, 3, 4], [49, 50, 2, -7, 1]], device=DEV)
    x[0, 3, 1, 5] = math.nan
    codes = torch.full((2, 30, 192), 0x11, device=DEV, dtype=torch.uint8)
    scales = torch.full((2, 30), -5.0, device=DEV)
    dsa.dsa_norm_rope_e4m3(x, codes, scales, positions=pos, at_position=True, **kw)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX  # 30 and 49 are table rows, but no cache rows
    assert bool(scales[0, 3].isnan()) and bool(codes.view(E4M3)[0, 3].float().isnan().all())
    ref = _norm_rope64(x, pos=pos, **kw).flatten(2)
    for b, i, p in ((0, 0, 0), (0, 4, 4), (1, 2, 2), (1, 4, 1)):
        _assert_codes(codes.view(E4M3)[b, p], scales[b, p], ref[b, i], ref[b, i].abs().amax() / 448)
        codes[b, p], scales[b, p] = 0x11, -5.0
    codes[0, 3], scales[0, 3] = 0x11, -5.0
    assert bool((codes == 0x11).all()) and bool((scales == -5).all())


# --- the latent cache --------------------------------------------------------------------------

def _cache(B, cap, page, seed=0, fill=True, spread=0.0):
    """A paged cache (page 0: no table) with shuffled pages; every row, used or not, holds data."""
    g = _gen(seed + 31)
    if page:
        per = -(-cap // page)
        pages = B * per + 2
        table = torch.randperm(pages, generator=g, device=DEV)[:B * per].int().reshape(B, per).contiguous()
    else:
        pages, page, table = B, cap, None
    scales = torch.exp2(torch.randn((pages, page), generator=g, device=DEV) * spread) * 0.01
    codes = torch.randn((pages, page, 512), generator=g, device=DEV) * 100
    return dict(codes=codes.clamp(-448, 448).to(E4M3) if fill else torch.zeros_like(codes).to(E4M3), scales=scales,
                rope=torch.randn((pages, page, 64), generator=g, device=DEV).mul(100).bfloat16(), block_table=table)


def _flat(cache, b, pos):
    page = cache["scales"].shape[1]
    if cache["block_table"] is None:
        return b * page + pos
    return cache["block_table"][b, pos // page].long() * page + pos % page


def _rows64(cache, b, pos):
    r = _flat(cache, b, pos)
    s = cache["scales"].reshape(-1)[r].double()[..., None]
    c = cache["codes"].view(torch.uint8).reshape(-1, 512)[r].view(E4M3).double()
    return torch.cat((c, cache["rope"].reshape(-1, 64)[r].double()), -1) * s


@pytest.mark.parametrize("B,n,cap,page", [(1, 1, 1, 1), (1, 1, 40, 0), (3, 5, 40, 16), (2, 37, 100, 48), (2, 9, 30, 7),
                                          (4, 300, 300, 64), (1, 70, 90, 1), (2, 33, 64, 0)])
@pytest.mark.parametrize("inter,norm,rope", [(True, True, True), (False, True, True), (False, False, True), (True, True, False)])
def test_latent_append_matches_64_bits(B, n, cap, page, inter, norm, rope):
    g = _gen(n + cap)
    cache = _cache(B, cap, page)
    before = {k: v.clone() for k, v in cache.items() if v is not None}
    x = torch.randn((B, n, 576), generator=g, device=DEV) * torch.exp2(4 * torch.rand((B, n, 1), generator=g, device=DEV) - 2)
    x = x.bfloat16()
    w = 1 + 0.3 * torch.randn(512, generator=g, device=DEV) if norm else None
    cos, sin = _angles(cap, 32) if rope else (None, None)
    pos = torch.stack([torch.randperm(cap, generator=g, device=DEV)[:n] for _ in range(B)])
    dsa.dsa_latent_append(x, cache, weight=w, cos=cos, sin=sin, interleaved=inter, positions=pos)
    assert dsa.read_device_flags(DEV) == 0
    lat = _norm64(x[..., :512], "rms" if norm else "none", w, None, 1e-6)
    r = x[..., 512:].double()
    if rope:
        r = _rope64(r, cos[pos], sin[pos], 0, inter)
    s = lat.abs().amax(-1) / 448
    at = _flat(cache, torch.arange(B, device=DEV)[:, None], pos)
    codes, scales, kr = cache["codes"].reshape(-1, 512), cache["scales"].reshape(-1), cache["rope"].reshape(-1, 64)
    _assert_codes(codes.view(torch.uint8)[at].view(E4M3), scales[at], lat, s)
    _assert_bf16(kr[at], r / s[..., None], "rope")
    for name, t in (("codes", codes.view(torch.uint8)), ("scales", scales), ("rope", kr)):
        old = before[name].reshape(t.shape[0], -1) if name != "scales" else before[name].reshape(-1)
        old = old.view(torch.uint8) if name == "codes" else old
        mask = torch.ones(t.shape[0], dtype=torch.bool, device=DEV)
        mask[at.reshape(-1)] = False
        assert torch.equal(t[mask], old[mask]), f"{name}: a row that was not appended changed"


def test_latent_append_strides_host_positions_and_padding():
    B, n, cap = 2, 6, 50
    wide = torch.randn((B, n + 1, 640), generator=_gen(2), device=DEV).bfloat16()
    x = wide[:, :n, 64:]
    cos, sin = _angles(cap, 32)
    a, b = _cache(B, cap, 16), _cache(B, cap, 16)
    dsa.dsa_latent_append(x, a, cos=cos, sin=sin, pos0=11)
    dsa.dsa_latent_append(x.contiguous(), b, cos=cos, sin=sin, positions=(11 + torch.arange(n, device=DEV)).expand(B, n).contiguous())
    for k in ("codes", "scales", "rope"):
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))
    pos = torch.tensor([[0, -1, 49, 50, 4, 5], [-1, -1, 3, -2, 2 ** 40, 6]], device=DEV)
    c = _cache(B, cap, 16)
    c["block_table"][1, 0] = 99  # positions 0..15 of sequence 1 have no page
    old = {k: c[k].clone() for k in ("codes", "scales", "rope")}
    dsa.dsa_latent_append(x, c, cos=cos, sin=sin, positions=pos)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    hit = _flat(c, torch.zeros(4, dtype=torch.long, device=DEV), torch.tensor([0, 49, 4, 5], device=DEV))
    changed = (c["scales"] != old["scales"]).reshape(-1).nonzero().flatten()
    assert sorted(changed.tolist()) == sorted(hit.tolist())


def test_latent_append_zero_tiny_and_non_finite_rows():
    cache = _cache(1, 8, 4)
    x = torch.zeros((1, 5, 576), device=DEV, dtype=torch.bfloat16)
    x[0, :, 512:] = 1.0
    x[0, 1, :512] = 2.0 ** -100
    x[0, 2, 7] = math.nan
    x[0, 3, 9] = math.inf
    x[0, 4, :512] = 3.0
    dsa.dsa_latent_append(x, cache)  # neither norm nor rotation
    y = dsa.dsa_latent_read(cache, n=5)
    s = cache["scales"].reshape(-1)[_flat(cache, torch.zeros(5, dtype=torch.long, device=DEV), torch.arange(5, device=DEV))]
    assert float(s[0]) == 2.0 ** -60 and float(s[1]) == 2.0 ** -60
    assert bool((y[0, :2, :512] == 0).all()) and bool((y[0, :2, 512:] == 1).all())  # a power of two: exact
    assert bool(s[2].isnan()) and bool(y[0, 2].isnan().all())
    assert bool(s[3].isinf()) and bool(y[0, 3, 9].isnan())
    assert bool((y[0, 4, :512] == 3).all())


@pytest.mark.parametrize("B,n,cap,page", [(1, 1, 1, 1), (3, 70, 100, 16), (2, 129, 200, 48), (2, 20, 33, 0), (1, 2048, 5000, 64)])
def test_latent_read_is_the_rounded_product(B, n, cap, page):
    cache = _cache(B, cap, page, spread=3.0)
    b = torch.arange(B, device=DEV)[:, None]
    want = lambda pos: _rows64(cache, b, pos).float().bfloat16()  # noqa: E731  (the fp32 product, rounded)
    n0 = cap - n
    got = dsa.dsa_latent_read(cache, n=n, pos0=n0)
    assert torch.equal(got, want((n0 + torch.arange(n, device=DEV)).expand(B, n)))
    idx = torch.randint(0, cap, (B, n), generator=_gen(n), device=DEV, dtype=torch.int32)
    idx[:, ::5] = -1
    got = dsa.dsa_latent_read(cache, idx)
    assert dsa.read_device_flags(DEV) == 0
    w = want(idx.clamp(min=0).long())
    w[idx < 0] = 0
    assert torch.equal(got, w)


def test_latent_read_bad_positions_and_pages():
    cache = _cache(2, 40, 16)
    cache["block_table"][0, 1], cache["block_table"][1, 2] = -3, 1 << 30
    idx = torch.tensor([[0, 16, 47, 48, -5], [32, 31, -1, 2 ** 31 - 1, 3]], device=DEV, dtype=torch.int32)
    got = dsa.dsa_latent_read(cache, idx)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    ok = torch.tensor([[1, 0, 1, 0, 0], [0, 1, 0, 0, 1]], device=DEV, dtype=torch.bool)
    assert bool((got[~ok] == 0).all())
    b = torch.arange(2, device=DEV)[:, None].expand(2, 5)
    assert torch.equal(got[ok], _rows64(cache, b[ok], idx[ok].long()).float().bfloat16())


def test_latent_cache_past_32_bit_offsets():
    """Rows whose byte offsets pass 2^32: written, read back and attended."""
    rows = (1 << 23) + 4096  # 4 GiB of codes, and a little
    cache = dict(codes=torch.zeros((1, rows, 512), device=DEV, dtype=torch.uint8), scales=torch.ones((1, rows), device=DEV),
                 rope=torch.zeros((1, rows, 64), device=DEV, dtype=torch.bfloat16), block_table=None)
    x = torch.randn((1, 4096, 576), generator=_gen(8), device=DEV).bfloat16()
    dsa.dsa_latent_append(x, cache, pos0=rows - 4096)
    y = dsa.dsa_latent_read(cache, n=4096, pos0=rows - 4096)
    assert bool((cache["codes"][0, :rows - 4096].amax() == 0).all())
    assert bool(((y.double() - x.double()).abs() <= (E4M3_STEP + BF16_STEP) * x.double().abs() + 2.0 ** -9 *
                 x[..., :512].double().abs().amax(-1, keepdim=True) / 448).all())
    idx = (rows - 1 - torch.arange(300, device=DEV)).flip(0).int().reshape(1, 1, 300).contiguous()
    q = torch.randn((1, 1, 8, 576), generator=_gen(9), device=DEV).bfloat16()
    _check_attn(dict(q=q, cache=cache, scale=1 / 24), idx)
    del cache, x, y
    torch.cuda.empty_cache()


# --- attention over the cache ------------------------------------------------------------------

def _attn64(at, idx):
    """(out, lse, tolerance) row by row.  A weight is held to 2^-8 of itself and to 2^-14 of the
    row's largest scaled weight, whatever its own size; a result is then rounded to bf16."""
    q, cache = at["q"], at["cache"]
    B, T, H, _ = q.shape
    S = at.get("S") or 1 << 62
    out = torch.zeros((B, T, H, 512), device=DEV, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((B, T, H), -math.inf, device=DEV, dtype=torch.float64)
    for b in range(B):
        for t in range(T):
            sel = idx[b, t if idx.shape[1] > 1 else 0].long()
            sel = sel[(sel >= 0) & (sel < S)]
            if not sel.numel():
                continue
            rows = _rows64(cache, torch.full_like(sel, b), sel)
            sc = (q[b, t].double() @ rows.T) * at["scale"]
            p = torch.softmax(sc, -1)
            v = rows[:, :512]
            out[b, t] = p @ v
            lse[b, t] = torch.logsumexp(sc, -1)
            s = cache["scales"].reshape(-1)[_flat(cache, torch.full_like(sel, b), sel)].double()
            unit = (v / s[:, None]).abs().sum(0)
            tol[b, t] = BF16_STEP * (out[b, t].abs() + p @ v.abs()) + 2.0 ** -14 * (p * s).amax(-1, keepdim=True) * unit
    return out, lse, tol


def _check_attn(at, idx, lse_tol=2.0 ** -14, **kw):
    o, l = dsa.dsa_latent_attn(at, idx, **kw)
    ref, rl, tol = _attn64(at, idx)
    bad = (o.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values off, worst {float(((o.double() - ref).abs() / tol.clamp(min=1e-300)).max()):.3g}x"
    assert torch.equal(l == -math.inf, rl == -math.inf)
    fin = rl != -math.inf
    # scores are fp32 sums of 576 products: 2^-18 of the largest score, and the logarithm's own
    top = at["q"].float().abs().amax()
    d = (l.double() - rl)[fin].abs()
    assert bool((d <= lse_tol * (1 + rl[fin].abs())).all()), f"lse off by {float(d.max()):.3g} (|q| to {float(top):.3g})"
    return o, l


def _idx(B, T, S, k, seed=0, holes=True):
    g = _gen(seed + 77)
    r = torch.rand((B, T, S), generator=g, device=DEV)
    n = min(k, S)
    idx = torch.full((B, T, k), -1, device=DEV, dtype=torch.int32)
    idx[..., :n] = r.topk(n, -1).indices.sort(-1).values.int()
    if holes:
        idx = torch.where(torch.rand((B, T, k), generator=g, device=DEV) < 0.1, -1, idx)
    return idx.contiguous()


def _q(B, T, H, mul=2.0, seed=0):
    g = _gen(seed + 5)
    temp = torch.exp2(4 * torch.rand((H, 1), generator=g, device=DEV) - 2)
    return (torch.randn((B, T, H, 576), generator=g, device=DEV) * temp * mul).bfloat16()


@pytest.mark.parametrize("B,T,H,S,k,page", [
    (1, 1, 64, 5000, 2048, 64),     # a decode step
    (1, 1, 1, 1, 1, 1),             # one token, one head, one key
    (2, 3, 8, 40, 31, 16),
    (1, 4, 16, 100, 32, 48),
    (2, 5, 20, 100, 33, 7),
    (1, 3, 63, 200, 63, 64),
    (1, 3, 64, 200, 64, 64),
    (3, 2, 65, 200, 65, 64),
    (1, 2, 128, 700, 511, 100),
    (4, 1, 64, 3000, 2048, 64),
    (1, 3, 64, 5000, 4096, 256),
    (2, 90, 64, 400, 129, 64),      # more rows than SMs
    (2, 200, 16, 400, 300, 0),      # no block table
    (1, 7, 32, 30, 100, 16),        # fewer keys than k
    (1, 1, 64, 9000, 8999, 64),     # a long index row
])
def test_latent_attn_matches_64_bits(B, T, H, S, k, page):
    cache = _cache(B, S, page, seed=k)
    _check_attn(dict(q=_q(B, T, H), cache=cache, scale=1 / 24, S=S), _idx(B, T, S, k, seed=H))
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("mul", [1e-3, 8.0, 40.0])
@pytest.mark.parametrize("spread", [0.0, 2.0])
def test_latent_attn_flat_and_peaked_rows(mul, spread):
    """Scores from all equal to one key taking everything, and row scales spread over decades."""
    cache = _cache(2, 600, 64, spread=spread)
    for T in (1, 100):
        _check_attn(dict(q=_q(2, T, 64, mul), cache=cache, scale=1 / 24), _idx(2, T, 600, 512))


def test_latent_attn_rising_scores():
    """Every block's scores far above the previous block's: the reference maximum is raised, and
    the sums rescaled, at every block (and never, in the falling order)."""
    S = 640
    cache = _cache(1, S, 64)
    q = _q(1, 120, 64, 1.0)
    cache["rope"].zero_()
    flat = cache["rope"].view(-1, 64)
    pos = torch.arange(S, device=DEV)
    at = _flat(cache, torch.zeros_like(pos), pos)
    q[..., 512] = 8.0
    for sign in (1, -1):
        flat[at, 0] = ((pos // 32) * 16.0 * sign / 0.01).bfloat16()  # 5.3 nats a block of 32
        cache["scales"].fill_(0.01)
        for T in (1, 120):
            _check_attn(dict(q=q[:, :T], cache=cache, scale=1 / 24), _idx(1, T, S, S, holes=False))


def test_latent_attn_sink_key_and_many_small_weights():
    """One key ahead of 2,047 equal ones by 0 to 12 nats: the many small weights stay exact enough
    together."""
    S = 2048
    cache = _cache(1, S, 64)
    cache["scales"].fill_(0.01)
    cache["rope"].zero_()
    q = torch.zeros((1, 160, 64, 576), device=DEV, dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(0, 12, 64, device=DEV).bfloat16()
    for at_pos in (0, 1000, S - 1):
        c = dict(cache, rope=cache["rope"].clone())
        c["rope"].view(-1, 64)[_flat(c, torch.zeros(1, dtype=torch.long, device=DEV), torch.tensor([at_pos], device=DEV)), 0] = 100.0
        for T in (1, 160):
            _check_attn(dict(q=q[:, :T], cache=c, scale=1.0), _idx(1, T, S, S, holes=False))


def test_latent_attn_empty_and_sparse_rows():
    cache = _cache(2, 300, 64)
    idx = _idx(2, 6, 300, 256)
    idx[0, 1], idx[1, 5] = -1, -1
    idx[0, 2, :255] = -1          # only the last entry may be valid
    idx[0, 2, 255] = 17
    idx[1, 0, 1:] = -1            # only the first
    idx[1, 0, 0] = 299
    idx[1, 1, :100] = -1          # leading blocks empty
    idx[1, 2, 64:200] = -1        # blocks in the middle empty
    for H in (64, 5):
        o, l = _check_attn(dict(q=_q(2, 6, H), cache=cache, scale=0.05), idx)
        assert bool((o[0, 1] == 0).all()) and bool((l[0, 1] == -math.inf).all())
    big = idx.repeat(1, 40, 1).contiguous()
    _check_attn(dict(q=_q(2, 240, 64), cache=cache, scale=0.05), big)


@pytest.mark.parametrize("T,H,S,k,mul", [(3000, 16, 2000, 700, 2.0), (1500, 64, 4000, 1500, 12.0), (2000, 70, 500, 64, 2.0)])
def test_latent_attn_many_rows_per_cta(T, H, S, k, mul):
    """Rows of every length, empty ones among them, one after another in each CTA: sampled rows
    against 64 bits, the whole against a second run."""
    cache = _cache(1, S, 64)
    idx = _idx(1, T, S, k)
    n = torch.randint(0, k + 1, (T,), generator=_gen(T), device=DEV)
    n[::9], n[4::9], n[5::9] = 0, k, 1
    n[100:400] = n[100:400].clamp(max=64)      # long runs of one-block and empty rows
    n[200:230] = 0
    idx[0][torch.arange(k, device=DEV) >= n[:, None]] = -1
    at = dict(q=_q(1, T, H, mul), cache=cache, scale=1 / 24)
    o, l = dsa.dsa_latent_attn(at, idx)
    assert dsa.read_device_flags(DEV) == 0
    for _ in range(3):
        o2, l2 = dsa.dsa_latent_attn(at, idx)
        assert torch.equal(o, o2) and torch.equal(l, l2)
    rows = torch.arange(0, T, T // 60, device=DEV)
    ref, rl, tol = _attn64(dict(at, q=at["q"][:, rows]), idx[:, rows])
    assert not bool(((o[:, rows].double() - ref).abs() > tol).any())
    assert torch.equal(l[:, rows] == -math.inf, rl == -math.inf)
    assert bool(((l[:, rows].double() - rl)[rl != -math.inf].abs() <= 2.0 ** -14 * (1 + rl[rl != -math.inf].abs())).all())
    assert bool((o[0, n == 0] == 0).all()) and dsa.read_device_flags(DEV) == 0


def test_latent_attn_repeated_positions_count_twice():
    cache = _cache(1, 50, 16)
    idx = torch.tensor([3, 3, 3, 9, 40, 40] * 30, device=DEV, dtype=torch.int32).reshape(1, 1, 180)
    _check_attn(dict(q=_q(1, 1, 64), cache=cache, scale=0.05), idx)


def test_latent_attn_bad_indices_and_pages_are_skipped_and_flagged():
    cache = _cache(1, 100, 16)
    at = dict(q=_q(1, 2, 64), cache=cache, scale=0.05, S=90)
    good = _idx(1, 2, 90, 64, holes=False)
    bad = good.clone()
    bad[0, 0, 5], bad[0, 0, 6], bad[0, 1, 63] = 90, -2, 2 ** 31 - 1
    masked = good.clone()
    masked[0, 0, 5], masked[0, 0, 6], masked[0, 1, 63] = -1, -1, -1
    o, l = dsa.dsa_latent_attn(at, bad)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    _check_attn(at, masked)
    o2, l2 = dsa.dsa_latent_attn(at, masked)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    assert dsa.read_device_flags(DEV) == 0
    lost = cache["block_table"].clone()
    lost[0, 2] = cache["scales"].shape[0]  # positions 32..47
    o, l = dsa.dsa_latent_attn(dict(at, cache=dict(cache, block_table=lost)), good)
    assert dsa.read_device_flags(DEV) == dsa.FLAG_BAD_INDEX
    o2, l2 = dsa.dsa_latent_attn(at, torch.where((good >= 32) & (good < 48), -1, good))
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("T", [1, 170])
def test_latent_attn_ignores_what_it_does_not_select(T):
    """NaN and infinities in rows that are masked, unselected or behind the sequence."""
    B, S = 1, 500
    cache = _cache(B, S, 48)
    idx = _idx(B, T, S, 300)
    at = dict(q=_q(B, T, 64), cache=cache, scale=0.05, S=S)
    want = dsa.dsa_latent_attn(at, idx)
    used = torch.zeros(cache["scales"].numel(), dtype=torch.bool, device=DEV)
    sel = idx[idx >= 0].long()
    used[_flat(cache, torch.zeros_like(sel), sel)] = True
    dirty = {k: v.clone() for k, v in cache.items()}
    dirty["codes"].view(torch.uint8).view(-1, 512)[~used] = 0x7F  # NaN
    dirty["scales"].view(-1)[~used] = math.inf
    dirty["rope"].view(-1, 64)[~used] = -math.inf
    got = dsa.dsa_latent_attn(dict(at, cache=dirty), idx)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_latent_attn_nan_reaches_only_its_rows():
    cache = _cache(1, 300, 64)
    idx = _idx(1, 200, 300, 128)
    q = _q(1, 200, 64)
    want, wl = dsa.dsa_latent_attn(dict(q=q, cache=cache, scale=0.05), idx)
    q2 = q.clone()
    q2[0, 3, 7, 100] = math.nan
    got, gl = dsa.dsa_latent_attn(dict(q=q2, cache=cache, scale=0.05), idx)
    assert bool(got[0, 3, 7].isnan().all()) and bool(gl[0, 3, 7].isnan())
    got[0, 3, 7], gl[0, 3, 7] = want[0, 3, 7], wl[0, 3, 7]
    assert torch.equal(got, want) and torch.equal(gl, wl)
    # a key whose score is minus infinity weighs nothing
    c = {k: v.clone() for k, v in cache.items()}
    pos = int(idx[0, 0][idx[0, 0] >= 0][3])
    c["rope"].view(-1, 64)[_flat(c, torch.zeros(1, dtype=torch.long, device=DEV), torch.tensor([pos], device=DEV)), 5] = -math.inf
    q3 = q.clone()
    q3[..., 517] = q3[..., 517].abs() + 0.5
    a, al = dsa.dsa_latent_attn(dict(q=q3, cache=c, scale=0.05), idx)
    _check_attn(dict(q=q3, cache=cache, scale=0.05), torch.where(idx == pos, -1, idx))
    b, bl = dsa.dsa_latent_attn(dict(q=q3, cache=cache, scale=0.05), torch.where(idx == pos, -1, idx))
    assert bool(((a.double() - b.double()).abs() <= 2 * BF16_STEP * b.double().abs().amax()).all())
    assert bool(((al - bl).abs() <= 1e-4).all())


def test_latent_attn_strided_queries_shared_rows_and_optional_lse():
    B, T, H = 2, 4, 24
    cache = _cache(B, 400, 64)
    wide = torch.randn((B, T + 1, H + 2, 576), generator=_gen(4), device=DEV).bfloat16()
    q = wide[:, 1:, 1:H + 1]
    idx = _idx(B, 1, 400, 200)
    o, l = _check_attn(dict(q=q, cache=cache, scale=0.05), idx)
    o2, l2 = dsa.dsa_latent_attn(dict(q=q.contiguous(), cache=cache, scale=0.05), idx.expand(B, T, 200).contiguous(), lse=False)
    assert l2 is None and torch.equal(o, o2)


def test_latent_attn_of_the_row_s_own_bytes():
    """A cache written by the plain append (codes and scales of the latent part) is attended too."""
    B, S = 2, 130
    x = torch.randn((B, S, 512), generator=_gen(6), device=DEV).bfloat16()
    codes, scales = torch.zeros((B, S, 512), device=DEV, dtype=torch.uint8), torch.ones((B, S), device=DEV)
    dsa.dsa_quantize_e4m3_append(x, codes, scales)
    cache = dict(codes=codes, scales=scales, rope=torch.zeros((B, S, 64), device=DEV, dtype=torch.bfloat16), block_table=None)
    _check_attn(dict(q=_q(B, 3, 64), cache=cache, scale=1 / 24), _idx(B, 3, S, 100))


def _decode_call(seed):
    cache = _cache(4, 3000, 64, seed=seed)
    return dict(q=_q(4, 1, 64, seed=seed), cache=cache, scale=1 / 24), _idx(4, 1, 3000, 2048, seed=seed)


def test_latent_attn_on_two_streams_at_once():
    calls = [_decode_call(s) for s in (1, 2)]
    want = [dsa.dsa_latent_attn(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(dsa.dsa_latent_attn(*calls[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_captured_graphs_keep_their_own_scratch():
    """Two graphs of split (decode) calls, replayed at the same time with new queries in place."""
    calls = [_decode_call(s) for s in (3, 4)]
    for c in calls:
        dsa.dsa_latent_attn(*c)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dsa.dsa_latent_attn(*c))
        graphs.append(g)
    fresh = [_decode_call(s)[0]["q"] for s in (13, 14)]
    for c, q in zip(calls, fresh):
        c[0]["q"].copy_(q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, o in zip(calls, outs):
        w = dsa.dsa_latent_attn(*c)
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_latent_attn_caller_workspace():
    at, idx = _decode_call(5)
    want = dsa.dsa_latent_attn(at, idx)
    a = dsa.latent_attn_struct(at, idx)
    need = dsa.load_library().dsa_latent_attn_workspace_size(ctypes.byref(a), idx.shape[2])
    big = torch.zeros(need, dtype=torch.uint8, device=DEV)
    got = dsa.dsa_latent_attn(at, idx, ws=big)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    small = torch.zeros(dsa.WS_MIN, dtype=torch.uint8, device=DEV)  # no room for split parts: unsplit
    _check_attn(at, idx, ws=small)


# --- the operators together --------------------------------------------------------------------

def test_serving_chain_from_projections_to_attention():
    """What a serving step does with them: a prompt's indexer keys and latent rows appended with
    norm and rotation, the FP8 indexer and top-k over the appended keys, attention over the paged
    latent cache, then single new tokens on top; against the same chain in 64 bits, and the cache
    read back for the bf16 path."""
    B, S, H, k = 2, 900, 64, 256
    g = _gen(42)
    new = 3
    cap = S + new
    cos, sin = _angles(cap, 32)
    hid = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    kv, ik = hid(B, cap, 576), hid(B, cap, 1, 128)
    w_kv = 1 + 0.2 * torch.randn(512, generator=g, device=DEV)
    w_ik, b_ik = 1 + 0.2 * torch.randn(128, generator=g, device=DEV), 0.1 * torch.randn(128, generator=g, device=DEV)
    cache = _cache(B, cap, 48, fill=False)
    k_codes = torch.zeros((B, cap, 128), device=DEV, dtype=torch.uint8)
    k_scale = torch.ones((B, cap), device=DEV)

    def append(lo, hi):
        dsa.dsa_latent_append(kv[:, lo:hi], cache, weight=w_kv, cos=cos, sin=sin, interleaved=True, pos0=lo)
        dsa.dsa_norm_rope_e4m3(ik[:, lo:hi], k_codes, k_scale, norm="layer", weight=w_ik, bias=b_ik, cos=cos, sin=sin, pos0=lo,
                               at_position=True)

    def step(lo, hi):
        """Queries lo .. hi - 1: indexer top-k, then attention; (out, lse, idx, q)."""
        T = hi - lo
        iq, q_raw, w = hid(B, T, 64, 128), hid(B, T, H, 576), torch.rand((B, T, 64), generator=g, device=DEV) / 8
        q_codes = torch.zeros((B, T, 64 * 128), device=DEV, dtype=torch.uint8)
        q_scale = torch.ones((B, T), device=DEV)
        dsa.dsa_norm_rope_e4m3(iq, q_codes, q_scale, cos=cos, sin=sin, pos0=lo)
        ix = dict(q=q_codes.view(E4M3).view(B, T, 64, 128), q_scale=q_scale, w=w, k=k_codes.view(E4M3), k_scale=k_scale,
                  q_pos0=lo, diag=1)
        idx = dsa.dsa_topk(k, ix=ix)
        q = q_raw.clone()
        dsa.dsa_norm_rope(q_raw[..., 512:], cos=cos, sin=sin, interleaved=True, pos0=lo, out=q[..., 512:])
        ref_q = _rope64(q_raw.double(), cos[lo:hi][None, :, None], sin[lo:hi][None, :, None], 512, True)
        _assert_bf16(q, ref_q, "queries")
        o, l = _check_attn(dict(q=q, cache=cache, scale=1 / 24, S=cap), idx)
        assert bool((idx.amax(-1) <= torch.arange(lo, hi, device=DEV)).all())
        return o, l, idx, q

    append(0, S)
    step(S - 40, S)          # the last chunk of the prompt
    for t in range(S, S + new):
        append(t, t + 1)
        o, l, idx, q = step(t, t + 1)
    # the cache read back serves the bf16 path: the same selection there
    rows = dsa.dsa_latent_read(cache, n=cap)
    o2, l2 = dsa.dsa_sparse_attn(dict(q=q, k=rows, v=None, d_v=512, scale=1 / 24), idx)
    assert bool(((o.double() - o2.double()).abs() <= 2e-2).all()) and bool(((l - l2).abs() <= 1e-2).all())
    lat = _norm64(kv[..., :512], "rms", w_kv, None, 1e-6)
    assert bool(((rows[..., :512].double() - lat).abs() <= (E4M3_STEP + BF16_STEP) * lat.abs() +
                 2.0 ** -9 * lat.abs().amax(-1, keepdim=True) / 448).all())
    assert dsa.read_device_flags(DEV) == 0


def test_trace_names_the_cache_kernels():
    cache = _cache(1, 8, 4)
    x = torch.randn((1, 4, 576), device=DEV).bfloat16()
    dsa.trace_enable(64)
    try:
        dsa.dsa_latent_append(x, cache)
        dsa.dsa_latent_read(cache, n=4)
        dsa.dsa_norm_rope(x.view(1, 4, 9, 64), norm="rms")
        kinds = [r[0] for r in dsa.trace_read()]
    finally:
        dsa.trace_disable()
    assert kinds == ["cache"] * 3


def test_captured_appends_norms_and_reads_replay():
    """One decode step's cache work in a graph: positions advance in place between replays."""
    B, cap = 3, 40
    cos, sin = _angles(cap, 32)
    x = torch.randn((B, 1, 576), generator=_gen(1), device=DEV).bfloat16()
    pos = torch.zeros((B, 1), device=DEV, dtype=torch.int64)
    a, b = _cache(B, cap, 16), _cache(B, cap, 16)
    kc = torch.zeros((B, cap, 64), device=DEV, dtype=torch.uint8)
    ks = torch.ones((B, cap), device=DEV)

    def work(c):
        dsa.dsa_latent_append(x, c, cos=cos, sin=sin, positions=pos)
        dsa.dsa_norm_rope_e4m3(x[..., 512:].unflatten(-1, (1, 64)), kc, ks, norm="rms", positions=pos, at_position=True)
        return dsa.dsa_latent_read(c, pos.int())

    work(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = work(a)
    for t in range(5):
        pos.fill_(7 * t)
        x.normal_(generator=_gen(t))
        g.replay()
        want = work(b)
        assert torch.equal(y, want)
    for t in range(5):
        p = torch.full((B, 1), 7 * t, device=DEV, dtype=torch.int32)
        assert torch.equal(dsa.dsa_latent_read(a, p), dsa.dsa_latent_read(b, p))
    assert dsa.read_device_flags(DEV) == 0


def test_synth_latent_shape_is_the_cache_s():
    wl = synth.WORKLOADS["prefill_16k"]
    assert (wl.DQK, wl.DV) == (576, 512)


@pytest.mark.parametrize("B,T,H,S,k", [(1, 400, 64, 4000, 512), (2, 1, 128, 4000, 2048), (1, 900, 16, 3000, 64)])
def test_latent_attn_waits_that_run_out(B, T, H, S, k):
    """A limit of one cycle: every wait that is not complete at the first look gives up, the kernel
    ends what it has in flight and raises the flag; the same call with the default limit is right."""
    cache = _cache(B, S, 64)
    at = dict(q=_q(B, T, H), cache=cache, scale=1 / 24)
    idx = _idx(B, T, S, k)
    want, lse = dsa.dsa_latent_attn(at, idx)
    assert dsa.read_device_flags(DEV) == 0
    raised = False
    for _ in range(3):
        try:
            dsa.set_wait_limit(1)
            dsa.dsa_latent_attn(at, idx)
            torch.cuda.synchronize()
        finally:
            dsa.set_wait_limit(0)
        flags = dsa.read_device_flags(DEV)  # read, and cleared, after every call
        raised = raised or bool(flags & dsa.FLAG_TIMEOUT)
    assert raised
    o, l = dsa.dsa_latent_attn(at, idx)
    assert dsa.read_device_flags(DEV) == 0
    assert torch.equal(o, want) and torch.equal(l, lse)


def test_broadcast_operands_are_refused():
    """A stride of 0 means dense to the library: a broadcast view would be read past its end."""
    x = torch.zeros(1, 3, 4, 64, device=DEV, dtype=torch.bfloat16)
    for view in (x.expand(2, 3, 4, 64), x[:, :1].expand(1, 5, 4, 64), x[:, :, :1].expand(1, 3, 7, 64)):
        with pytest.raises(AssertionError, match="broadcast"):
            dsa.dsa_norm_rope(view)
        with pytest.raises(AssertionError, match="broadcast"):
            dsa.dsa_norm_rope(torch.zeros(view.shape, device=DEV, dtype=torch.bfloat16), out=view)
    cache = _cache(2, 20, 16)
    row = torch.zeros(1, 1, 576, device=DEV, dtype=torch.bfloat16)
    for view in (row.expand(2, 1, 576), row.expand(2, 4, 576)):
        with pytest.raises(AssertionError, match="broadcast"):
            dsa.dsa_latent_append(view, cache)
    at = dict(q=_q(1, 1, 8).expand(2, 1, 8, 576), cache=cache, scale=0.05)
    with pytest.raises(AssertionError, match="broadcast"):
        dsa.dsa_latent_attn(at, _idx(2, 1, 20, 4))
    with pytest.raises(AssertionError):
        dsa.dsa_latent_attn(dict(at, q=_q(2, 1, 8), S=2 ** 32 + 5), _idx(2, 1, 20, 4))


@pytest.mark.parametrize("rows", [2, 16, 21, 26, 33, 45, 60, 76, 77, 153])
@pytest.mark.parametrize("H", [64, 20, 128])
def test_latent_attn_rows_of_every_split(rows, H):
    """From eight parts a row to one: rows cut short, so that parts are empty, and empty rows."""
    S, k = 1500, 1100
    cache = _cache(1, S, 48)
    idx = _idx(1, rows, S, k)
    n = torch.randint(0, k + 1, (rows,), generator=_gen(rows), device=DEV)
    n[0], n[-1], n[rows // 2] = 130, k, 0
    idx[0][torch.arange(k, device=DEV) >= n[:, None]] = -1
    at = dict(q=_q(1, rows, H), cache=cache, scale=1 / 24)
    _check_attn(at, idx)
    o, l = dsa.dsa_latent_attn(at, idx)
    o2, l2 = dsa.dsa_latent_attn(at, idx)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    assert bool((o[0, n == 0] == 0).all()) and bool((l[0, n == 0] == -math.inf).all())


# --- rope values that the row's scale does not bound ---------------------------------------------

def _append_rope(rope, top, **kw):
    """(stored rope values, scales) of rows with the rope values `rope` [n, 64] and latent values
    whose largest is `top`, on the host."""
    cache = _cache(1, rope.shape[0], 0, fill=False)
    x = torch.zeros((1, rope.shape[0], 576), device=DEV, dtype=torch.bfloat16)
    x[0, :, 3] = top
    x[0, :, 512:] = rope.to(DEV)
    dsa.dsa_latent_append(x, cache, **kw)
    return cache["rope"][0].cpu(), cache["scales"][0].cpu()


def _assert_same(got, want):
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} differ, first {got[bad][:4]} for {want[bad][:4]}"


def _bf16_values():
    """Every bf16 value, in rows of 64."""
    return torch.arange(-2 ** 15, 2 ** 15).to(torch.int16).view(torch.bfloat16).reshape(-1, 64)


# scales of 2^-60 (an all-zero latent row), 2^-52, ordinary ones, 2^50, 2^60 and beyond
LATENT_TOPS = [0.0, 448 * 2.0 ** -52, 0.01, 1.0, 3.0, 448 * 2.0 ** 50, 448 * 2.0 ** 60, 1e30, 3e38]


@pytest.mark.parametrize("top", LATENT_TOPS)
def test_latent_append_rope_is_the_ieee_quotient(top):
    """rope = bf16(value / scale), bit for bit, for every finite bf16 value: quotients that overflow
    are infinite, not NaN."""
    v = _bf16_values()
    v = torch.where(v.isfinite(), v, 0.0)
    got, s = _append_rope(v, top)
    _assert_same(got, (v.float() / s[:, None]).bfloat16())


@pytest.mark.parametrize("top", LATENT_TOPS)
@pytest.mark.parametrize("inter", [False, True])
def test_latent_append_infinite_rope_values_stay_infinite(top, inter):
    """A pair (inf, c) turned by an angle whose cosine and sine are both positive is (inf, inf)."""
    v = torch.ones((4, 64))
    a = slice(0, None, 2) if inter else slice(0, 32)
    v[1, a], v[2, a], v[3, a] = math.inf, -math.inf, math.nan
    cos, sin = torch.full((4, 32), 0.6, device=DEV), torch.full((4, 32), 0.8, device=DEV)
    got, _ = _append_rope(v.bfloat16(), top, cos=cos, sin=sin, interleaved=inter)
    assert bool(got[0].isfinite().all())
    assert bool((got[1] == math.inf).all()) and bool((got[2] == -math.inf).all()) and bool(got[3].isnan().all())


@pytest.mark.parametrize("top", LATENT_TOPS)
def test_latent_append_without_rotation_keeps_each_rope_value_to_itself(top):
    """Every bf16 value, infinities and NaN among them, beside finite partners in both pairings."""
    v = _bf16_values()
    for rows in (v, torch.stack((v, torch.ones_like(v)), -1).reshape(-1, 64),
                 torch.cat((v.reshape(-1, 32), torch.ones_like(v).reshape(-1, 32)), -1)):
        for inter in (False, True):
            got, s = _append_rope(rows, top, interleaved=inter)
            _assert_same(got, (rows.float() / s[:, None]).bfloat16())


# --- attention: sums and accuracy ----------------------------------------------------------------

@pytest.mark.parametrize("T", [1, 160])
def test_latent_attn_rows_of_the_least_scale_far_above_the_first_block(T):
    """Ordinary rows, then rows with nothing but rope values (an all-zero latent row's scale is 2^-60)
    whose scores lie 30 to 110 nats above them: the row sums, which weigh a row by 1 / scale, stay
    finite whatever the distance, in one part (T = 160) and in several."""
    S, first = 2048, 64
    cache = _cache(1, S, 64)
    cache["rope"].zero_()
    cache["scales"].fill_(0.01)
    at = _flat(cache, torch.zeros(S - first, dtype=torch.long, device=DEV), torch.arange(first, S, device=DEV))
    cache["codes"].view(torch.uint8).view(-1, 512)[at] = 0
    cache["scales"].view(-1)[at] = 2.0 ** -60
    cache["rope"].view(-1, 64)[at, 0] = 2.0 ** 60  # a rope value of 1
    q = torch.zeros((1, T, 64, 576), device=DEV, dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(30, 110, 64, device=DEV).bfloat16()
    _check_attn(dict(q=q, cache=cache, scale=1.0), _idx(1, T, S, S, holes=False))
    assert dsa.read_device_flags(DEV) == 0


@pytest.mark.parametrize("k", [64, 129, 192, 257, 384, 448, 511])
def test_latent_attn_short_index_rows_are_not_split(k):
    """Joining parts takes as long as six blocks of keys: a single row of up to 511 entries is one
    part, so it comes out bit for bit as it does among many rows."""
    cache = _cache(1, 3000, 64, seed=k)
    q, idx = _q(1, 200, 64, seed=k), _idx(1, 200, 3000, k, seed=k)
    want, wl = dsa.dsa_latent_attn(dict(q=q, cache=cache, scale=1 / 24), idx)
    got, gl = dsa.dsa_latent_attn(dict(q=q[:, 7:8], cache=cache, scale=1 / 24), idx[:, 7:8].contiguous())
    assert torch.equal(got, want[:, 7:8]) and torch.equal(gl, wl[:, 7:8])


@pytest.mark.parametrize("k", [512, 513, 575, 576, 640, 767, 768, 1025])
@pytest.mark.parametrize("rows", [1, 30, 70])
def test_latent_attn_around_the_lengths_that_are_split(k, rows):
    cache = _cache(1, 1200, 48, seed=k)
    _check_attn(dict(q=_q(1, rows, 64), cache=cache, scale=1 / 24), _idx(1, rows, 1200, k, seed=rows))


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("mul", [1e-3, 0.25])
def test_latent_attn_flat_rows_norm_wise(T, mul):
    """Heads that weigh all of 2,048 rows alike: the sum of independent values of either sign is some
    45 times smaller than the sum of their magnitudes, which bounds no such result.  Rounding the
    result takes 2^-8 of its norm.  A weight is off by 2^-8 of itself at most; equal weights are off
    alike, which scales the result, and unequal ones add up like the independent values they weigh:
    2^-8 of the norm again, a third more for the spread of 512 products' norms.  (Without its second
    term a weight is off by 2^-4, and a lost row of 2,048 takes 2^-5.5.)"""
    cache = _cache(1, 4000, 64)
    at = dict(q=_q(1, T, 64, mul), cache=cache, scale=1 / 24)
    idx = _idx(1, T, 4000, 2048, holes=False)
    o, _ = dsa.dsa_latent_attn(at, idx)
    ref, _, _ = _attn64(at, idx)
    off = (o.double() - ref).norm(dim=-1)
    assert bool((off <= (1 + 4 / 3) * BF16_STEP * ref.norm(dim=-1)).all()), f"{float((off / ref.norm(dim=-1)).max()):.3g}"


def test_latent_attn_longest_index_row():
    cache = _cache(1, 70000, 64)
    _check_attn(dict(q=_q(1, 1, 20), cache=cache, scale=1 / 24), _idx(1, 1, 70000, 65536))


@pytest.mark.parametrize("T", [1, 170])
def test_latent_attn_rows_whose_every_score_is_minus_infinity_are_empty(T):
    cache = _cache(1, 900, 64)
    cache["rope"][..., 5] = -math.inf
    q = _q(1, T, 64)
    q[..., 517] = q[..., 517].abs() + 0.5
    o, l = dsa.dsa_latent_attn(dict(q=q, cache=cache, scale=0.05), _idx(1, T, 900, 700))
    assert bool((o == 0).all()) and bool((l == -math.inf).all())


def test_latent_attn_of_very_large_and_very_small_queries():
    """Powers of two moved from the softmax scale into the queries change nothing."""
    cache = _cache(2, 600, 64)
    q, idx = _q(2, 3, 64, 1.0), _idx(2, 3, 600, 300)
    want, wl = dsa.dsa_latent_attn(dict(q=q, cache=cache, scale=1 / 24), idx)
    for e in (90, -80):
        o, l = dsa.dsa_latent_attn(dict(q=(q.float() * 2.0 ** e).bfloat16(), cache=cache, scale=2.0 ** -e / 24), idx)
        assert torch.equal(o, want) and torch.equal(l, wl)


# --- flag words ----------------------------------------------------------------------------------

def _read_flags(ws):
    """The flag word of a workspace, on the calling thread's current stream."""
    v = ctypes.c_uint32()
    status = dsa.load_library().dsa_read_device_flags(ctypes.c_void_p(ws.data_ptr()), ctypes.byref(v),
                                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0
    return int(v.value)


def test_flags_raised_while_another_stream_reads_are_not_lost():
    """One thread reads the word without pause while calls with a bad index raise it on a stream of
    their own: each raised bit is in one of the reads, the reader's or the caller's own."""
    cache = _cache(1, 20, 16)
    at = dict(q=_q(1, 1, 1), cache=cache, scale=0.05)
    idx = torch.tensor([[[5, 40]]], device=DEV, dtype=torch.int32)  # 40: past the 32 rows of the sequence
    ws = torch.zeros(dsa.WS_MIN, dtype=torch.uint8, device=DEV)
    dsa.dsa_latent_attn(at, idx, ws=ws)
    assert _read_flags(ws) == dsa.FLAG_BAD_INDEX and _read_flags(ws) == 0
    rounds, seen, stop = [0], [0], threading.Event()

    def reader():
        with torch.cuda.stream(torch.cuda.Stream()):
            while not stop.is_set():
                seen[0] += _read_flags(ws) != 0
                rounds[0] += 1

    t = threading.Thread(target=reader)
    t.start()
    lost = 0
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(500):
                before = seen[0]
                dsa.dsa_latent_attn(at, idx, ws=ws)
                own = _read_flags(ws)
                now = rounds[0]
                while rounds[0] < now + 2 and t.is_alive():  # a read that was under way has been counted
                    pass
                lost += seen[0] == before and not own
    finally:
        stop.set()
        t.join()
    assert lost == 0 and _read_flags(ws) == 0
    assert dsa.read_device_flags(DEV) == 0


def test_latent_attn_flags_go_to_the_word_that_the_call_names():
    """The size query asks for the flag word only; a caller's workspace, or the word that the arguments
    name, takes the call's flags, and the device's own word stays clean."""
    cache = _cache(1, 20, 16)
    at = dict(q=_q(1, 1, 8), cache=cache, scale=0.05)
    bad = torch.tensor([[[5, 40]]], device=DEV, dtype=torch.int32)  # 40: past the 32 rows of the sequence
    lib = dsa.load_library()
    a = dsa.latent_attn_struct(at, bad)
    assert lib.dsa_latent_attn_workspace_size(ctypes.byref(a), 2) == dsa.WS_MIN
    ws = torch.zeros(dsa.WS_MIN, dtype=torch.uint8, device=DEV)
    dsa.dsa_latent_attn(at, bad, ws=ws)
    assert dsa.read_device_flags(DEV) == 0 and _read_flags(ws) == dsa.FLAG_BAD_INDEX
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty((1, 1, 8, 512), dtype=torch.bfloat16, device=DEV)
    a.flags = word.data_ptr()
    assert lib.dsa_latent_attn(ctypes.byref(a), bad.data_ptr(), 2, out.data_ptr(), None, ws.data_ptr(), dsa.WS_MIN,
                               torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(word) == dsa.FLAG_BAD_INDEX and _read_flags(ws) == 0
    with pytest.raises(dsa.DsaError):
        dsa.dsa_latent_attn(at, bad, ws=ws[:-16])
    assert dsa.read_device_flags(DEV) == 0


def test_read_device_flags_refuses_host_memory():
    ws = torch.zeros(dsa.WS_MIN, dtype=torch.uint8)
    v = ctypes.c_uint32()
    assert dsa.load_library().dsa_read_device_flags(ctypes.c_void_p(ws.data_ptr()), ctypes.byref(v), None) == 1
