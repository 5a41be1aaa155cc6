"""C-ABI checks of the latent cache and norm entry points that need no GPU: struct layouts, and the
host-side validation that rejects a bad call before any launch."""
import contextlib
import ctypes
import os
import subprocess
import types

import pytest
import torch

import long_context_sparse_tcgen05_gb300 as dsa
from long_context_sparse_tcgen05_gb300 import build as dsa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 1 << 20  # a 16-byte aligned address that no rejected call touches


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


def test_struct_layouts_match_header(tmp_path):
    structs = [("dsa_norm_rope_args", dsa.NormRopeArgs), ("dsa_latent_cache", dsa.LatentCache),
               ("dsa_latent_append_args", dsa.LatentAppendArgs), ("dsa_latent_attn_args", dsa.LatentAttnArgs)]
    lines, want = [], []
    for name, cls in structs:
        lines.append(f'printf("%zu ", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void){' + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()] == want


def _edit(s, edits):
    for k, v in edits.items():
        obj, *rest = k.split(".")
        setattr(getattr(s, obj), rest[0], v) if rest else setattr(s, obj, v)
    return s


def _norm(**kw):
    a = dsa.NormRopeArgs(B=2, n=3, H=4, d=64, x=FAKE, norm=1, eps=1e-6, weight=FAKE, cos=FAKE, sin=FAKE, rope_off=0,
                         rope_dim=64, max_pos=100, positions=FAKE)
    return _edit(a, kw)


NORM_BAD = [
    (dict(B=0), INVALID), (dict(n=-1), INVALID), (dict(H=0), INVALID), (dict(x=None), INVALID),
    (dict(d=12), UNSUPPORTED), (dict(d=1032), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(norm=3), INVALID),
    (dict(norm=0), INVALID), (dict(norm=1, bias=FAKE), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x_stride_h=56), INVALID), (dict(x_stride_b=-8), INVALID), (dict(x_stride_t=12), MISALIGNED),
    (dict(x=FAKE + 2), MISALIGNED), (dict(weight=FAKE + 4), MISALIGNED), (dict(positions=FAKE + 4), MISALIGNED),
    (dict(rope_off=8), INVALID), (dict(rope_dim=-16), INVALID), (dict(rope_off=4, rope_dim=16), UNSUPPORTED),
    (dict(rope_dim=24), UNSUPPORTED), (dict(rope_dim=12, interleaved=1), UNSUPPORTED), (dict(cos=None), INVALID),
    (dict(sin=None), INVALID), (dict(max_pos=0), INVALID), (dict(cos=FAKE + 4), MISALIGNED),
    (dict(positions=None, pos0=98), INVALID), (dict(positions=None, pos0=-1), INVALID),
    (dict(rope_off=2 ** 31 - 8), INVALID),
]


@pytest.mark.parametrize("edits,status", NORM_BAD)
def test_norm_rope_refusals(lib, edits, status):
    a = _norm(**edits)
    before = lib.dsa_launch_count()
    assert lib.dsa_norm_rope(ctypes.byref(a), FAKE, 0, 0, 0, FAKE, 256, None) == status
    assert lib.dsa_norm_rope_e4m3(ctypes.byref(a), FAKE, FAKE, 100, 1, FAKE, 256, None) == status
    assert lib.dsa_last_error() and lib.dsa_launch_count() == before


@pytest.mark.parametrize("edits,status", [
    (dict(B=1 << 16, n=1 << 13, H=16, d=64), UNSUPPORTED), (dict(B=1 << 16, n=1 << 13, H=4, d=512, rope_dim=64), UNSUPPORTED),
    (dict(positions=None, pos0=-1, rope_dim=0), INVALID),
])
def test_norm_rope_refuses_what_its_kernels_cannot_count(lib, edits, status):
    a = _norm(**edits)
    assert lib.dsa_norm_rope(ctypes.byref(a), FAKE, 0, 0, 0, FAKE, 256, None) == status


def test_norm_rope_output_refusals(lib):
    a = ctypes.byref(_norm())
    call = lambda out=FAKE, sb=0, st=0, sh=0, ws=FAKE, n=256: lib.dsa_norm_rope(a, out, sb, st, sh, ws, n, None)  # noqa: E731
    assert call(out=None) == INVALID and call(out=FAKE + 8) == MISALIGNED
    assert call(sb=-8) == INVALID and call(sh=56) == INVALID and call(st=260) == MISALIGNED
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE and call(ws=FAKE + 8) == MISALIGNED
    assert lib.dsa_norm_rope(None, FAKE, 0, 0, 0, FAKE, 256, None) == INVALID
    q = lambda a=a, codes=FAKE, scales=FAKE, cap=100, at=1: lib.dsa_norm_rope_e4m3(a, codes, scales, cap, at, FAKE, 256, None)  # noqa: E731
    assert q(codes=None) == INVALID and q(scales=None) == INVALID and q(cap=0) == INVALID and q(cap=2, at=0) == INVALID
    assert q(codes=FAKE + 4) == MISALIGNED and q(scales=FAKE + 2) == MISALIGNED
    assert q(a=ctypes.byref(_norm(H=17, d=1024))) == UNSUPPORTED
    assert q(a=ctypes.byref(_norm(H=257))) == UNSUPPORTED
    assert q(a=ctypes.byref(_norm(positions=None, pos0=40)), cap=42) == INVALID  # past the cache, not the tables


def test_calls_of_no_tokens_launch_nothing(lib):
    before = lib.dsa_launch_count()
    assert lib.dsa_norm_rope(ctypes.byref(_norm(n=0)), FAKE, 0, 0, 0, FAKE, 256, None) == OK
    assert lib.dsa_norm_rope_e4m3(ctypes.byref(_norm(n=0)), FAKE, FAKE, 100, 1, FAKE, 256, None) == OK
    c = _cache()
    assert lib.dsa_latent_append(ctypes.byref(_append(n=0)), ctypes.byref(c), FAKE, 256, None) == OK
    assert lib.dsa_latent_read(ctypes.byref(c), 2, 0, FAKE, 0, FAKE, FAKE, 256, None) == OK
    assert lib.dsa_launch_count() == before


def _cache(**kw):
    return _edit(dsa.LatentCache(n_pages=10, page_size=16, table_ld=4, codes=FAKE, scales=FAKE, rope=FAKE, block_table=FAKE), kw)


CACHE_BAD = [
    (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(table_ld=0), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(rope=None), INVALID), (dict(codes=FAKE + 8), MISALIGNED),
    (dict(rope=FAKE + 2), MISALIGNED), (dict(scales=FAKE + 2), MISALIGNED), (dict(block_table=FAKE + 1), MISALIGNED),
    (dict(block_table=None, n_pages=1), INVALID),
]


def _append(**kw):
    return _edit(dsa.LatentAppendArgs(B=2, n=3, x=FAKE, weight=FAKE, eps=1e-6, cos=FAKE, sin=FAKE, max_pos=100, positions=FAKE), kw)


def _attn(**kw):
    return _edit(dsa.LatentAttnArgs(B=2, T=3, S=60, H=64, scale=0.04, q=FAKE, cache=_cache(), idx_T=3), kw)


def _attend(lib, a, idx=FAKE, k=16, out=FAKE, lse=FAKE, ws=FAKE, n=256):
    return lib.dsa_latent_attn(a and ctypes.byref(a), idx, k, out, lse, ws, n, None)


@pytest.mark.parametrize("edits,status", CACHE_BAD)
def test_cache_refusals(lib, edits, status):
    c = _cache(**edits)
    before = lib.dsa_launch_count()
    assert lib.dsa_latent_append(ctypes.byref(_append()), ctypes.byref(c), FAKE, 256, None) == status
    assert lib.dsa_latent_read(ctypes.byref(c), 2, 3, FAKE, 0, FAKE, FAKE, 256, None) == status
    assert _attend(lib, _attn(cache=c)) == status
    assert lib.dsa_launch_count() == before


@pytest.mark.parametrize("edits,status", [
    (dict(B=0), INVALID), (dict(n=-1), INVALID), (dict(x=None), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID),
    (dict(max_pos=0), INVALID), (dict(eps=-1.0), INVALID), (dict(x_stride_t=568), INVALID), (dict(x_stride_b=-8), INVALID),
    (dict(x_stride_t=580), MISALIGNED), (dict(x=FAKE + 8), MISALIGNED), (dict(weight=FAKE + 4), MISALIGNED),
    (dict(cos=FAKE + 4), MISALIGNED), (dict(positions=FAKE + 4), MISALIGNED), (dict(positions=None, pos0=62), INVALID),
    (dict(positions=None, pos0=0, max_pos=2), INVALID), (dict(positions=None, pos0=-1), INVALID),
])
def test_append_refusals(lib, edits, status):
    before = lib.dsa_launch_count()
    assert lib.dsa_latent_append(ctypes.byref(_append(**edits)), ctypes.byref(_cache()), FAKE, 256, None) == status
    assert lib.dsa_launch_count() == before


def test_append_and_read_pointer_refusals(lib):
    c = ctypes.byref(_cache())
    assert lib.dsa_latent_append(None, c, FAKE, 256, None) == INVALID
    assert lib.dsa_latent_append(ctypes.byref(_append()), None, FAKE, 256, None) == INVALID
    assert lib.dsa_latent_append(ctypes.byref(_append()), c, FAKE, 100, None) == WORKSPACE
    read = lambda B=2, n=3, idx=FAKE, pos0=0, out=FAKE, ws=FAKE: lib.dsa_latent_read(c, B, n, idx, pos0, out, ws, 256, None)  # noqa: E731
    assert read(B=0) == INVALID and read(n=-1) == INVALID and read(out=None) == INVALID and read(out=FAKE + 8) == MISALIGNED
    assert read(idx=None, pos0=62) == INVALID and read(idx=None, pos0=-1) == INVALID and read(idx=FAKE + 2) == MISALIGNED
    assert read(ws=None) == WORKSPACE
    assert lib.dsa_latent_read(None, 2, 3, FAKE, 0, FAKE, FAKE, 256, None) == INVALID


@pytest.mark.parametrize("edits,status", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(S=0), INVALID), (dict(S=65), INVALID), (dict(H=0), UNSUPPORTED),
    (dict(H=129), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), MISALIGNED), (dict(q_stride_t=64 * 576 - 8), INVALID),
    (dict(q_stride_b=4), MISALIGNED), (dict(q_stride_b=-8), INVALID), (dict(idx_T=2), INVALID), (dict(idx_T=0), INVALID),
    (dict(flags=FAKE + 2), MISALIGNED), (dict(B=1 << 20, T=32, idx_T=32), UNSUPPORTED),
])
def test_latent_attn_refusals(lib, edits, status):
    before = lib.dsa_launch_count()
    assert _attend(lib, _attn(**edits)) == status
    assert lib.dsa_launch_count() == before


def test_latent_attn_call_refusals(lib):
    a = _attn()
    assert _attend(lib, None) == INVALID and _attend(lib, a, idx=None) == INVALID and _attend(lib, a, out=None) == INVALID
    assert _attend(lib, a, k=0) == UNSUPPORTED and _attend(lib, a, k=65537) == UNSUPPORTED
    assert _attend(lib, a, out=FAKE + 8) == MISALIGNED and _attend(lib, a, idx=FAKE + 2) == MISALIGNED
    assert _attend(lib, a, lse=FAKE + 1) == MISALIGNED
    assert _attend(lib, a, ws=None) == WORKSPACE and _attend(lib, a, n=255) == WORKSPACE and _attend(lib, a, ws=FAKE + 8) == MISALIGNED


def test_latent_attn_workspace_query(lib):
    size = lambda a, k: lib.dsa_latent_attn_workspace_size(a and ctypes.byref(a), k)  # noqa: E731
    assert size(None, 16) == 256 and size(_attn(H=0), 16) == 256 and size(_attn(), 0) == 256
    assert size(_attn(), 2048) >= 256


@pytest.mark.parametrize("device,index", [("cuda:1", 1), ("cuda:0", 0), ("cuda", 0), (None, 0)])
def test_read_device_flags_reads_the_named_device_on_its_own_stream(monkeypatch, device, index):
    """Device 0 is current; each device has its workspace, its flag word and its current stream."""
    current, reads = [0], []
    words = {(i, kind): FAKE + 4096 * i + 256 * kind for i in (0, 1) for kind in (0, 1)}
    bits = {words[i, 0]: 1 << i for i in (0, 1)} | {words[i, 1]: 4 << i for i in (0, 1)}

    class Memory:
        def __init__(self, i, kind):
            self.device, self._addr = torch.device("cuda", i), words[i, kind]

        def data_ptr(self):
            return self._addr

    class Library:
        def dsa_read_device_flags(self, ws, out, stream):
            addr = ctypes.cast(ws, ctypes.c_void_p).value
            out._obj.value = bits[addr]
            reads.append((addr, stream.value, current[0]))
            return 0

    @contextlib.contextmanager
    def on(dev):
        before, current[0] = current[0], dev.index
        yield
        current[0] = before

    def stream_of(dev=None):
        return types.SimpleNamespace(cuda_stream=1000 + (current[0] if dev is None else dev.index))

    def workspace(nbytes=256, device=None):
        i = None if device is None else torch.device(device).index
        return Memory(current[0] if i is None else i, 0)

    monkeypatch.setattr(dsa, "load_library", Library)
    monkeypatch.setattr(dsa, "workspace", workspace)
    monkeypatch.setattr(dsa, "_flags", {torch.device("cuda", i): Memory(i, 1) for i in (0, 1)})
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", stream_of)
    assert dsa.read_device_flags(device) == 5 << index
    assert sorted(reads) == [(words[index, kind], 1000 + index, index) for kind in (0, 1)]


# --- the 4-bit cache and attention over all rows ---------------------------------------------------

def _cache4(**kw):
    return _edit(dsa.Latent4Cache(n_pages=10, page_size=16, table_ld=4, codes=FAKE, groups=FAKE, scales=FAKE, rope=FAKE, block_table=FAKE), kw)


def _attn4(**kw):
    return _edit(dsa.Latent4AttnArgs(B=2, T=3, S=60, H=64, scale=0.04, q=FAKE, cache=_cache4(), idx_T=3), kw)


def _dense(lib, a, lens=FAKE, causal=1, out=FAKE, lse=FAKE, ws=FAKE, n=1 << 30):
    call = lib.dsa_latent4_attn_dense if isinstance(a, dsa.Latent4AttnArgs) else lib.dsa_latent_attn_dense
    return call(ctypes.byref(a), lens, causal, out, lse, ws, n, None)


def test_struct_layouts_of_the_4_bit_cache_match_header(tmp_path):
    lines, want = [], []
    for name, cls in (("dsa_latent4_cache", dsa.Latent4Cache), ("dsa_latent4_attn_args", dsa.Latent4AttnArgs)):
        lines.append(f'printf("%zu ", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void){' + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()] == want


def test_packed_images_are_the_structs():
    """The binding packs whole structs: every field where ctypes has it."""
    image = dsa._CACHE4.pack(1, 2, 3, 4, 5, 6, 7, 8)
    c = dsa.Latent4Cache.from_buffer_copy(image)
    assert [getattr(c, f) for f, _ in c._fields_] == [1, 2, 3, 4, 5, 6, 7, 8]
    a = dsa.Latent4AttnArgs.from_buffer_copy(dsa._ATTN_HEAD.pack(11, 12, 13, 14, 0.5, 15, 16, 17) + image + dsa._ATTN_TAIL.pack(18, 19))
    assert (a.B, a.T, a.S, a.H, a.scale, a.q, a.q_stride_b, a.q_stride_t, a.cache.block_table, a.idx_T, a.flags) == (11, 12, 13, 14, 0.5, 15, 16, 17, 8, 18, 19)
    image = dsa._CACHE.pack(1, 2, 3, 4, 5, 6, 7)
    a = dsa.LatentAttnArgs.from_buffer_copy(dsa._ATTN_HEAD.pack(11, 12, 13, 14, 0.5, 15, 16, 17) + image + dsa._ATTN_TAIL.pack(18, 19))
    assert (a.H, a.cache.n_pages, a.cache.block_table, a.idx_T, a.flags) == (14, 1, 7, 18, 19)
    p = dsa.LatentAppendArgs.from_buffer_copy(dsa._APPEND.pack(1, 2, 3, 4, 5, 6, 0.25, 7, 8, 9, 10, 11, 12))
    assert [getattr(p, f) for f, _ in p._fields_] == [1, 2, 3, 4, 5, 6, 0.25, 7, 8, 9, 10, 11, 12]


@pytest.mark.parametrize("edits,status", CACHE_BAD + [(dict(groups=None), INVALID)])
def test_4_bit_cache_refusals(lib, edits, status):
    c = _cache4(**edits)
    before = lib.dsa_launch_count()
    assert lib.dsa_latent4_append(ctypes.byref(_append()), ctypes.byref(c), FAKE, 256, None) == status
    assert lib.dsa_latent4_read(ctypes.byref(c), 2, 3, FAKE, 0, FAKE, FAKE, 256, None) == status
    assert lib.dsa_latent4_unpack(ctypes.byref(c), 2, 3, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 256, None) == status
    a = _attn4(cache=c)
    assert lib.dsa_latent4_attn(ctypes.byref(a), FAKE, 16, FAKE, FAKE, FAKE, 256, None) == status
    assert _dense(lib, a) == status
    assert lib.dsa_launch_count() == before


def test_4_bit_call_refusals(lib):
    c = ctypes.byref(_cache4())
    before = lib.dsa_launch_count()
    assert lib.dsa_latent4_append(ctypes.byref(_append(x_stride_t=568)), c, FAKE, 256, None) == INVALID
    assert lib.dsa_latent4_append(ctypes.byref(_append(positions=None, pos0=62)), c, FAKE, 256, None) == INVALID
    assert lib.dsa_latent4_append(ctypes.byref(_append()), None, FAKE, 256, None) == INVALID
    assert lib.dsa_latent4_append(None, c, FAKE, 256, None) == INVALID
    assert lib.dsa_latent4_append(ctypes.byref(_append()), c, FAKE, 255, None) == WORKSPACE
    assert lib.dsa_latent4_append(ctypes.byref(_append(n=0)), c, FAKE, 256, None) == OK
    unpack = lambda B=2, n=3, idx=FAKE, pos0=0, codes=FAKE, scales=FAKE, rope=FAKE, ws=FAKE: lib.dsa_latent4_unpack(c, B, n, idx, pos0, codes, scales, rope, ws, 256, None)  # noqa: E731
    assert unpack(codes=None) == INVALID and unpack(scales=None) == INVALID and unpack(rope=None) == INVALID
    assert unpack(codes=FAKE + 8) == MISALIGNED and unpack(rope=FAKE + 8) == MISALIGNED and unpack(scales=FAKE + 2) == MISALIGNED
    assert unpack(idx=FAKE + 2) == MISALIGNED and unpack(idx=None, pos0=62) == INVALID and unpack(idx=None, pos0=-1) == INVALID
    assert unpack(B=0) == INVALID and unpack(n=-1) == INVALID and unpack(ws=None) == WORKSPACE and unpack(n=0) == OK
    assert lib.dsa_latent4_read(c, 2, 3, FAKE, 0, None, FAKE, 256, None) == INVALID
    assert lib.dsa_latent4_read(c, 2, 0, FAKE, 0, FAKE, FAKE, 256, None) == OK
    a = _attn4()
    call = lambda a=a, idx=FAKE, k=16, out=FAKE: lib.dsa_latent4_attn(a and ctypes.byref(a), idx, k, out, FAKE, FAKE, 256, None)  # noqa: E731
    assert call(a=None) == INVALID and call(idx=None) == INVALID and call(out=None) == INVALID and call(k=0) == UNSUPPORTED
    assert call(a=_attn4(idx_T=2)) == INVALID and call(a=_attn4(H=129)) == UNSUPPORTED and call(a=_attn4(S=65)) == INVALID
    assert lib.dsa_launch_count() == before


@pytest.mark.parametrize("edits,status", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(S=0), INVALID), (dict(S=65), INVALID), (dict(H=0), UNSUPPORTED),
    (dict(H=129), UNSUPPORTED), (dict(B=1 << 13, T=1 << 13), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), MISALIGNED), (dict(q_stride_t=64 * 576 - 8), INVALID), (dict(q_stride_b=-8), INVALID),
    (dict(q_stride_b=3 * 64 * 576 + 4), MISALIGNED), (dict(flags=FAKE + 2), MISALIGNED),
])
def test_dense_attention_refusals(lib, edits, status):
    before = lib.dsa_launch_count()
    assert _dense(lib, _attn4(**edits)) == status
    assert _dense(lib, _attn(**edits)) == status
    assert lib.dsa_last_error() and lib.dsa_launch_count() == before


def test_dense_attention_call_refusals_and_workspace(lib):
    before = lib.dsa_launch_count()
    for a in (_attn4(), _attn(), _attn4(idx_T=0)):  # (idx_T is not read)
        assert _dense(lib, a, lens=None) == INVALID and _dense(lib, a, out=None) == INVALID
        assert _dense(lib, a, lens=FAKE + 2) == MISALIGNED and _dense(lib, a, out=FAKE + 8) == MISALIGNED and _dense(lib, a, lse=FAKE + 2) == MISALIGNED
        assert _dense(lib, a, ws=None) == WORKSPACE and _dense(lib, a, ws=FAKE + 8) == MISALIGNED
        need = lib.dsa_latent_attn_dense_workspace_size(2, 3, 60, 64)
        assert _dense(lib, a, n=need - 1) == WORKSPACE and need > 256
    size = lib.dsa_latent_attn_dense_workspace_size
    assert size(0, 1, 1, 1) == size(1, 1, 1, 129) == 256  # calls that are refused
    assert size(1, 1, 2 ** 31 - 1, 64) >= size(1, 1, 64, 64) > 256
    assert lib.dsa_launch_count() == before


def test_a_refused_kernel_image_is_told_with_its_own_registers(tmp_path):
    """The entry points over launchers that refuse their kernels: the message names what that cache's kernels are built with."""
    src = tmp_path / "refused.cu"
    src.write_text(r'''
#include "dsa_latent_api.cu"
namespace dsa {
dsa_status record_error(dsa_status s, const char* msg) { return printf("%s\n", msg), s; }
int norm_rope_units(int) { return 0; }
cudaError_t launch_norm_rope(const NormRopeLaunch&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_latent_append(const LatentAppendLaunch&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_latent_read(const LatentReadLaunch&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_latent_attn(const LatentAttnLaunch&, cudaStream_t) { return cudaErrorInvalidKernelImage; }
cudaError_t launch_latent4_attn(const LatentAttnLaunch&, cudaStream_t) { return cudaErrorInvalidKernelImage; }
cudaError_t launch_latent_dense(LatentAttnLaunch, void*, cudaStream_t) { return cudaErrorInvalidKernelImage; }
size_t latent_dense_scratch(LatentAttnLaunch) { return 0; }
}  // namespace dsa
int main() {
  static_assert(dsa::kLatentAttnRegs != dsa::kLatent4AttnRegs);
  void* m = reinterpret_cast<void*>(1 << 20);
  int32_t* i = static_cast<int32_t*>(m);
  dsa_latent_attn_args a{1, 1, 4, 64, 0.5f, m, 0, 0, {1, 4, 0, static_cast<uint8_t*>(m), static_cast<float*>(m), m, nullptr}, 1, nullptr};
  dsa_latent4_attn_args b{1, 1, 4, 64, 0.5f, m, 0, 0, {1, 4, 0, static_cast<uint8_t*>(m), static_cast<uint8_t*>(m), static_cast<float*>(m), m, nullptr}, 1, nullptr};
  dsa_latent_attn(&a, i, 1, m, nullptr, m, 1 << 20, nullptr);
  dsa_latent_attn_dense(&a, i, 1, m, nullptr, m, 1 << 20, nullptr);
  dsa_latent4_attn(&b, i, 1, m, nullptr, m, 1 << 20, nullptr);
  dsa_latent4_attn_dense(&b, i, 1, m, nullptr, m, 1 << 20, nullptr);
  printf("%d %d\n", dsa::kLatentAttnRegs, dsa::kLatent4AttnRegs);
}
''')
    exe = tmp_path / "refused"
    subprocess.run([dsa_build.NVCC, *dsa_build.ARCH, *dsa_build.FLAGS, "-cudart", "static", str(src), "-o", str(exe)], check=True)
    *told, regs = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    eight, four = regs.split()
    assert len(told) == 4
    assert all(f" {eight} registers" in m for m in told[:2]) and all(f" {four} registers" in m for m in told[2:]), told
