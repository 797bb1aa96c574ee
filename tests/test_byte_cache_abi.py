"""CPU checks of the 8-bit cache's calls and those on shared pages: what the host refuses,
before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import linear_attention_layer_gb300 as kda
from tests.test_cache_abi import FAKE, INVALID, OUT, ROOT, UNSUPPORTED, _desc, lib  # noqa: F401


def test_struct_layout_matches_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f[0] for f in kda.KdaByteCache._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"kda.h\"\n"
                   "int main(void) {\n  printf(\"%zu\\n\", sizeof(kda_byte_cache_t));\n" +
                   "".join(f'  printf("%zu\\n", offsetof(kda_byte_cache_t, {f}));\n' for f in fields) +
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = [getattr(kda.KdaByteCache, f).offset for f in fields]
    assert got == [ctypes.sizeof(kda.KdaByteCache)] + want


def _cache(**over):
    p = dict(pages=0x10000, num_pages=4, page_size=32, num_kv_heads=2, head_dim=128)
    p.update(over)
    return ctypes.byref(kda.KdaByteCache(**p))


@pytest.mark.parametrize("over,status", [
    (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), INVALID),
    (dict(page_size=8192), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_kv_heads=4097), UNSUPPORTED), (dict(num_pages=1 << 26), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(pages=None), INVALID),
    (dict(pages=0x10008), INVALID)])
def test_bad_cache_refused(lib, over, status):  # noqa: F811
    c = _cache(**over)
    assert lib.kda_byte_cache_append(c, 1, 3, FAKE, FAKE, None, FAKE, None) == status
    assert lib.kda_byte_cache_read(c, 1, 3, FAKE, FAKE, OUT, None) == status
    n, d = ctypes.c_size_t(0), ctypes.byref(_desc())
    assert lib.kda_byte_cache_attention_workspace_size(c, d, ctypes.byref(n)) == status
    assert lib.kda_byte_cache_attention(c, d, FAKE, FAKE, FAKE, FAKE, OUT, None, None) == status


@pytest.mark.parametrize("args", [
    (7, 3, FAKE, FAKE, None, FAKE), (1, -1, FAKE, FAKE, None, FAKE),
    (1, 3, None, FAKE, None, FAKE), (1, 3, FAKE, None, None, FAKE),
    (1, 3, FAKE, FAKE, None, None), (1, 3, ctypes.c_void_p(0x10001), FAKE, None, FAKE),
    (0, 3, FAKE, ctypes.c_void_p(0x10002), None, FAKE),
    (1, 3, FAKE, FAKE, None, ctypes.c_void_p(0x10004))])
def test_append_refuses(lib, args):  # noqa: F811
    assert lib.kda_byte_cache_append(_cache(), *args, None) == INVALID


def test_append_refuses_long_strides(lib):  # noqa: F811
    strides = (ctypes.c_int64 * 4)(256, 128, 1 << 31, 128)
    assert lib.kda_byte_cache_append(_cache(), 1, 3, FAKE, FAKE, strides, FAKE, None) == UNSUPPORTED


@pytest.mark.parametrize("args", [
    (7, 3, FAKE, FAKE, OUT), (1, -1, FAKE, FAKE, OUT), (1, 3, None, FAKE, OUT),
    (1, 3, FAKE, None, OUT), (1, 3, FAKE, OUT, None), (1, 3, FAKE, OUT, OUT),
    (1, 3, FAKE, ctypes.c_void_p(0x10008), OUT)])
def test_read_refuses(lib, args):  # noqa: F811
    assert lib.kda_byte_cache_read(_cache(), *args, None) == INVALID


@pytest.mark.parametrize("over", [
    dict(num_seqs=-1), dict(total_tokens=-1), dict(num_heads=0), dict(num_heads=7),
    dict(max_new=0), dict(max_blocks=-1), dict(io_dtype=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_strides=(0, 128)), dict(q_strides=(128, 0))])
def test_attention_refuses_descriptor(lib, over):  # noqa: F811
    d, n = ctypes.byref(_desc(**over)), ctypes.c_size_t(0)
    assert lib.kda_byte_cache_attention_workspace_size(_cache(), d, ctypes.byref(n)) == INVALID
    assert lib.kda_byte_cache_attention(_cache(), d, FAKE, FAKE, FAKE, FAKE, OUT, None, None) == INVALID


@pytest.mark.parametrize("args", [
    (None, FAKE, FAKE, FAKE, OUT, None), (FAKE, None, FAKE, FAKE, OUT, None),
    (FAKE, FAKE, None, FAKE, OUT, None), (FAKE, FAKE, FAKE, None, OUT, None),
    (FAKE, FAKE, FAKE, FAKE, None, None), (FAKE, FAKE, FAKE, FAKE, FAKE, None),
    (ctypes.c_void_p(0x10001), FAKE, FAKE, FAKE, OUT, None),
    (FAKE, FAKE, FAKE, FAKE, ctypes.c_void_p(0x20008), None),
    (FAKE, ctypes.c_void_p(0x10002), FAKE, FAKE, OUT, None),
    (FAKE, FAKE, ctypes.c_void_p(0x10002), FAKE, OUT, None),
    (FAKE, FAKE, FAKE, ctypes.c_void_p(0x10002), OUT, None),
    (FAKE, FAKE, FAKE, FAKE, OUT, ctypes.c_void_p(0x30002))])
def test_attention_refuses_pointers(lib, args):  # noqa: F811
    room = ctypes.byref(_desc(workspace=1 << 30, workspace_bytes=1 << 40))
    assert lib.kda_byte_cache_attention(_cache(), room, *args, None) == INVALID


def test_attention_refuses_too_many_rows_and_too_little_room(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.kda_byte_cache_attention_workspace_size(
        _cache(), ctypes.byref(_desc(total_tokens=1 << 30)), ctypes.byref(n)) == UNSUPPORTED
    assert lib.kda_byte_cache_attention_workspace_size(_cache(), ctypes.byref(_desc()), None) == INVALID
    for over in (dict(workspace=None), dict(workspace_bytes=1), dict(workspace=(1 << 30) + 16)):
        d = dict(workspace=1 << 30, workspace_bytes=1 << 40)
        d.update(over)
        assert lib.kda_byte_cache_attention(_cache(), ctypes.byref(_desc(**d)), FAKE, FAKE, FAKE, FAKE,
                                        OUT, None, None) == INVALID


def test_no_work(lib):  # noqa: F811
    c = _cache()
    assert lib.kda_byte_cache_append(c, 1, 0, None, None, None, None, None) == 0
    assert lib.kda_byte_cache_read(c, 1, 0, None, None, None, None) == 0
    for over in (dict(num_seqs=0), dict(total_tokens=0)):
        assert lib.kda_byte_cache_attention(c, ctypes.byref(_desc(**over)), None, None, None, None,
                                        None, None, None) == 0


def _call(f, p, sized):
    v = [x if i < sized or i == len(p) - 1 else ctypes.c_void_p(x) for i, x in enumerate(p.values())]
    return f(*v, None)


FORK = dict(page=16, pages=16, old=2, seqs=3, blocks=4, ring=16, held=0x1000, table=0x2000,
            parents=0x3000, keep=0x4000, free=0x5000, span=0x6000, span_out=0x6000, kv=0x1000,
            out=0x7000, copies=0x8000, ws=0x10000, bytes=1 << 30)


@pytest.mark.parametrize("over", [
    dict(page=0), dict(page=17), dict(page=8192), dict(pages=-1), dict(old=-1), dict(seqs=-1),
    dict(blocks=-1), dict(ring=0), dict(ring=15), dict(held=None), dict(table=None),
    dict(parents=None), dict(keep=None), dict(free=None), dict(span=None), dict(span_out=None),
    dict(kv=None), dict(out=None), dict(copies=None), dict(ws=None), dict(ws=0x10010),
    dict(bytes=8), dict(out=0x2000), dict(copies=0x4000), dict(free=0x2000), dict(out=0x5000),
    dict(copies=0x7000), dict(kv=0x2000), dict(kv=0x7000), dict(held=0x1002), dict(span=0x6004),
    dict(copies=0x8002)])
def test_fork_refuses(lib, over):  # noqa: F811
    assert _call(lib.kda_cache_fork, {**FORK, **over}, 6) == INVALID


def test_fork_too_large(lib):  # noqa: F811
    for over in (dict(seqs=1 << 16, blocks=1 << 15), dict(old=1 << 16, blocks=1 << 15),
                 dict(pages=1 << 27, ring=1 << 27)):
        assert _call(lib.kda_cache_fork, {**FORK, **over}, 6) == UNSUPPORTED


COMPACT = dict(page=16, pages=16, seqs=3, blocks=4, ring=16, held=0x1000, table=0x2000, out=0x2000,
               copies=0x3000, free=0x4000, span=0x5000, ws=0x10000, bytes=1 << 30)


@pytest.mark.parametrize("over", [
    dict(page=0), dict(page=17), dict(pages=-1), dict(seqs=-1), dict(blocks=-1), dict(ring=0),
    dict(ring=15), dict(held=None), dict(table=None), dict(out=None), dict(copies=None),
    dict(free=None), dict(span=None), dict(ws=None), dict(ws=0x10010), dict(bytes=8),
    dict(copies=0x2000), dict(free=0x1000), dict(copies=0x4000), dict(out=0x1000),
    dict(held=0x1002), dict(span=0x5004), dict(span=0x3000)])
def test_compact_refuses(lib, over):  # noqa: F811
    assert _call(lib.kda_cache_compact, {**COMPACT, **over}, 5) == INVALID


def test_compact_too_large(lib):  # noqa: F811
    for over in (dict(seqs=1 << 16, blocks=1 << 15), dict(pages=1 << 27, ring=1 << 27)):
        assert _call(lib.kda_cache_compact, {**COMPACT, **over}, 5) == UNSUPPORTED


def test_copy_refuses(lib):  # noqa: F811
    two = (ctypes.c_void_p * 2)(0x10000, 0x20000)
    odd = (ctypes.c_void_p * 2)(0x10000, 0x20008)
    none = (ctypes.c_void_p * 2)(0x10000, None)
    good = [2, two, 4, 2, 32, 2064, 3, FAKE]
    for at, bad, status in [(0, -1, INVALID), (1, odd, INVALID), (1, none, INVALID),
                            (1, None, INVALID), (2, -1, INVALID), (3, 0, INVALID),
                            (4, 24, INVALID), (5, 0, INVALID), (5, 2056, INVALID),
                            (6, -1, INVALID), (7, None, INVALID), (3, 4097, UNSUPPORTED),
                            (7, ctypes.c_void_p(0x10002), INVALID), (5, 1 << 17, UNSUPPORTED),
                            (2, 1 << 27, UNSUPPORTED)]:
        args = list(good)
        args[at] = bad
        assert lib.kda_cache_copy(*args, None) == status, (at, bad)
    # a page of more than 2^31 bytes
    assert lib.kda_cache_copy(2, two, 4, 4096, 4096, 4112, 3, FAKE, None) == UNSUPPORTED
    assert lib.kda_cache_copy(0, None, 4, 2, 32, 2064, 3, FAKE, None) == 0
    assert lib.kda_cache_copy(2, two, 4, 2, 32, 2064, 0, None, None) == 0


def test_workspace_sizes(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.kda_cache_fork_workspace_size(-1, 1, ctypes.byref(n)) == INVALID
    assert lib.kda_cache_fork_workspace_size(1, -1, ctypes.byref(n)) == INVALID
    assert lib.kda_cache_fork_workspace_size(1, 1, None) == INVALID
    assert lib.kda_cache_compact_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert lib.kda_cache_compact_workspace_size(1, None) == INVALID
    assert kda.cache_fork_workspace_size(1000, 10) >= 3 * 128 + 4000 + 80
    assert kda.cache_compact_workspace_size(1000) >= 2 * 128


def test_binding_refuses():
    with pytest.raises(ValueError):
        kda.byte_cache_empty(4, 24, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        kda.byte_cache_empty(4, 32, 2, 96, device="cpu")
    cache = kda.byte_cache_empty(4, 32, 2, 128, device="cpu")
    assert cache.shape == (4, 2, 2, 32 * 128 + 16)
    x, slots = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    lens, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.byte_cache_append(x, x, slots, cache),
                 lambda: kda.byte_cache_read(slots, cache),
                 lambda: kda.byte_cache_attention(x, cache, lens[None], lens, cu, max_new=1),
                 lambda: kda.cache_fork(lens, lens[None], lens, lens, lens, slots[:2],
                                        page_size=16, num_pages=1),
                 lambda: kda.cache_compact(lens, lens[None], lens, page_size=16, num_pages=1),
                 lambda: kda.cache_copy(cache, torch.zeros(1, 3, dtype=torch.int32)),
                 lambda: kda.byte_cache_attention(x, cache, lens[None], lens, cu, max_new=1,
                                              workspace="none")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("shape", [(1, 1, 64), (5, 1, 64), (1, 4, 64)])
def test_binding_refuses_broadcast_queries(lib, shape):  # noqa: F811
    q = torch.zeros(shape).expand(5, 4, 64)
    cache = kda.byte_cache_empty(1, 16, 2, 64, device="cpu")
    lens, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="broadcast"):
        kda.byte_cache_attention(q, cache, lens[None], lens, cu, max_new=1)


def test_binding_refuses_a_stream_of_another_device(lib):  # noqa: F811
    class Elsewhere:
        device = torch.device("cuda", 1)

    cache = kda.byte_cache_empty(1, 16, 2, 64, device="cpu")
    lens, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    slots, x = torch.zeros(1, dtype=torch.int64), torch.zeros(1, 2, 64)
    for call in (lambda s: kda.byte_cache_append(x, x, slots, cache, stream=s),
                 lambda s: kda.byte_cache_read(slots, cache, stream=s),
                 lambda s: kda.byte_cache_attention(x, cache, lens[None], lens, cu, max_new=1,
                                                stream=s),
                 lambda s: kda.cache_fork(lens, lens[None], lens, lens, lens, slots, page_size=16,
                                          num_pages=1, stream=s),
                 lambda s: kda.cache_compact(lens, lens[None], lens, page_size=16, num_pages=1,
                                             stream=s),
                 lambda s: kda.cache_copy(cache, lens, stream=s)):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call(Elsewhere())
