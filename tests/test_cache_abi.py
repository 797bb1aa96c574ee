"""CPU checks of the cache calls: what the host refuses, before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import linear_attention_layer_gb300 as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
OUT = ctypes.c_void_p(0x20000)
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return kda.load()


@pytest.mark.parametrize("name,struct", [("kda_cache_t", kda.KdaCache),
                                         ("kda_attention_t", kda.KdaAttention)])
def test_struct_layout_matches_header(tmp_path, name, struct):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f[0] for f in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"kda.h\"\n"
                   f"int main(void) {{\n  printf(\"%zu\\n\", sizeof({name}));\n" +
                   "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) +
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def _cache(**over):
    p = dict(pages=0x10000, num_pages=4, page_size=32, num_kv_heads=2, head_dim=128)
    p.update(over)
    c = kda.KdaCache()
    for k, v in p.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID),
              (dict(page_size=24), INVALID), (dict(page_size=8192), INVALID),
              (dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=4097), UNSUPPORTED),
              (dict(num_pages=1 << 26), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
              (dict(head_dim=0), UNSUPPORTED), (dict(pages=None), INVALID),
              (dict(pages=0x10008), INVALID), (dict(k_exponent=0x10002), INVALID)]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_cache_refused(lib, over, status):
    c = ctypes.byref(_cache(**over))
    assert lib.kda_cache_append(c, 1, 3, FAKE, FAKE, None, FAKE, None) == status
    assert lib.kda_cache_read(c, 1, 3, FAKE, FAKE, OUT, None) == status
    n = ctypes.c_size_t(0)
    d = _desc()
    assert lib.kda_cache_attention_workspace_size(c, ctypes.byref(d), ctypes.byref(n)) == status
    assert lib.kda_cache_attention(c, ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, OUT, None,
                                   None) == status


@pytest.mark.parametrize("args", [
    (7, 3, FAKE, FAKE, None, FAKE), (1, -1, FAKE, FAKE, None, FAKE),
    (1, 3, None, FAKE, None, FAKE), (1, 3, FAKE, None, None, FAKE),
    (1, 3, FAKE, FAKE, None, None), (1, 3, ctypes.c_void_p(0x10001), FAKE, None, FAKE),
    (0, 3, FAKE, ctypes.c_void_p(0x10002), None, FAKE),
    (1, 3, FAKE, FAKE, None, ctypes.c_void_p(0x10004))])
def test_append_refuses(lib, args):
    assert lib.kda_cache_append(ctypes.byref(_cache()), *args, None) == INVALID


def test_append_refuses_long_strides(lib):
    strides = (ctypes.c_int64 * 4)(256, 128, 1 << 31, 128)
    assert lib.kda_cache_append(ctypes.byref(_cache()), 1, 3, FAKE, FAKE, strides, FAKE,
                                None) == UNSUPPORTED


@pytest.mark.parametrize("args", [
    (7, 3, FAKE, FAKE, OUT), (1, -1, FAKE, FAKE, OUT), (1, 3, None, FAKE, OUT),
    (1, 3, FAKE, None, OUT), (1, 3, FAKE, OUT, None), (1, 3, FAKE, OUT, OUT),
    (1, 3, FAKE, ctypes.c_void_p(0x10008), OUT)])
def test_read_refuses(lib, args):
    assert lib.kda_cache_read(ctypes.byref(_cache()), *args, None) == INVALID


def test_no_tokens_is_no_work(lib):
    c = ctypes.byref(_cache())
    assert lib.kda_cache_append(c, 1, 0, None, None, None, None, None) == 0
    assert lib.kda_cache_read(c, 1, 0, None, None, None, None) == 0
    for over in (dict(num_seqs=0), dict(total_tokens=0)):
        assert lib.kda_cache_attention(c, ctypes.byref(_desc(**over)), None, None, None, None,
                                       None, None, None) == 0


def _tables(lib, **over):
    p = dict(page=16, seqs=2, blocks=4, tokens=8, ring=16, held=0x1000, seq=0x1000, new=0x3000,
             table=0x4000, free=0x5000, span=0x6000, span_out=0x6000, kv=0x1000, cu=0x8000,
             slots=0x9000)
    p.update(over)
    v = list(p.values())
    return lib.kda_cache_tables(*v[:5], *[ctypes.c_void_p(x) for x in v[5:]], None)


@pytest.mark.parametrize("over", [
    dict(page=0), dict(page=17), dict(page=8192), dict(seqs=-1), dict(blocks=-1), dict(tokens=-1),
    dict(ring=0), dict(held=None), dict(seq=None), dict(new=None), dict(table=None),
    dict(free=None), dict(span=None), dict(span_out=None), dict(kv=None), dict(cu=None),
    dict(slots=None), dict(kv=0x3000), dict(cu=0x1000), dict(slots=0x3000), dict(table=0x1000),
    dict(kv=0x8000)])
def test_tables_refuses(lib, over):
    assert _tables(lib, **over) == INVALID


def test_tables_too_large(lib):
    assert _tables(lib, seqs=1 << 16, blocks=1 << 15) == UNSUPPORTED


def _desc(**over):
    p = dict(num_seqs=2, total_tokens=3, num_heads=8, max_new=2, max_blocks=4, io_dtype=1,
             scale=0.1)
    p.update(over)
    d = kda.KdaAttention()
    for k, v in p.items():
        if k == "q_strides":
            d.q_strides[0], d.q_strides[1] = v
        else:
            setattr(d, k, v)
    return d


@pytest.mark.parametrize("over", [
    dict(num_seqs=-1), dict(total_tokens=-1), dict(num_heads=0), dict(num_heads=7),
    dict(max_new=0), dict(max_blocks=-1), dict(io_dtype=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_strides=(0, 128)), dict(q_strides=(128, 0))])
def test_attention_refuses_descriptor(lib, over):
    d = _desc(**over)
    c = ctypes.byref(_cache())
    n = ctypes.c_size_t(0)
    assert lib.kda_cache_attention_workspace_size(c, ctypes.byref(d), ctypes.byref(n)) == INVALID
    assert lib.kda_cache_attention(c, ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, OUT, None,
                                   None) == INVALID


def test_attention_too_many_rows(lib):
    d, n = _desc(total_tokens=1 << 30), ctypes.c_size_t(0)
    assert lib.kda_cache_attention_workspace_size(ctypes.byref(_cache()), ctypes.byref(d),
                                                  ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("args", [
    (None, FAKE, FAKE, FAKE, OUT, None), (FAKE, None, FAKE, FAKE, OUT, None),
    (FAKE, FAKE, None, FAKE, OUT, None), (FAKE, FAKE, FAKE, None, OUT, None),
    (FAKE, FAKE, FAKE, FAKE, None, None), (FAKE, FAKE, FAKE, FAKE, FAKE, None),
    (ctypes.c_void_p(0x10001), FAKE, FAKE, FAKE, OUT, None),
    (FAKE, FAKE, FAKE, FAKE, ctypes.c_void_p(0x20008), None),
    (FAKE, FAKE, FAKE, FAKE, OUT, ctypes.c_void_p(0x30002))])
def test_attention_refuses_pointers(lib, args):
    assert lib.kda_cache_attention(ctypes.byref(_cache()), ctypes.byref(_desc()), *args,
                                   None) == INVALID


def test_workspace_size_needs_a_place(lib):
    assert lib.kda_cache_attention_workspace_size(ctypes.byref(_cache()), ctypes.byref(_desc()),
                                                  None) == INVALID


def test_binding_refuses():
    with pytest.raises(ValueError):
        kda.cache_empty(4, 24, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        kda.cache_empty(4, 32, 2, 96, device="cpu")
    cache = kda.cache_empty(4, 32, 2, 128, device="cpu")
    assert cache.shape == (4, 2, 2, 18 * 128)
    x, slots = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # not on a GPU
        kda.cache_append(x, x, slots, cache)
    with pytest.raises(ValueError):
        kda.cache_read(slots, cache)
    with pytest.raises(ValueError):
        kda.cache_attention(x, cache, torch.zeros(1, 1, dtype=torch.int32),
                            torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                            max_new=1)


@pytest.mark.parametrize("shape", [(1, 1, 64), (5, 1, 64), (1, 4, 64)])
def test_binding_refuses_broadcast_queries(lib, shape):
    """Stride 0 over more than one token or head: two such would be taken for packed, and read
    past the end.  Refused before anything else is looked at."""
    q = torch.zeros(shape).expand(5, 4, 64)
    cache = kda.cache_empty(1, 16, 2, 64, device="cpu")
    lens, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="broadcast"):
        kda.cache_attention(q, cache, lens[None], lens, cu, max_new=1)


@pytest.mark.parametrize("name,address", [
    ("held", 0x1002), ("seq", 0x1002), ("new", 0x3001), ("table", 0x4002), ("free", 0x5002),
    ("span", 0x6004), ("span_out", 0x6004), ("kv", 0x7002), ("cu", 0x8002), ("slots", 0x9004)])
def test_tables_refuses_misaligned(lib, name, address):
    assert _tables(lib, **{name: address}) == INVALID


@pytest.mark.parametrize("which", [1, 2, 3])
def test_attention_refuses_misaligned_tables(lib, which):
    args = [FAKE, FAKE, FAKE, FAKE, OUT, None]
    args[which] = ctypes.c_void_p(0x10002)
    room = _desc(workspace=1 << 30, workspace_bytes=1 << 40)
    assert lib.kda_cache_attention(ctypes.byref(_cache()), ctypes.byref(room), *args,
                                   None) == INVALID


def test_binding_refuses_a_stream_of_another_device(lib):
    """The calls run on the current stream of their tensors' device: a stream of another one
    would be passed over without a word."""
    class Elsewhere:
        device = torch.device("cuda", 1)

    cache = kda.cache_empty(1, 16, 2, 64, device="cpu")
    lens, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    slots, x = torch.zeros(1, dtype=torch.int64), torch.zeros(1, 2, 64)
    for call in (lambda s: kda.cache_tables(lens, lens, lens, lens[None], lens, slots,
                                            page_size=16, max_tokens=1, stream=s),
                 lambda s: kda.cache_append(x, x, slots, cache, stream=s),
                 lambda s: kda.cache_read(slots, cache, stream=s),
                 lambda s: kda.cache_attention(x, cache, lens[None], lens, cu, max_new=1,
                                               stream=s)):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call(Elsewhere())
