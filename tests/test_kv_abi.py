"""Host-side checks of the paged cache's entry points that need no GPU: struct layouts, the arguments each call
refuses before any launch, page sizes, and the Python wrappers' refusals."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session")
def lib():
    from tiled_exact_attention_gb300 import build as b

    b.build()
    from tiled_exact_attention_gb300 import _lib

    return _lib.load()


def test_struct_layouts(tmp_path):
    from tiled_exact_attention_gb300._lib import KvAppendArgs, KvcacheInt4Args, KvGatherInt4Args

    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    mirrors = {"fa_kv_append_args": KvAppendArgs, "fa_kv_gather_int4_args": KvGatherInt4Args,
               "fa_kvcache_int4_args": KvcacheInt4Args}
    lines = []
    for c, py in mirrors.items():
        lines.append(f'printf("{c} size %zu 0\\n", sizeof({c}));')
        lines += [f'printf("{c} {n} %zu %zu\\n", offsetof({c}, {n}), sizeof((({c}*)0)->{n}));' for n, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fa.h"\nint main(void) {\n' + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    for ln in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.splitlines():
        struct, name, a, b = ln.split()
        if name == "size":
            assert ctypes.sizeof(mirrors[struct]) == int(a), struct
        else:
            f = getattr(mirrors[struct], name)
            assert (f.offset, f.size) == (int(a), int(b)), (struct, name)


def test_packers_match_the_mirrors():
    """The packers put every value where the ctypes mirrors (checked against the header) have it."""
    import ctypes as ct

    from tiled_exact_attention_gb300 import _lib

    for packer, mirror in ((_lib.KV_APPEND, _lib.KvAppendArgs), (_lib.KV_GATHER_INT4, _lib.KvGatherInt4Args),
                           (_lib.KVCACHE_INT4, _lib.KvcacheInt4Args)):
        flat = sum(getattr(t, "_length_", 1) for _, t in mirror._fields_)
        raw = packer.pack(*range(1, flat + 1))
        assert len(raw) == ct.sizeof(mirror)
        got, n = mirror.from_buffer_copy(raw), 0
        for name, t in mirror._fields_:
            value = getattr(got, name)
            for x in (list(value) if hasattr(t, "_length_") else [value]):
                n += 1
                assert x == n, (mirror.__name__, name)


def _append_args(**kw):
    from tiled_exact_attention_gb300._lib import KvAppendArgs

    a = KvAppendArgs()
    a.dtype, a.b, a.total, a.hq, a.hkv, a.d = 0, 2, 10, 8, 2, 128
    for f in ("q", "q_out", "k", "v", "cu_seqlens", "seqlens_k", "cos_sin", "block_table", "k_cache", "v_cache",
              "cache"):
        setattr(a, f, 4096)
    a.q_strides = a.q_out_strides = (8 * 128, 128)
    a.k_strides = a.v_strides = (2 * 128, 128)
    a.rotary_dim, a.max_positions = 128, 1000
    a.num_pages, a.page_size, a.block_table_stride, a.block_table_width = 16, 64, 4, 4
    a.k_cache_strides = a.v_cache_strides = (64 * 256, 256, 128)
    a.group = 64
    a.cache_strides = (2 * 64 * 144, 64 * 144)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BOTH = [("dtype", 2, 1), ("b", 0, 1), ("total", -1, 1), ("hq", -1, 1), ("hkv", 0, 1), ("d", 96, 2), ("d", 32, 2),
        ("total", (1 << 30) + 1, 2), ("interleaved", 2, 1), ("rotary_dim", -8, 1), ("rotary_dim", 136, 1),
        ("rotary_dim", 24, 2), ("cos_sin", 0, 1), ("cos_sin", 4100, 1), ("max_positions", 0, 1), ("num_pages", 0, 1),
        ("page_size", 0, 1), ("page_size", 96, 2), ("block_table", 0, 1), ("block_table", 4098, 1),
        ("block_table_stride", -1, 1), ("block_table_width", 0, 1), ("seqlens_k", 0, 1), ("cu_seqlens", 4097, 1), ("k", 0, 1), ("v", 4104, 1),
        ("q", 0, 1), ("q_out", 0, 1), ("q_out", 4100, 1), ("k_strides", (250, 128), 1), ("v_strides", (256, 0), 1),
        ("q_strides", (-1024, 128), 1), ("q_out_strides", (1024, 4), 1)]


@pytest.mark.parametrize("field,value,expect", BOTH)
def test_append_refusals(lib, field, value, expect):
    a = _append_args(**{field: value})
    assert lib.fa_kv_append(ctypes.byref(a), None) == expect
    assert lib.fa_kv_append_int4(ctypes.byref(a), None) == expect


def test_append_refusals_of_each_cache(lib):
    for field, value in (("k_cache", 0), ("v_cache", 4100), ("k_cache_strides", (64 * 256, 256, 4)),
                         ("v_cache_strides", (0, 256, 128))):
        assert lib.fa_kv_append(ctypes.byref(_append_args(**{field: value})), None) == 1, field
    for field, value, expect in (("cache", 0, 1), ("cache", 4104, 1), ("group", 16, 2), ("group", 256, 2),
                                 ("cache_strides", (2 * 64 * 144, 64 * 144 - 16), 1), ("cache_strides", (100, 64 * 144), 1)):
        assert lib.fa_kv_append_int4(ctypes.byref(_append_args(**{field: value})), None) == expect, field
    assert lib.fa_kv_append_int4(ctypes.byref(_append_args(d=64, rotary_dim=64, group=128)), None) == 2
    assert lib.fa_kv_append_int4(None, None) == 1 and lib.fa_kv_append(None, None) == 1


def test_append_of_nothing_needs_no_device(lib):
    assert lib.fa_kv_append(ctypes.byref(_append_args(total=0, k=0, v=0, q=0, q_out=0)), None) == 0
    assert lib.fa_kv_append_int4(ctypes.byref(_append_args(total=0)), None) == 0
    # equal shares of the rows without prefix sums
    assert lib.fa_kv_append(ctypes.byref(_append_args(total=9, cu_seqlens=0)), None) == 1
    # interleaved rotation needs whole chunks of pairs only
    assert lib.fa_kv_append(ctypes.byref(_append_args(total=0, rotary_dim=24, interleaved=1)), None) == 0


def test_page_bytes(lib):
    assert lib.fa_kvcache_int4_page_bytes(64, 128, 128) == 64 * (128 + 8)
    assert lib.fa_kvcache_int4_page_bytes(256, 64, 32) == 256 * (64 + 16)
    assert lib.fa_kvcache_int4_page_bytes(64, 256, 32) == 64 * (256 + 64)
    for bad in ((0, 128, 128), (96, 128, 128), (64, 96, 32), (64, 64, 128), (64, 128, 16), (-64, 128, 64)):
        assert lib.fa_kvcache_int4_page_bytes(*bad) == 0


def _gather_args(**kw):
    from tiled_exact_attention_gb300._lib import KvGatherInt4Args

    a = KvGatherInt4Args()
    a.dtype, a.b, a.total, a.hkv, a.d, a.group = 1, 2, 10, 2, 128, 32
    for f in ("cache", "block_table", "seqlens_k", "cu_seqlens", "k", "v"):
        setattr(a, f, 4096)
    a.cache_strides = (2 * 64 * 160, 64 * 160)
    a.num_pages, a.page_size, a.block_table_stride, a.block_table_width = 16, 64, 4, 4
    a.k_strides = a.v_strides = (256, 128)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("field,value,expect", [
    ("dtype", 5, 1), ("b", 0, 1), ("total", -1, 1), ("hkv", 0, 1), ("d", 80, 2), ("group", 48, 2), ("cache", 0, 1),
    ("cache_strides", (2 * 64 * 160, 64 * 160 + 8), 1), ("page_size", 32, 2), ("block_table", 0, 1), ("k", 0, 1),
    ("v", 4098, 1), ("k_strides", (256, 12), 1), ("cu_seqlens", 4097, 1), ("total", (1 << 30) + 1, 2)])
def test_gather_refusals(lib, field, value, expect):
    assert lib.fa_kv_gather_int4(ctypes.byref(_gather_args(**{field: value})), None) == expect


def _attend_args(**kw):
    from tiled_exact_attention_gb300._lib import KvcacheInt4Args

    a = KvcacheInt4Args()
    a.dtype, a.b, a.sq, a.hq, a.hkv, a.d, a.group = 0, 2, 1, 8, 2, 128, 128
    for f in ("q", "cache", "block_table", "seqlens_k", "o", "lse"):
        setattr(a, f, 4096)
    a.q_strides = a.o_strides = (8 * 128, 8 * 128, 128)
    a.cache_strides = (2 * 64 * 136, 64 * 136)
    a.num_pages, a.page_size, a.block_table_stride, a.block_table_width = 16, 64, 4, 4
    a.scale = 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("field,value,expect", [
    ("dtype", -1, 1), ("b", 0, 1), ("sq", -1, 1), ("hq", 7, 1), ("hkv", 0, 1), ("d", 96, 2), ("group", 96, 2),
    ("b", 65536, 2), ("sq", 16385, 2), ("block_table_width", 0, 1), ("scale", 0.0, 1), ("scale", float("inf"), 1), ("softcap", -1.0, 1),
    ("softcap", float("nan"), 1), ("local", 2, 1), ("cache", 4104, 1), ("page_size", 100, 2), ("seqlens_k", 0, 1),
    ("q", 0, 1), ("o", 4100, 1), ("lse", 0, 1), ("q_strides", (1024, 1024, 100), 1), ("o_strides", (1024, 0, 128), 1)])
def test_attend_refusals(lib, field, value, expect):
    a = _attend_args(**{field: value})
    assert lib.fa_fwd_kvcache_int4(ctypes.byref(a), None, 0, None) == expect
    assert lib.fa_kvcache_int4_workspace_size(ctypes.byref(a)) == 0


def test_attend_refusals_of_combinations(lib):
    assert lib.fa_fwd_kvcache_int4(ctypes.byref(_attend_args(local=1, window_left=-2)), None, 0, None) == 1
    assert lib.fa_fwd_kvcache_int4(ctypes.byref(_attend_args(sq=0)), None, 0, None) == 0  # nothing to do
    assert lib.fa_fwd_kvcache_int4(None, None, 0, None) == 1
    assert lib.fa_fwd_kvcache_int4(ctypes.byref(_attend_args()), None, 0, None) in (1, 3)  # no workspace / no device


def test_wrappers_refuse_host_tensors():
    import tiled_exact_attention_gb300 as fa

    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 1, dtype=torch.int32)
    c16 = torch.zeros(2, 64, 1, 64, dtype=torch.bfloat16)
    c4 = torch.zeros(2, 1, 64 * 72, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fa.fa_kv_append(x, x, c16, c16, block_table=t, seqlens_k=i)
    with pytest.raises(ValueError):
        fa.fa_kv_append_int4(x, x, c4, group=64, block_table=t, seqlens_k=i)
    with pytest.raises(ValueError):
        fa.fa_kv_gather_int4(c4, group=64, block_table=t, seqlens_k=i, total=2, d=64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_kv_gather_int4(c4, group=64, block_table=t, seqlens_k=i)
    with pytest.raises(ValueError):
        fa.fa_fwd_kvcache_int4(x, c4, group=64, block_table=t, seqlens_k=i)
