"""Host-side checks of libfa_paged.so (no GPU needed, nothing is launched): every function
of include/fa_paged.h is exported and bound, bad arguments are refused before the device is
touched, and every kernel fits the register file at its block size."""

import ctypes
import os
import re

import pytest

from exact_io_aware_69_b200 import build, fa

HEADER = os.path.join(build.INCLUDE, "fa_paged.h")
P = 0x7F0000000000  # fake, well-aligned device addresses


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return fa.load_paged()


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(fa_[a-z_0-9]+)\s*\(", text))
    assert names == set(fa.PAGED_SIGNATURES)
    for name in names:
        assert hasattr(lib, name), name


def strides(b=4096, h=128, n=1024):
    return b, h, n


def cache(**kw):
    c = dict(k_pages=P, v_pages=P + 0x100000, k_page=16 * 256, k_head=128, k_row=256,
             v_page=16 * 256, v_head=128, v_row=256, table=P + 0x200000, cu_q=P + 0x300000,
             seq_k=P + 0x400000, table_row=8, table_width=8, num_pages=100, page_size=16, heads=2,
             d=128, batch=3, tokens=5, dtype=fa.FA_BF16)
    assert set(kw) <= set(c)
    c.update(kw)
    return [v or 0 for v in c.values()]


def pack(fields, values, defaults):
    assert set(values) <= set(defaults)
    flat = []
    for v in {**defaults, **values}.values():
        flat += list(v) if isinstance(v, (tuple, list)) else [v or 0]
    return fields.pack(*flat)


def rope(lib, **kw):
    return lib.fa_rope(pack(fa._ROPE_ARGS, kw, dict(
        xq=P, yq=P + 0x100000, sq=strides(), syq=strides(), hq=4, xk=P + 0x200000,
        yk=P + 0x300000, sk=strides(), syk=strides(), hk=2, pos=P + 0x400000, row=64,
        freqs=P + 0x500000, rot=64, il=0, inv=0, B=2, N=64, d=128, dtype=fa.FA_BF16,
        mag=1.0)), None)


def test_the_bindings_structs_are_the_headers(tmp_path):
    """Sizes and the offset of a late field of each argument struct, from the C compiler."""
    import subprocess
    source = tmp_path / "sizes.c"
    source.write_text('#include "fa_paged.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                      'int main(void) { printf("%zu %zu %zu %zu %zu %zu", sizeof(fa_rope_args), '
                      'sizeof(fa_paged_append_args), sizeof(fa_paged_attention_args), '
                      'offsetof(fa_rope_args, magnitude), offsetof(fa_paged_append_args, '
                      'magnitude), offsetof(fa_paged_attention_args, workspace_bytes)); }')
    subprocess.run(["gcc", "-I", build.INCLUDE, str(source), "-o", str(tmp_path / "sizes")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "sizes")], capture_output=True,
                                          check=True).stdout.split()]
    assert got == [fa._ROPE_ARGS.size, fa._APPEND_ARGS.size, fa._ATTENTION_ARGS.size,
                   fa._ROPE_ARGS.size - 4, fa._APPEND_ARGS.size - 8,
                   fa._ATTENTION_ARGS.size - 8]


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), fa.FA_ERR_INVALID), (dict(N=-1), fa.FA_ERR_INVALID),
    (dict(hq=-1), fa.FA_ERR_INVALID), (dict(d=0), fa.FA_ERR_INVALID),
    (dict(xq=None), fa.FA_ERR_INVALID), (dict(yq=P + 8), fa.FA_ERR_INVALID),
    (dict(xk=P + 2), fa.FA_ERR_INVALID), (dict(yk=None), fa.FA_ERR_INVALID),
    (dict(sk=strides(n=4)), fa.FA_ERR_INVALID),
    (dict(syq=strides(h=-8)), fa.FA_ERR_INVALID), (dict(pos=P + 2), fa.FA_ERR_INVALID),
    (dict(row=-1), fa.FA_ERR_INVALID), (dict(freqs=None), fa.FA_ERR_INVALID),
    (dict(freqs=P + 4), fa.FA_ERR_INVALID), (dict(rot=144), fa.FA_ERR_INVALID),
    (dict(rot=0), fa.FA_ERR_INVALID), (dict(rot=24), fa.FA_ERR_UNSUPPORTED),
    (dict(mag=float("inf")), fa.FA_ERR_INVALID), (dict(d=72, rot=16), fa.FA_ERR_UNSUPPORTED),
    (dict(d=1040), fa.FA_ERR_UNSUPPORTED), (dict(dtype=2), fa.FA_ERR_UNSUPPORTED),
    (dict(B=0), fa.FA_OK), (dict(N=0, xq=None), fa.FA_OK), (dict(hq=0, hk=0), fa.FA_OK),
])
def test_rope_rejects_before_launch(lib, kw, code):
    assert rope(lib, **kw) == code


BAD_CACHE = [
    (dict(batch=-1), fa.FA_ERR_INVALID), (dict(tokens=-1), fa.FA_ERR_INVALID),
    (dict(heads=0), fa.FA_ERR_INVALID), (dict(table_row=-1), fa.FA_ERR_INVALID),
    (dict(k_pages=None), fa.FA_ERR_INVALID), (dict(v_pages=P + 8), fa.FA_ERR_INVALID),
    (dict(k_row=260), fa.FA_ERR_INVALID), (dict(v_page=-8), fa.FA_ERR_INVALID),
    (dict(table=None), fa.FA_ERR_INVALID), (dict(cu_q=P + 2), fa.FA_ERR_INVALID),
    (dict(seq_k=None), fa.FA_ERR_INVALID), (dict(page_size=8), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=48), fa.FA_ERR_UNSUPPORTED), (dict(page_size=2048), fa.FA_ERR_UNSUPPORTED),
    (dict(d=72), fa.FA_ERR_UNSUPPORTED), (dict(dtype=5), fa.FA_ERR_UNSUPPORTED),
    (dict(batch=20000), fa.FA_ERR_UNSUPPORTED), (dict(table_width=1 << 25), fa.FA_ERR_UNSUPPORTED),
    (dict(batch=0), fa.FA_OK), (dict(tokens=0, cu_q=None), fa.FA_OK),
]


def append(lib, c, **kw):
    return lib.fa_paged_append(pack(fa._APPEND_ARGS, kw, dict(
        cache=c, k=P + 0x500000, v=P + 0x600000, sk=strides(), sv=strides(), xq=P + 0x700000,
        yq=P + 0x800000, sq=strides(), syq=strides(), hq=4, pos=0, freqs=P + 0x900000, rot=64,
        il=0, mag=1.0)), None)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(num_pages=0), fa.FA_ERR_INVALID), (dict(table_width=0), fa.FA_ERR_INVALID)])
def test_append_rejects_a_bad_cache(lib, kw, code):
    assert append(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), fa.FA_ERR_INVALID), (dict(v=P + 4), fa.FA_ERR_INVALID),
    (dict(sv=strides(h=12)), fa.FA_ERR_INVALID),
    (dict(hq=-1), fa.FA_ERR_INVALID), (dict(freqs=None), fa.FA_ERR_INVALID),
    (dict(yq=None), fa.FA_ERR_INVALID), (dict(rot=200), fa.FA_ERR_INVALID),
    (dict(rot=40), fa.FA_ERR_UNSUPPORTED), (dict(pos=P + 1), fa.FA_ERR_INVALID),
    (dict(mag=float("nan")), fa.FA_ERR_INVALID),
])
def test_append_rejects_before_launch(lib, kw, code):
    assert append(lib, cache(), **kw) == code


def attention(lib, c, **kw):
    return lib.fa_paged_attention(pack(fa._ATTENTION_ARGS, kw, dict(
        cache=c, q=P + 0x500000, o=P + 0x600000, L=P + 0x700000, sq=strides(), so=strides(), hq=8,
        max_q=2, wl=-1, wr=0, scale=0.1, ws=P + 0x800000, ws_bytes=1 << 40)), None)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [(dict(d=80), fa.FA_ERR_UNSUPPORTED)])
def test_attention_rejects_a_bad_cache(lib, kw, code):
    assert attention(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), fa.FA_ERR_INVALID), (dict(o=P + 8), fa.FA_ERR_INVALID),
    (dict(L=None), fa.FA_ERR_INVALID), (dict(sq=strides(n=12)), fa.FA_ERR_INVALID),
    (dict(sq=strides(h=0)), fa.FA_ERR_UNSUPPORTED), (dict(ws=None), fa.FA_ERR_INVALID),
    (dict(ws=P + 0x800010), fa.FA_ERR_INVALID), (dict(ws_bytes=1000), fa.FA_ERR_INVALID),
    (dict(hq=7), fa.FA_ERR_INVALID),
    (dict(max_q=-1), fa.FA_ERR_INVALID), (dict(scale=0.0), fa.FA_ERR_INVALID),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID), (dict(hq=2 * 129), fa.FA_ERR_UNSUPPORTED),
    (dict(hq=0), fa.FA_OK),
])
def test_attention_rejects_before_launch(lib, kw, code):
    assert attention(lib, cache(), **kw) == code


def test_null_arguments(lib):
    for name in ("fa_rope", "fa_paged_append", "fa_paged_attention"):
        assert getattr(lib, name)(None, None) == fa.FA_ERR_INVALID


def test_workspace_size(lib):
    """Two parts per CTA (148) of 16, 32 or 256 rows, d outputs and a log-sum-exp each, behind
    32 bytes per CTA."""
    for max_q, hq, heads, d, rows in ((1, 8, 8, 64, 16), (4, 32, 8, 128, 16), (5, 32, 8, 128, 32),
                                      (5, 32, 8, 64, 256), (24, 2, 2, 128, 32),
                                      (25, 2, 2, 128, 256), (33, 2, 2, 128, 256)):
        assert lib.fa_paged_workspace_size(1000, max_q, hq, heads, d) == \
            148 * 32 + 2 * 148 * rows * (d + 1) * 4
    assert lib.fa_paged_workspace_size(0, 1, 8, 2, 128) == 0
    assert lib.fa_paged_workspace_size(7, 2, 7, 2, 128) == ctypes.c_size_t(-1).value
    assert lib.fa_paged_workspace_size(-1, 1, 8, 2, 128) == ctypes.c_size_t(-1).value
    assert lib.fa_paged_workspace_size(4, 1, 8, 0, 128) == ctypes.c_size_t(-1).value


# Threads per block of every kernel the library launches.
BLOCK_THREADS = {"fa_rope_kernel": 128, "fa_paged_step_kernel": 256, "fa_paged_merge_kernel": 256,
                 "fa_paged_chunk_kernelILi64E": 640, "fa_paged_chunk_kernelILi128E": 384}


def test_every_kernel_fits_the_register_file_at_its_block_size():
    seen = set()
    for name, res in build.paged_resources().items():
        fam = [k for k in BLOCK_THREADS if k in name]
        assert len(fam) == 1, name
        seen.add(fam[0])
        warps = -(-BLOCK_THREADS[fam[0]] // 32)
        regs = -(-res["registers"] // 8) * 8  # allocated in units of 8 per thread
        assert regs * 32 * -(-warps // 4) <= 16384, (name, res["registers"])
    assert seen == set(BLOCK_THREADS)
