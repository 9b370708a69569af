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
    return ctypes.byref(fa._Strides(b, h, n))


def cache(**kw):
    c = dict(k_pages=P, v_pages=P + 0x100000, k_page=16 * 256, k_head=128, k_row=256,
             v_page=16 * 256, v_head=128, v_row=256, table=P + 0x200000, cu_q=P + 0x300000,
             seq_k=P + 0x400000, table_row=8, table_width=8, num_pages=100, page_size=16, heads=2,
             d=128, batch=3, tokens=5, dtype=fa.FA_BF16)
    c.update(kw)
    return fa._PagedCache(**c)


def rope(lib, **kw):
    a = dict(xq=P, sq=strides(), yq=P + 0x100000, syq=strides(), hq=4, xk=P + 0x200000,
             sk=strides(), yk=P + 0x300000, syk=strides(), hk=2, pos=P + 0x400000, row=64,
             freqs=P + 0x500000, rot=64, mag=1.0, il=0, inv=0, B=2, N=64, d=128,
             dtype=fa.FA_BF16, stream=None)
    a.update(kw)
    return lib.fa_rope(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), fa.FA_ERR_INVALID), (dict(N=-1), fa.FA_ERR_INVALID),
    (dict(hq=-1), fa.FA_ERR_INVALID), (dict(d=0), fa.FA_ERR_INVALID),
    (dict(xq=None), fa.FA_ERR_INVALID), (dict(yq=P + 8), fa.FA_ERR_INVALID),
    (dict(xk=P + 2), fa.FA_ERR_INVALID), (dict(yk=None), fa.FA_ERR_INVALID),
    (dict(sq=None), fa.FA_ERR_INVALID), (dict(sk=strides(n=4)), fa.FA_ERR_INVALID),
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
    a = dict(k=P + 0x500000, sk=strides(), v=P + 0x600000, sv=strides(), xq=P + 0x700000,
             sq=strides(), yq=P + 0x800000, syq=strides(), hq=4, pos=None, freqs=P + 0x900000,
             rot=64, mag=1.0, il=0, stream=None)
    a.update(kw)
    return lib.fa_paged_append(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(num_pages=0), fa.FA_ERR_INVALID), (dict(table_width=0), fa.FA_ERR_INVALID)])
def test_append_rejects_a_bad_cache(lib, kw, code):
    assert append(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), fa.FA_ERR_INVALID), (dict(v=P + 4), fa.FA_ERR_INVALID),
    (dict(sk=None), fa.FA_ERR_INVALID), (dict(sv=strides(h=12)), fa.FA_ERR_INVALID),
    (dict(hq=-1), fa.FA_ERR_INVALID), (dict(freqs=None), fa.FA_ERR_INVALID),
    (dict(yq=None), fa.FA_ERR_INVALID), (dict(rot=200), fa.FA_ERR_INVALID),
    (dict(rot=40), fa.FA_ERR_UNSUPPORTED), (dict(pos=P + 1), fa.FA_ERR_INVALID),
    (dict(mag=float("nan")), fa.FA_ERR_INVALID),
])
def test_append_rejects_before_launch(lib, kw, code):
    assert append(lib, cache(), **kw) == code


def attention(lib, c, **kw):
    a = dict(q=P + 0x500000, sq=strides(), o=P + 0x600000, so=strides(), L=P + 0x700000, hq=8,
             max_q=2, wl=-1, wr=0, scale=0.1, ws=P + 0x800000, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.fa_paged_attention(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("kw,code", BAD_CACHE + [(dict(d=80), fa.FA_ERR_UNSUPPORTED)])
def test_attention_rejects_a_bad_cache(lib, kw, code):
    assert attention(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), fa.FA_ERR_INVALID), (dict(o=P + 8), fa.FA_ERR_INVALID),
    (dict(L=None), fa.FA_ERR_INVALID), (dict(sq=strides(n=12)), fa.FA_ERR_INVALID),
    (dict(so=None), fa.FA_ERR_INVALID), (dict(hq=7), fa.FA_ERR_INVALID),
    (dict(max_q=-1), fa.FA_ERR_INVALID), (dict(scale=0.0), fa.FA_ERR_INVALID),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID), (dict(hq=2 * 129), fa.FA_ERR_UNSUPPORTED),
    (dict(hq=0), fa.FA_OK),
])
def test_attention_rejects_before_launch(lib, kw, code):
    assert attention(lib, cache(), **kw) == code


def test_workspace_size_refuses(lib):
    assert lib.fa_paged_workspace_size(-1, 1, 8, 2, 128) == ctypes.c_size_t(-1).value
    assert lib.fa_paged_workspace_size(4, 1, 8, 0, 128) == ctypes.c_size_t(-1).value


# Threads per block of every kernel the library launches.
# (fa_paged_step_kernel: 192 up to 32 query columns, 320 for 64)
BLOCK_THREADS = {"fa_rope_kernel": 256, "fa_paged_step_kernel": 192, "fa_paged_merge_kernel": 256,
                 "fa_paged_chunk_kernel": 384}


def test_every_kernel_fits_the_register_file_at_its_block_size():
    seen = set()
    for name, res in build.paged_resources().items():
        fam = [k for k in BLOCK_THREADS if k in name]
        assert len(fam) == 1, name
        seen.add(fam[0])
        wide = re.search(r"fa_paged_step_kernelILi\d+ELi64E", name)
        warps = -(-(320 if wide else BLOCK_THREADS[fam[0]]) // 32)
        regs = -(-res["registers"] // 8) * 8  # allocated in units of 8 per thread
        assert regs * 32 * -(-warps // 4) <= 16384, (name, res["registers"])
    assert seen == set(BLOCK_THREADS)
