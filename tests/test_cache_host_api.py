"""Checks of attention over packed sequences and paged caches that need no GPU: the header and the binding agree, sizes,
and the refusals, which all happen before any launch."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import block_sparse_attention_mean_gb300 as pkg
from block_sparse_attention_mean_gb300 import binding as bb
from block_sparse_attention_mean_gb300 import build as bbuild
from block_sparse_attention_mean_gb300 import cache_binding as cb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bsa_cache.h")
FAKE = 1 << 40  # an aligned non-null address that is never dereferenced on these paths
FAR = 1 << 36   # between two such tensors
SIZE = 1 << 34  # of a workspace


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return cb.load()


def refused(code, fn, *args, **kw):
    with pytest.raises(bb.BsaError) as e:
        fn(*args, **kw)
    assert e.value.code == code, str(e.value)


def test_header_symbols_exported(lib):
    names = sorted(re.findall(r"^bsa_status\s+(bsa_\w+)\s*\(", open(HEADER).read(), re.M))
    assert sorted(cb.EXPORTS) == names
    for n in names:
        assert getattr(lib, n) is not None
    assert f"BSA_CACHE_ROWS_WORKSPACE {cb.ROWS_WORKSPACE}\n" in open(HEADER).read()


@pytest.mark.parametrize("cc,std,lang", [("gcc", "-std=c99", "c"), ("g++", "-std=c++17", "c++")])
def test_header_is_plain_c_and_cpp(cc, std, lang):
    if shutil.which(cc) is None:
        pytest.skip(f"{cc} not available")
    r = subprocess.run([cc, std, "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-x", lang, HEADER],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_struct_layouts_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    mirrors = {"bsa_kv_cache": cb.KvCacheStruct, "bsa_page_table": cb.PageTable, "bsa_packed": cb.Packed}
    lines, expected = [], []
    for c, m in mirrors.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        expected.append(ctypes.sizeof(m))
        for name, _ in m._fields_:
            lines.append(f'printf("%zu\\n", offsetof({c}, {name}));')
            expected.append(getattr(m, name).offset)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include "{HEADER}"\nint main(void) {{\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == expected


def test_packed_descriptors_match_the_structures():
    for fmt, mirror in ((cb._CACHE, cb.KvCacheStruct), (cb._TABLE, cb.PageTable), (cb._PACKED, cb.Packed)):
        assert fmt.size == ctypes.sizeof(mirror)
        n = len(fmt.unpack(bytes(fmt.size)))
        got = mirror.from_buffer_copy(fmt.pack(*range(1, n + 1)))
        assert [getattr(got, f) for f, _ in mirror._fields_] == list(range(1, n + 1))


def test_package_offers_the_helpers():
    for n in ("KvCache", "cache_attention", "cache_check", "cache_read", "cache_workspace", "cache_write", "kv_cache",
              "prompt_attention"):
        assert getattr(pkg, n) is getattr(cb, n) and n in pkg.__all__


def test_workspace_sizes():
    size = cb.bsa_cache_workspace_size
    small = size(1, 1, 8, 8, 128)
    assert small >= cb.ROWS_WORKSPACE and small % 256 == 0
    assert size(65536, 4, 16, 16, 128) >= size(4096, 4, 16, 16, 128) >= size(0, 1, 16, 16, 128)
    assert size(1 << 20, 1000, 64, 1, 128) < 1 << 30
    for bad in ((-1, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 8, 3, 128), (1, 1, 8, 0, 128), (1, 1, 8, 8, 96),
                (1, 1, 258, 2, 64), (1, 1, 4, 8, 64), (2 ** 31 - 1, 1, 65535, 65535, 64)):
        refused(bb.ERR_SHAPE, size, *bad)


# ------------------------------------------------------------------ refusals of the C entry points


def kv(**more):
    c = dict(k=FAKE, v=FAKE + FAR, k_exp=FAKE + 2 * FAR, v_exp=FAKE + 3 * FAR, kind=cb.CACHE_E4M3, n_pages=10, page_size=64,
             heads=4, d=128)
    c.update(more)
    return cb.KvCacheStruct(*c.values())


def table(**more):
    t = dict(pages=FAKE + 4 * FAR, stride=8, B=3, width=8)
    t.update(more)
    return cb.PageTable(*t.values())


def packed(at, heads=4, d=128, **more):
    p = dict(ptr=FAKE + at * FAR, token=heads * d, head=d)
    p.update(more)
    return cb.Packed(*p.values())


LENS, CU, WS = FAKE + 8 * FAR, FAKE + 9 * FAR, FAKE + 10 * FAR

BAD_CACHES = [
    (bb.ERR_SHAPE, dict(d=96)), (bb.ERR_SHAPE, dict(heads=0)), (bb.ERR_SHAPE, dict(n_pages=0)),
    (bb.ERR_SHAPE, dict(page_size=48)), (bb.ERR_SHAPE, dict(page_size=8)), (bb.ERR_SHAPE, dict(page_size=512)),
    (bb.ERR_SHAPE, dict(page_size=0)), (bb.ERR_SHAPE, dict(n_pages=2 ** 31 - 1, heads=65535, page_size=256)),
    (bb.ERR_INVALID_ARG, dict(kind=2)), (bb.ERR_INVALID_ARG, dict(k=None)), (bb.ERR_INVALID_ARG, dict(v=FAKE + FAR + 8)),
    (bb.ERR_INVALID_ARG, dict(k_exp=None)), (bb.ERR_INVALID_ARG, dict(v_exp=FAKE + 1)),
]
BAD_TABLES = [(bb.ERR_SHAPE, dict(B=0)), (bb.ERR_SHAPE, dict(width=0)), (bb.ERR_INVALID_ARG, dict(pages=None)),
              (bb.ERR_INVALID_ARG, dict(pages=FAKE + 2)), (bb.ERR_INVALID_ARG, dict(stride=7)),
              (bb.ERR_INVALID_ARG, dict(stride=2 ** 62))]
BAD_PACKED = [dict(ptr=None), dict(ptr=FAKE + 8), dict(token=0), dict(head=0), dict(token=-512), dict(head=7), dict(token=2 ** 40),
              dict(head=2 ** 62)]


def write(c=None, k=None, v=None, dt=bb.BF16, T=5, t=None, lens=LENS, cu=CU, ws=WS, size=SIZE):
    cb.bsa_cache_write(c or kv(), k or packed(5), v or packed(6), dt, T, t or table(), lens, cu, ws, size, 0)


def read(c=None, k=None, v=None, dt=bb.BF16, T=5, t=None, cu=CU, ws=WS, size=SIZE):
    cb.bsa_cache_read(c or kv(), t or table(), cu, k or packed(5), v or packed(6), dt, T, ws, size, 0)


def decode(c=None, q=None, dt=bb.BF16, H=8, t=None, lens=LENS, scale=0.0, o=None, lse=FAKE + 7 * FAR, ws=WS, size=SIZE):
    cb.bsa_cache_attention(c or kv(), q or packed(5, 8), dt, H, t or table(), lens, scale, o or packed(6, 8), lse, ws, size, 0)


def prompt(q=None, k=None, v=None, dt=bb.BF16, Tq=100, Tk=100, B=3, H=8, Hk=4, d=128, cu_q=CU, cu_k=LENS, causal=1, scale=0.0,
           o=None, lse=FAKE + 7 * FAR, ws=WS, size=SIZE):
    cb.bsa_prompt_attention(q or packed(0, 8), k or packed(1), v or packed(2), dt, Tq, Tk, B, H, Hk, d, cu_q, cu_k, causal,
                            scale, o or packed(3, 8), lse, ws, size, 0)


@pytest.mark.parametrize("call", [write, read, decode])
def test_cache_and_table_refusals(call):
    for code, bad in BAD_CACHES:
        refused(code, call, c=kv(**bad))
    for code, bad in BAD_TABLES:
        refused(code, call, t=table(**bad))
    refused(bb.ERR_DTYPE, call, dt=bb.FP32)
    refused(bb.ERR_WORKSPACE, call, ws=None)
    refused(bb.ERR_WORKSPACE, call, ws=WS + 128)
    refused(bb.ERR_WORKSPACE, call, size=cb.ROWS_WORKSPACE - 1)
    refused(bb.ERR_INVALID_ARG, call, ws=FAKE)  # in the cache


def test_null_descriptors():
    c, k, t = kv(), packed(5), table()
    refused(bb.ERR_INVALID_ARG, cb.bsa_cache_write, None, k, k, 0, 1, t, LENS, CU, WS, SIZE, 0)
    refused(bb.ERR_INVALID_ARG, cb.bsa_cache_write, c, None, k, 0, 1, t, LENS, CU, WS, SIZE, 0)
    refused(bb.ERR_INVALID_ARG, cb.bsa_cache_write, c, k, k, 0, 1, None, LENS, CU, WS, SIZE, 0)
    refused(bb.ERR_INVALID_ARG, cb.bsa_cache_read, c, t, CU, k, None, 0, 1, WS, SIZE, 0)
    refused(bb.ERR_INVALID_ARG, cb.bsa_cache_attention, c, None, 0, 8, t, LENS, 0.0, k, None, WS, SIZE, 0)
    refused(bb.ERR_INVALID_ARG, cb.bsa_prompt_attention, None, k, k, 0, 1, 1, 1, 4, 4, 128, CU, CU, 1, 0.0, k, None, WS, SIZE, 0)


@pytest.mark.parametrize("call", [write, read])
def test_rows_refusals(call):
    for bad in BAD_PACKED:
        refused(bb.ERR_INVALID_ARG, call, k=packed(5, **bad))
        refused(bb.ERR_INVALID_ARG, call, v=packed(6, **bad))
    refused(bb.ERR_SHAPE, call, T=-1)
    refused(bb.ERR_INVALID_ARG, call, cu=CU + 2)


def test_write_refusals():
    refused(bb.ERR_INVALID_ARG, write, lens=None)
    refused(bb.ERR_INVALID_ARG, write, lens=LENS + 1)
    refused(bb.ERR_SHAPE, write, cu=None, T=5)  # one token a sequence: T is B
    # the cache must be clear of what is read, and of itself
    for name in ("k", "v", "k_exp", "v_exp"):
        for at in (FAKE + 5 * FAR, FAKE + 6 * FAR, FAKE + 4 * FAR, LENS, CU):
            refused(bb.ERR_INVALID_ARG, write, c=kv(**{name: at}))
    refused(bb.ERR_INVALID_ARG, write, c=kv(v=FAKE + 16))
    refused(bb.ERR_INVALID_ARG, write, c=kv(v_exp=FAKE))


def test_read_refusals():
    refused(bb.ERR_INVALID_ARG, read, cu=None)
    refused(bb.ERR_INVALID_ARG, read, v=packed(5))
    refused(bb.ERR_INVALID_ARG, read, k=packed(5, token=128))  # tokens over heads
    for at in (0, 1, 2, 3, 4, 9):
        refused(bb.ERR_INVALID_ARG, read, k=packed(at))


def test_decode_refusals():
    for bad in BAD_PACKED:
        refused(bb.ERR_INVALID_ARG, decode, q=packed(5, 8, **bad))
        refused(bb.ERR_INVALID_ARG, decode, o=packed(6, 8, **bad))
    for H in (0, 3, 6, -4, 65536 * 4):
        refused(bb.ERR_SHAPE, decode, H=H)
    for scale in (-1.0, float("nan"), float("inf")):
        refused(bb.ERR_INVALID_ARG, decode, scale=scale)
    refused(bb.ERR_INVALID_ARG, decode, lens=None)
    refused(bb.ERR_INVALID_ARG, decode, lse=LENS + 2)
    for at in (0, 1, 2, 3, 4, 5, 8, 10):
        refused(bb.ERR_INVALID_ARG, decode, o=packed(at, 8))
        refused(bb.ERR_INVALID_ARG, decode, lse=FAKE + at * FAR)
    refused(bb.ERR_INVALID_ARG, decode, lse=FAKE + 6 * FAR)
    refused(bb.ERR_WORKSPACE, decode, size=cb.ROWS_WORKSPACE)


def test_prompt_refusals():
    for bad in BAD_PACKED:
        refused(bb.ERR_INVALID_ARG, prompt, q=packed(0, 8, **bad))
        refused(bb.ERR_INVALID_ARG, prompt, k=packed(1, **bad))
        refused(bb.ERR_INVALID_ARG, prompt, v=packed(2, **bad))
        refused(bb.ERR_INVALID_ARG, prompt, o=packed(3, 8, **bad))
    for bad in (dict(d=80), dict(H=6), dict(Hk=0), dict(H=4 * 129), dict(B=0), dict(Tq=-1), dict(Tk=-1)):
        refused(bb.ERR_SHAPE, prompt, **bad)
    refused(bb.ERR_DTYPE, prompt, dt=bb.FP32)
    for bad in (dict(cu_q=None), dict(cu_k=None), dict(cu_k=LENS + 2), dict(lse=LENS + 2)):
        refused(bb.ERR_INVALID_ARG, prompt, **bad)
    for scale in (-1.0, float("nan"), float("inf")):
        refused(bb.ERR_INVALID_ARG, prompt, scale=scale)
    for at in (0, 1, 2, 8, 9, 10):
        refused(bb.ERR_INVALID_ARG, prompt, o=packed(at, 8))
        refused(bb.ERR_INVALID_ARG, prompt, lse=FAKE + at * FAR)
    refused(bb.ERR_INVALID_ARG, prompt, lse=FAKE + 3 * FAR)
    refused(bb.ERR_WORKSPACE, prompt, ws=None)
    refused(bb.ERR_WORKSPACE, prompt, size=cb.bsa_cache_workspace_size(0, 1, 8, 4, 128) // 2)


def test_views_of_one_projection_are_told_apart():
    """q, k, v interleaved in one buffer, results beside them in another: the checks pass (and the launch fails here)"""
    token = (8 + 4 + 4) * 128
    q, k, v = (cb.Packed(FAKE + 2 * 128 * at, token, 128) for at in (0, 8, 12))
    if not torch.cuda.is_available():
        refused(bb.ERR_CUDA, prompt, q=q, k=k, v=v, o=cb.Packed(FAKE + 3 * FAR, token, 128))
        refused(bb.ERR_CUDA, write, k=cb.Packed(FAKE + 5 * FAR + 2048, token, 128), v=cb.Packed(FAKE + 5 * FAR + 3 * 1024, token, 128))
    refused(bb.ERR_INVALID_ARG, prompt, q=q, k=k, v=v, o=cb.Packed(FAKE + 1024, token, 128))


# ------------------------------------------------------------------ refusals of the helpers


def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_helpers_refuse_host_tensors():
    cache = cb.KvCache(host(2, 4, 16, 64), host(2, 4, 16, 64))
    t, n = host(1, 2, dtype=torch.int32), host(1, dtype=torch.int32)
    refused(bb.ERR_INVALID_ARG, pkg.cache_write, cache, host(1, 4, 64), host(1, 4, 64), t, n)
    refused(bb.ERR_INVALID_ARG, pkg.cache_read, cache, t, host(2, dtype=torch.int32), 1)
    refused(bb.ERR_INVALID_ARG, pkg.cache_attention, host(1, 4, 64), cache, t, n)
    refused(bb.ERR_INVALID_ARG, pkg.prompt_attention, host(1, 4, 64), host(1, 4, 64), host(1, 4, 64), host(2, dtype=torch.int32))
    refused(bb.ERR_INVALID_ARG, pkg.cache_check, host(64, dtype=torch.uint8))
    refused(bb.ERR_INVALID_ARG, pkg.kv_cache, 1, 16, 1, 64, "int4", "cpu")


def on_any_device(monkeypatch):
    """lets the helpers' own checks run on host tensors; the library's calls are not reached"""
    monkeypatch.setattr(cb, "_cuda_device", lambda t, what: t.device)

    def not_reached(*args):
        raise AssertionError("the library was called")

    monkeypatch.setattr(cb, "_call", not_reached)


def test_helpers_refuse_tensors_that_do_not_go_together(monkeypatch):
    on_any_device(monkeypatch)
    I32 = torch.int32
    cache = pkg.kv_cache(3, 16, 4, 64, "bf16", "cpu")
    q8 = pkg.kv_cache(3, 16, 4, 64, "e4m3", "cpu")
    assert q8.k_exp.shape == (3, 4, 16) and q8.v.dtype == torch.float8_e4m3fn
    t, n, cu = host(2, 3, dtype=I32), host(2, dtype=I32), host(3, dtype=I32)
    k, ws = host(5, 4, 64), host(1 << 14, dtype=torch.uint8)

    def write(cache=cache, k=k, v=k, t=t, n=n, cu=cu):
        pkg.cache_write(cache, k, v, t, n, cu, ws=ws, check=False)

    refused(bb.ERR_SHAPE, write, v=host(5, 3, 64))
    refused(bb.ERR_SHAPE, write, k=host(4, 4, 64))
    refused(bb.ERR_DTYPE, write, v=k.float())
    refused(bb.ERR_INVALID_ARG, write, v=host(5, 64, 4).transpose(1, 2))  # channels not contiguous
    refused(bb.ERR_SHAPE, write, n=host(3, dtype=I32))
    refused(bb.ERR_DTYPE, write, n=n.long())
    refused(bb.ERR_SHAPE, write, cu=host(2, dtype=I32))
    refused(bb.ERR_SHAPE, write, t=host(3, dtype=I32))
    refused(bb.ERR_DTYPE, write, t=t.long())
    refused(bb.ERR_INVALID_ARG, write, t=host(2, 6, dtype=I32)[:, ::2])
    refused(bb.ERR_INVALID_ARG, write, n=host(2, 2, dtype=I32)[:, 0])
    refused(bb.ERR_INVALID_ARG, write, cache=cache._replace(k=host(4, 3, 16, 64).transpose(0, 1)))
    refused(bb.ERR_SHAPE, write, cache=cache._replace(v=host(3, 4, 32, 64)))
    refused(bb.ERR_DTYPE, write, cache=cache._replace(k=cache.k.float()))
    refused(bb.ERR_DTYPE, write, cache=q8._replace(v=cache.v))
    refused(bb.ERR_INVALID_ARG, write, cache=cache._replace(k_exp=q8.k_exp))
    refused(bb.ERR_INVALID_ARG, write, cache=q8._replace(v_exp=None))
    refused(bb.ERR_SHAPE, write, cache=q8._replace(v_exp=q8.v_exp[:2]))
    refused(bb.ERR_INVALID_ARG, pkg.cache_read, cache, t, cu, ws=ws, check=False)
    refused(bb.ERR_SHAPE, pkg.cache_read, cache, t, cu, out=(k, k[:4]), ws=ws, check=False)

    q = host(2, 8, 64)
    for bad, code in ((dict(q=host(3, 8, 64)), bb.ERR_SHAPE), (dict(q=host(2, 8, 128)), bb.ERR_SHAPE), (dict(q=q.float()), bb.ERR_DTYPE),
                      (dict(out=host(2, 8, 32)), bb.ERR_SHAPE), (dict(out=q.half()), bb.ERR_DTYPE),
                      (dict(lse=host(8, 2, dtype=torch.float32)), bb.ERR_SHAPE),
                      (dict(lse=host(8, 2, dtype=torch.float32).T), bb.ERR_INVALID_ARG),
                      (dict(q=q.clone().requires_grad_()), bb.ERR_INVALID_ARG)):
        args = dict(q=q, cache=cache, table=t, kv_lens=n, ws=ws, check=False)
        args.update(bad)
        refused(code, pkg.cache_attention, **args)
    p = host(10, 8, 64)
    for bad, code in ((dict(q=host(10, 8, 128)), bb.ERR_SHAPE), (dict(v=host(5, 2, 64)), bb.ERR_SHAPE), (dict(q=host(10, 64)), bb.ERR_SHAPE),
                      (dict(cu_k=host(4, dtype=I32)), bb.ERR_SHAPE), (dict(cu_q=cu.long()), bb.ERR_DTYPE),
                      (dict(out=host(9, 8, 64)), bb.ERR_SHAPE), (dict(lse=host(10, 8, dtype=torch.float32)), bb.ERR_SHAPE),
                      (dict(k=k.clone().requires_grad_()), bb.ERR_INVALID_ARG)):
        args = dict(q=p, k=k, v=k, cu_q=cu, cu_k=cu, ws=ws, check=False)
        args.update(bad)
        refused(code, pkg.prompt_attention, **args)


def test_a_cache_is_looked_at_in_every_call(monkeypatch):
    monkeypatch.setattr(cb, "_cuda_device", lambda t, what: t.device)
    seen = []
    monkeypatch.setattr(cb, "_call", lambda what, fn, device, ws, check, *args: seen.append(args[0]))
    cache = pkg.kv_cache(3, 16, 4, 64, "e4m3", "cpu")
    t, n, k, ws = host(2, 3, dtype=torch.int32), host(2, dtype=torch.int32), host(2, 4, 64), host(1 << 14, dtype=torch.uint8)

    def write():
        pkg.cache_write(cache, k, k, t, n, ws=ws, check=False)
        return struct.unpack("4P5i4x", seen[-1])

    assert write() == (*(x.data_ptr() for x in cache), 1, 3, 16, 4, 64)
    other = torch.empty_like(cache.k_exp)
    cache.k_exp.set_(other)  # its keys and values stay where they are
    assert write() == (cache.k.data_ptr(), cache.v.data_ptr(), other.data_ptr(), cache.v_exp.data_ptr(), 1, 3, 16, 4, 64)
    for x in cache:
        x.set_(x[:2])
    assert write()[5] == 2
    cache.k.set_(cache.k[:1])
    refused(bb.ERR_SHAPE, write)


def test_helpers_refuse_gradients_of_caches_and_sums(monkeypatch):
    on_any_device(monkeypatch)
    cache = pkg.kv_cache(3, 16, 4, 64, "bf16", "cpu")
    t, n, ws = host(2, 3, dtype=torch.int32), host(2, dtype=torch.int32), host(1 << 14, dtype=torch.uint8)
    lse = host(2, 8, dtype=torch.float32).requires_grad_()
    refused(bb.ERR_INVALID_ARG, pkg.cache_attention, host(2, 8, 64), cache, t, n, lse=lse, ws=ws, check=False)
    learned = cache._replace(v=cache.v.clone().requires_grad_())
    refused(bb.ERR_INVALID_ARG, pkg.cache_attention, host(2, 8, 64), learned, t, n, ws=ws, check=False)
    refused(bb.ERR_INVALID_ARG, pkg.cache_write, learned, host(2, 4, 64), host(2, 4, 64), t, n, ws=ws, check=False)
    with torch.no_grad(), pytest.raises(AssertionError, match="library was called"):
        pkg.cache_attention(host(2, 8, 64), learned, t, n, lse=lse, ws=ws, check=False)


def test_helpers_refuse_tangents(monkeypatch):
    """each operand in turn; what carries none passes, and so does everything in a torch.autograd.Function's forward"""
    monkeypatch.setattr(cb, "_cuda_device", lambda t, what: t.device)
    reached = []
    monkeypatch.setattr(cb, "_call", lambda what, *args: reached.append(what))
    cache, q8 = pkg.kv_cache(3, 16, 4, 64, "bf16", "cpu"), pkg.kv_cache(3, 16, 4, 64, "e4m3", "cpu")
    t, n, cu, ws = host(2, 3, dtype=torch.int32), host(2, dtype=torch.int32), host(3, dtype=torch.int32), host(1 << 14, dtype=torch.uint8)
    q, kv = host(2, 8, 64), host(2, 4, 64)
    more = dict(ws=ws, check=False)
    calls = [
        (lambda k, v, ck, cv: pkg.cache_write(cb.KvCache(ck, cv), k, v, t, n, **more), dict(k=kv, v=kv, ck=cache.k, cv=cache.v)),
        (lambda ck, cv, ok, ov: pkg.cache_read(cb.KvCache(ck, cv), t, cu, out=(ok, ov), **more), dict(ck=cache.k, cv=cache.v, ok=kv, ov=kv)),
        (lambda q, ck, cv, out, lse: pkg.cache_attention(q, cb.KvCache(ck, cv), t, n, out=out, lse=lse, **more),
         dict(q=q, ck=cache.k, cv=cache.v, out=q, lse=host(2, 8, dtype=torch.float32))),
        (lambda q, k, v, out, lse: pkg.prompt_attention(q, k, v, cu, out=out, lse=lse, **more),
         dict(q=q, k=kv, v=kv, out=q, lse=host(8, 2, dtype=torch.float32))),
    ]
    ad = torch.autograd.forward_ad
    for fn, tensors in calls:
        with ad.dual_level():
            fn(**tensors)
            for name, x in tensors.items():
                before = len(reached)
                refused(bb.ERR_INVALID_ARG, fn, **dict(tensors, **{name: ad.make_dual(x.clone(), torch.ones_like(x))}))
                assert len(reached) == before
    with ad.dual_level():
        pkg.cache_write(q8, kv, kv, t, n, **more)

        class Wrapped(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x):
                return pkg.prompt_attention(x, kv, kv, cu, lse=host(8, 2, dtype=torch.float32), **more)[0]

            @staticmethod
            def jvp(ctx, dx):
                return dx

        out = Wrapped.apply(ad.make_dual(q.clone(), torch.ones_like(q)))
        assert (ad.unpack_dual(out).tangent == 1).all()
