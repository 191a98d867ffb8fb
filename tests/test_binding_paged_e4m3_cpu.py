"""Argument checks of the quantised paged cache's calls in the binding, on the CPU: a bad argument never reaches the library,
and well-formed CPU tensors get as far as the device check."""
import ctypes
import os
import subprocess

import torch

from prefix_cached_kv_gb300 import binding
from tests.test_binding_paged_cpu import _batch, _cache, _ctx, _raises, i32

E4M3, E8M0, U8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8


def _quantized(device=torch.device("cuda", 0)):
    c = binding.QuantizedPagedCache.__new__(binding.QuantizedPagedCache)
    c.dtype, c.device, c.H_kv, c.D, c.page_size, c.n_pages, c._ws = E4M3, device, 2, 64, 16, 5, {}
    return c


def test_cache():
    k, s = torch.zeros((5, 2, 16, 64), dtype=U8).view(E4M3), torch.zeros((5, 2, 16), dtype=U8)
    f = binding.QuantizedPagedCache
    _raises(lambda: f(k, k[:4], s, s), "one shape")
    _raises(lambda: f(k[0], k[0], s, s), "one shape")
    _raises(lambda: f(k.view(U8), k.view(U8), s, s), "k: dtype")
    _raises(lambda: f(k, torch.zeros(k.shape, dtype=torch.float16), s, s), "v: dtype")
    _raises(lambda: f(k.transpose(2, 3), k.transpose(2, 3), s, s), "last dimension must be contiguous")
    _raises(lambda: f(k, k, s.float(), s), "k_scale: dtype")
    _raises(lambda: f(k, k, s, s[:, :1]), "v_scale: shape")
    _raises(lambda: f(k, k, s, torch.zeros((5, 16, 2), dtype=U8).transpose(1, 2)), "v_scale: must be contiguous")
    _raises(lambda: f(k, k, s, s.view(E8M0)), "must be on the CUDA device")


def test_append():
    c, cache = _ctx(), _quantized()
    K = torch.zeros((3, 2, 64), dtype=torch.float16)
    tab, n = _batch()
    f = lambda K=K, V=K, tab=tab, n=n, **kw: c.paged_append(cache, tab, n, K, V, **kw)   # noqa: E731
    _raises(lambda: f(K=K[:, :1]), "K must be")
    _raises(lambda: f(K=K.double()), "K: dtype")
    _raises(lambda: f(K=K.view(torch.uint8).view(E4M3)[..., :64]), "K: dtype")
    _raises(lambda: f(V=K.float()), "V: dtype")
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        _raises(lambda: f(K=K.to(dt), V=K.to(dt)), "must be on the CUDA device")
    _raises(lambda: c.paged_append(_cache(), tab, n, K.bfloat16(), K.bfloat16()), "K: dtype")      # a 16-bit cache as before


def test_attend():
    c, cache = _ctx(), _quantized()
    Q = torch.zeros((3, 4, 64), dtype=torch.float16)
    tab, n = _batch()
    f = lambda Q=Q, **kw: c.paged_attend(cache, tab, n, Q, **kw)   # noqa: E731
    _raises(lambda: f(Q=Q.float()), "Q: dtype")
    _raises(lambda: f(Q=Q[..., :32]), "Q must be")
    _raises(lambda: f(O=Q.bfloat16()), "O: dtype")
    _raises(lambda: f(Q=Q.bfloat16(), O=Q), "O: dtype")
    _raises(lambda: f(), "must be on the CUDA device")
    _raises(lambda: f(Q=Q.bfloat16()), "must be on the CUDA device")


def test_read():
    c, cache = _ctx(), _quantized()
    tab, n = _batch()
    o = torch.zeros((3, 2, 64))
    f = lambda **kw: c.paged_read(cache, tab, n, **kw)   # noqa: E731
    _raises(lambda: c.paged_read(_cache(), tab, n), "a QuantizedPagedCache is needed")
    _raises(lambda: f(dtype=torch.int8), "dtype")
    _raises(lambda: f(K_out=o), "go together")
    _raises(lambda: f(K_out=o[0], V_out=o[0]), "K_out must be")
    _raises(lambda: f(K_out=o, V_out=o.half()), "V_out: dtype")
    _raises(lambda: f(K_out=o, V_out=o[:, :1]), "V_out: shape")
    _raises(lambda: f(K_out=o[..., ::2], V_out=o[..., ::2]), "K_out: shape")
    _raises(lambda: f(T=4, K_out=o, V_out=o), "K_out: shape")
    _raises(lambda: f(T=4), "cu_rows is needed")
    _raises(lambda: f(T=-1), "T=-1")
    _raises(lambda: f(cu_rows=torch.zeros(4, dtype=i32)), "T is needed")
    _raises(lambda: f(T=9, cu_rows=torch.zeros(3, dtype=i32)), "cu_rows: shape")
    _raises(lambda: f(T=2 ** 31), "2^31")
    _raises(lambda: f(), "must be on the CUDA device")
    _raises(lambda: f(K_out=o, V_out=o), "must be on the CUDA device")


def test_structure_matches_the_header(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [n for n, _ in binding.PagedCacheE4m3T._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pck.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu ", offsetof(pck_paged_cache_e4m3, {n}));\n' for n in names)
                   + 'printf("%zu", sizeof(pck_paged_cache_e4m3));\nreturn 0;\n}\n')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(binding.PagedCacheE4m3T, n).offset for n in names] + [ctypes.sizeof(binding.PagedCacheE4m3T)]
