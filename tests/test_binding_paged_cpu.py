"""Argument checks of the paged-tail calls' binding, on the CPU: a bad argument never reaches the
library, and well-formed CPU tensors get as far as the device check."""
import pytest
import torch

from prefix_cached_kv_gb300 import binding

i32 = torch.int32


class _NoLib:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called with arguments the binding should have rejected")


def _ctx():
    c = binding.Context.__new__(binding.Context)   # no device: never created in the library
    c.lib, c.h, c.device = _NoLib(), None, torch.device("cuda", 0)
    return c


def _cache(dtype=torch.float16, device=torch.device("cuda", 0)):
    c = binding.PagedCache.__new__(binding.PagedCache)
    c.dtype, c.device, c.H_kv, c.D, c.page_size, c.n_pages, c._ws = dtype, device, 2, 64, 16, 5, {}
    return c


def _raises(fn, text):
    with pytest.raises(ValueError) as e:
        fn()
    assert text in str(e.value), str(e.value)


def test_cache():
    k = torch.zeros((5, 2, 16, 64), dtype=torch.float16)
    _raises(lambda: binding.PagedCache(k, k[:4]), "one shape and dtype")
    _raises(lambda: binding.PagedCache(k, k.bfloat16()), "one shape and dtype")
    _raises(lambda: binding.PagedCache(k[0], k[0]), "one shape and dtype")
    _raises(lambda: binding.PagedCache(k.float(), k.float()), "k: dtype")
    _raises(lambda: binding.PagedCache(k.transpose(2, 3), k.transpose(2, 3)), "last dimension must be contiguous")
    _raises(lambda: binding.PagedCache(k, k), "must be on the CUDA device")


def test_qk_norm_rope():
    c = _ctx()
    Q, K = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64))
    pos, cs = torch.zeros(3, dtype=i32), torch.zeros((9, 32))
    f = lambda Q=Q, K=K, pos=pos, cs=cs, **kw: c.qk_norm_rope(Q, K, pos, cs, **kw)   # noqa: E731
    _raises(lambda: f(Q=None, K=None), "must be given")
    _raises(lambda: f(Q=Q.double()), "dtype")
    _raises(lambda: f(K=K.half()), "K: dtype")
    _raises(lambda: f(K=K[:2]), "K: shape")
    _raises(lambda: f(Q=Q[0]), "must be given")
    _raises(lambda: f(Q=torch.zeros((3, 64, 4)).transpose(1, 2)), "Q: the last dimension")
    _raises(lambda: f(Q_out=Q.half()), "Q_out: dtype")
    _raises(lambda: f(K_out=K[:, :1]), "K_out: shape")
    _raises(lambda: f(Q=None, Q_out=Q), "Q_out or a weight without Q")
    _raises(lambda: f(q_weight=torch.zeros(32)), "Q_weight: shape")
    _raises(lambda: f(q_weight=torch.zeros(64), norm=False), "a weight without the norm")
    _raises(lambda: f(pos=None), "cos_sin without positions")
    _raises(lambda: f(pos=pos.long()), "positions: dtype")
    _raises(lambda: f(pos=pos[:2]), "positions: shape")
    _raises(lambda: f(cs=None), "positions without cos_sin")
    _raises(lambda: f(cs=cs.double()), "cos_sin: dtype")
    _raises(lambda: f(cs=cs[:, ::2]), "cos_sin: must be contiguous")
    _raises(lambda: f(), "must be on the CUDA device")


def _batch(B=3, W=4):
    return torch.zeros((B, W), dtype=i32), torch.zeros(B, dtype=i32)


def test_append():
    c, cache = _ctx(), _cache()
    K = torch.zeros((3, 2, 64), dtype=torch.float16)
    tab, n = _batch()
    f = lambda K=K, V=K, tab=tab, n=n, **kw: c.paged_append(cache, tab, n, K, V, **kw)   # noqa: E731
    _raises(lambda: f(K=K[:, :1]), "K must be")
    _raises(lambda: f(K=K.bfloat16()), "K: dtype")
    _raises(lambda: f(V=K[:2]), "V: shape")
    _raises(lambda: f(V=K.float()), "V: dtype")
    _raises(lambda: f(Q=K[:2]), "Q: shape")
    _raises(lambda: f(Q=K, Q_out=K.float()), "Q_out: dtype")
    _raises(lambda: f(Q_out=K), "without Q")
    _raises(lambda: f(q_weight=K[0, 0]), "without Q")
    _raises(lambda: f(k_weight=K[0, 0], norm=False), "a weight without the norm")
    _raises(lambda: f(k_weight=K[0, 0].float()), "k_weight: dtype")
    _raises(lambda: f(positions=n), "positions without cos_sin")
    _raises(lambda: f(tab=tab.long()), "table: dtype")
    _raises(lambda: f(tab=tab[:2]), "table: shape")
    _raises(lambda: f(tab=torch.zeros((4, 3), dtype=i32).t()), "table: must be contiguous")
    _raises(lambda: f(n=n[:2], tab=tab[:2]), "cu_rows is needed")
    _raises(lambda: f(n=n.long()), "kv_len: dtype")
    _raises(lambda: f(cu_rows=n), "cu_rows: shape")
    _raises(lambda: f(), "must be on the CUDA device")
    _raises(lambda: c.paged_append(_cache(device=torch.device("cuda", 1)), tab, n, K, K), "cache: must be on the CUDA device")


def test_attend():
    c, cache = _ctx(), _cache()
    Q = torch.zeros((3, 4, 64), dtype=torch.float16)
    tab, n = _batch()
    lse = torch.zeros((3, 4))
    f = lambda Q=Q, tab=tab, n=n, **kw: c.paged_attend(cache, tab, n, Q, **kw)   # noqa: E731
    _raises(lambda: f(Q=Q[..., :32]), "Q must be")
    _raises(lambda: f(Q=Q.float()), "Q: dtype")
    _raises(lambda: f(O=Q.float()), "O: dtype")
    _raises(lambda: f(O=Q[:2]), "O: shape")
    _raises(lambda: f(O=torch.zeros((4, 3, 64), dtype=torch.float16).transpose(0, 1)), "O: must be contiguous")
    _raises(lambda: f(LSE=lse.half()), "LSE: dtype")
    _raises(lambda: f(LSE=lse.t()), "LSE: shape")
    _raises(lambda: f(prior=(Q, lse)), "prior O: dtype")
    _raises(lambda: f(prior=(Q.float(), lse[:2])), "prior LSE: shape")
    _raises(lambda: f(n=n[:2], tab=tab[:2]), "cu_rows is needed")
    _raises(lambda: f(), "must be on the CUDA device")


def test_packed_arguments_match_the_header(tmp_path):
    """The formats in which the binding writes pck_rows and pck_rotary, and its structures, against the C compiler's."""
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pck.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu ", offsetof({t}, {f}));\n' for t, fs in (
                       ("pck_rows", "in out H in_row in_head out_row out_head weight"),
                       ("pck_rotary", "cos_sin n_pos R interleaved positions"),
                       ("pck_paged_cache", "K V dtype H_kv D page_size n_pages k_page k_head k_token v_page v_head v_token"),
                       ("pck_paged_batch", "B T cu_rows kv_len table max_pages max_rows")) for f in fs.split())
                   + 'printf("%zu %zu %zu %zu", sizeof(pck_rows), sizeof(pck_rotary), sizeof(pck_paged_cache), sizeof(pck_paged_batch));\nreturn 0;\n}\n')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()]
    rows, rot = [0, 8, 16, 24, 32, 40, 48, 56], [0, 8, 12, 16, 24]
    structs = [getattr(t, n).offset for t in (binding.PagedCacheT, binding.PagedBatchT) for n, *_ in t._fields_]
    assert got == rows + rot + structs + [binding._ROWS.size, binding._ROTARY.size, ctypes.sizeof(binding.PagedCacheT), ctypes.sizeof(binding.PagedBatchT)]
    assert binding._ROWS.unpack(binding._ROWS.pack(*range(1, 9))) == tuple(range(1, 9))
    at = binding._ROWS.pack(1, 2, 3, 4, 5, 6, 7, 8)
    assert [int.from_bytes(at[o:o + (4 if o == 16 else 8)], "little") for o in rows] == list(range(1, 9))
    at = binding._ROTARY.pack(1, 2, 3, 4, 5)
    assert [int.from_bytes(at[o:o + (4 if o in (8, 12, 16) else 8)], "little") for o in rot] == list(range(1, 6))
