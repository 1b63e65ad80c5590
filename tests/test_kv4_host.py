"""The paged 4-bit cache without a GPU: its format against exact arithmetic, and the calls that are refused."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import kv4_reference as R
from block_discrete_diffusion_b200 import build, dg


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dg.lib()


def test_reference_rounding_is_nearest_even_in_exact_arithmetic():
    rng = np.random.default_rng(0)
    levels = [Fraction(float(v)) for v in R.LEVELS]
    scales = [Fraction(float(v)) for v in R.scale_value(np.arange(227))]
    rows = rng.standard_normal((40, 16)) * np.exp2(rng.integers(-18, 14, (40, 1)))
    rows = (rows.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)   # bf16 values
    rows[0] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]       # ties
    code, byte = R.quantise(rows)

    def best(x, grid):
        i = min(range(len(grid)), key=lambda i: (abs(grid[i] - x), i % 2))
        return i

    for x, c, b in zip(rows, code, byte):
        exact = [Fraction(float(v)) for v in x]
        want = best(max(abs(v) for v in exact) / 6, scales)
        assert b[0] == want
        for v, got in zip(exact, c):
            i = best(abs(v) / scales[want], levels) if scales[want] else 0
            assert got & 7 == i and (got >= 8) == (v < 0)


@pytest.mark.parametrize("dh", [64, 128])
def test_layout_is_a_bijection(dh):
    for (byte, shift, scale), base in zip(R.grids(dh), (0, 32 * dh)):
        assert len(set((2 * byte + shift // 4).ravel())) == 64 * dh
        assert byte.min() == base and byte.max() == base + 32 * dh - 1
        assert len(set(scale.ravel())) == 4 * dh
    assert R.grids(dh)[0][2].min() == 64 * dh and R.grids(dh)[1][2].max() == 72 * dh - 1


def test_book_rules():
    b = R.Book(3, 8, 4)
    assert b.extend([70, 0, 0]) == [] and b.table[0][:2] == [0, 1]
    assert b.fork([0], [1]) and b.refs[:2] == [2, 2]
    assert b.extend([1, 1, 0]) == [(1, 2), (1, 3)] and b.refs[:4] == [2, 0, 1, 1]
    assert b.free([0]) and b.compact() == [(3, 1)] and b.table[1][:2] == [0, 1]


def cache(**kw):
    c = dict(n_layers=2, n_kv=2, d_head=64, n_pages=5, n_seq=3, max_pages=4)
    c.update(kw)
    c = dg.dg_kv4_cache_t(*(c[k] for k in ("n_layers", "n_kv", "d_head", "n_pages", "n_seq", "max_pages")), 4096, 1 << 40,
                          8192, 1 << 40)
    return c


def test_sizes(lib):
    c = cache()
    assert dg.dg_kv4_pool_bytes(c) == 2 * 5 * 2 * 72 * 64
    assert dg.dg_kv4_book_bytes(c) == 4 * (16 + 4 + 4 * 8 + 12)
    assert lib.dg_kv4_attend_workspace_bytes(ctypes.byref(c), 3, 1) == 0


SHAPES = [dict(d_head=96), dict(n_kv=0), dict(n_layers=-1), dict(n_seq=4097), dict(n_pages=(1 << 24) + 1),
          dict(n_seq=4096, max_pages=1 << 18), dict(n_seq=4096, n_kv=16)]


@pytest.mark.parametrize("kw", SHAPES)
def test_shapes_refused(lib, kw):
    c = cache(**kw)
    assert dg.dg_kv4_pool_bytes(c) == 0 and dg.dg_kv4_book_bytes(c) == 0
    assert lib.dg_kv4_init(ctypes.byref(c), None) == dg.DG_ERR_INVALID_ARG
    assert b"dg_kv4_init" in lib.dg_last_error()


def test_buffers_refused(lib):
    for name, v, st in (("d_pool", None, dg.DG_ERR_INVALID_ARG), ("d_book", 8200, dg.DG_ERR_INVALID_ARG),
                        ("pool_bytes", 100, dg.DG_ERR_CAPACITY), ("book_bytes", 100, dg.DG_ERR_CAPACITY)):
        c = cache()
        setattr(c, name, v)
        r = ctypes.byref(c)
        rows = dg.dg_kv4_rows(4096, 4096, 128, 128, 64, 128, 128, 64, None, 1, 0)
        attn = dg.dg_kv4_attn(4096, 4096, None, None, 256, 256, 64, 256, 256, 64, 4, 1, 0, 0, 1.0)
        code = ctypes.c_int()
        for got in (lib.dg_kv4_init(r, None), lib.dg_kv4_extend(r, 4096, None), lib.dg_kv4_fork(r, 4096, 4096, 1, None),
                    lib.dg_kv4_free(r, 4096, 1, None), lib.dg_kv4_compact(r, None),
                    lib.dg_kv4_append(r, 0, ctypes.byref(rows), None), lib.dg_kv4_read(r, 0, ctypes.byref(rows), None),
                    lib.dg_kv4_attend(r, 0, ctypes.byref(attn), 4096, 1 << 40, None),
                    lib.dg_kv4_error(r, None, ctypes.byref(code))):
            assert got == st
    assert lib.dg_kv4_init(None, None) == dg.DG_ERR_INVALID_ARG


def test_page_calls_refused(lib):
    c = cache()
    r = ctypes.byref(c)
    bad = dg.DG_ERR_INVALID_ARG
    assert lib.dg_kv4_extend(r, None, None) == bad
    assert lib.dg_kv4_fork(r, None, 4096, 1, None) == bad and lib.dg_kv4_fork(r, 4096, 4096, 4, None) == bad
    assert lib.dg_kv4_free(r, 4096, 0, None) == bad and lib.dg_kv4_free(r, None, 1, None) == bad
    assert lib.dg_kv4_error(r, None, None) == bad


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=4100), dict(k_row=4), dict(v_head=60), dict(rows=0), dict(dtype=2),
                                dict(layer=2), dict(layer=-1)])
def test_rows_refused(lib, kw):
    a = dict(k=4096, v=4096, k_seq=128, k_row=128, k_head=64, v_seq=128, v_row=128, v_head=64, d_rows=None, rows=1, dtype=0)
    layer = kw.get("layer", 0)
    a.update({k: v for k, v in kw.items() if k != "layer"})
    rows = dg.dg_kv4_rows(*a.values())
    for fn in (lib.dg_kv4_append, lib.dg_kv4_read):
        assert fn(ctypes.byref(cache()), layer, ctypes.byref(rows), None) == dg.DG_ERR_INVALID_ARG
    assert lib.dg_kv4_append(ctypes.byref(cache()), 0, None, None) == dg.DG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=4104), dict(q_row=12), dict(o_seq=1), dict(n_q=3), dict(n_q=0),
                                dict(rows=0), dict(rows=65537), dict(dtype=5), dict(causal=2), dict(scale=0.0),
                                dict(scale=float("nan")), dict(scale=float("inf")), dict(layer=2),
                                dict(ws=None), dict(ws_bytes=10)])
def test_attend_refused(lib, kw):
    a = dict(q=4096, out=4096, lse=None, d_rows=None, q_seq=256, q_row=256, q_head=64, o_seq=256, o_row=256, o_head=64,
             n_q=4, rows=1, dtype=0, causal=0, scale=1.0)
    a.update({k: v for k, v in kw.items() if k in a})
    attn = dg.dg_kv4_attn(*a.values())
    want = dg.DG_ERR_CAPACITY if "ws" in kw or "ws_bytes" in kw else dg.DG_ERR_INVALID_ARG
    assert lib.dg_kv4_attend(ctypes.byref(cache()), kw.get("layer", 0), ctypes.byref(attn), kw.get("ws", 4096),
                             kw.get("ws_bytes", 1 << 40), None) == want
    assert b"dg_kv4_attend" in lib.dg_last_error()


def test_binding_structs_match_the_header_layout(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = {"dg_kv4_cache": dg.dg_kv4_cache_t, "dg_kv4_rows": dg.dg_kv4_rows, "dg_kv4_attn": dg.dg_kv4_attn}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dg.h"', "int main(void) {"]
    for name, s in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c99", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, value = line.split()
        s = structs[name]
        assert int(value) == (ctypes.sizeof(s) if field == "size" else getattr(s, field).offset), line


def test_prefix_calls_refused(lib):
    c = cache()
    assert lib.dg_store_prefix_kv4(None, 0, ctypes.byref(c), 0) == dg.DG_ERR_INVALID_ARG
    assert lib.dg_load_prefix_kv4(None, 0, 1, ctypes.byref(c), 0) == dg.DG_ERR_INVALID_ARG
    assert b"dg_load_prefix_kv4" in lib.dg_last_error()
