"""CPU tests of the paged cache: the oracle's pins (hand-worked plans, codes and blocks), the
C layout of the parameter structs, and every refusal that is decided before a launch."""
import ctypes
import math
import pathlib
import subprocess

import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
from head_rank_attention_b200 import _binding as B
from oracle import paged

ROOT = pathlib.Path(__file__).resolve().parents[1]


# ------------------------------------------------------------------------------- oracle
def test_plan_by_hand():
    """Pages of 32: sequence 0 crosses into a new page, 1 ends (two pages back), 2 starts."""
    table = np.array([[7, -1, -1], [3, 4, -1], [-1, -1, -1]])
    ring = np.array([5, 6, -9, -9, -9, 0, 1, 2])  # free: 0 1 2 5 6 at 5, 6, 7, 0, 1
    p = paged.page_plan([31, 40, 0], [3, -1, 33], table, ring, [5, 10], 32, 40)
    assert p["status"] == [0, 0, 0, 0]
    assert p["lens"].tolist() == [34, 0, 33]
    assert p["table"].tolist() == [[7, 0, -1], [3, 4, -1], [1, 2, -1]]
    assert p["ring"].tolist() == [5, 6, 3, 4, -9, 0, 1, 2]
    assert p["free"] == [8, 12]
    assert p["start"].tolist() == [0, 3, 3, 36]
    assert p["slots"][:4].tolist() == [7 * 32 + 31, 0, 1, 32] and p["slots"][35:].tolist() == [2 * 32, -1, -1, -1, -1]
    assert p["positions"][:4].tolist() == [31, 32, 33, 0] and p["positions"][35] == 32


@pytest.mark.parametrize("case,status", [
    (dict(lens=[-1, 0]), [1, 0, 0, 0]),
    (dict(lens=[0, 65]), [1, 1, 0, 0]),
    (dict(lens=[0, 60], new=[1, 5]), [2, 1, 0, 0]),
    (dict(new=[9, 9]), [3, 0, 18, 16]),
    (dict(lens=[32, 0], free=[3, 4], new=[1, 2]), [4, 0, 2, 1]),
    (dict(free=[4, 3]), [5, 0, 0, 0]),
    (dict(lens=[64, 0], new=[-1, 0], free=[0, 3]), [5, 0, 0, 0]),  # more pages back than are out
])
def test_plan_refusals(case, status):
    a = dict(lens=[0, 0], new=[1, 1], free=[0, 4])
    a.update(case)
    p = paged.page_plan(a["lens"], a["new"], np.zeros((2, 2), int), np.arange(4), a["free"], 32, 16)
    assert p["status"] == status and (p["slots"] == -1).all() and p["lens"].tolist() == a["lens"]


def test_nearest_codes():
    """int8: halves to even; e4m3: the numbers themselves, and torch's cast of fp32 values."""
    assert paged.nearest([0.5, 1.5, -2.5, 126.5, 127.4, -300.0], "int8").tolist() == [0, 2, -2, 126, 127, -127]
    grid = paged.e4m3_values()
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(grid, every)
    assert np.array_equal(paged.nearest(-grid, "e4m3"), -grid)
    half = (grid[1:] + grid[:-1]) / 2
    y = np.concatenate([half, np.nextafter(half.astype(np.float32), np.float32(0)), np.linspace(0, 448, 9999)])
    cast = torch.tensor(y, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.nearest(y.astype(np.float32), "e4m3"), cast)


def test_a_block_grows():
    """127 under scale 1 becomes 64 under 2 (63.5 to even); a smaller token leaves the scale."""
    codes = np.zeros((4, 128))
    x = np.zeros((1, 128))
    x[0, 0] = 127.0
    codes, s = paged.append_block(codes, 9.0, x, [0], "int8")
    assert s == 1.0 and codes[0, 0] == 127
    x[0, 0] = 254.0
    codes, s = paged.append_block(codes, s, x, [1], "int8")
    assert s == 2.0 and codes[0, 0] == 64 and codes[1, 0] == 127
    x[0, 0] = 3.0
    codes, s = paged.append_block(codes, s, x, [2], "int8")
    assert s == 2.0 and codes[2, 0] == 2  # 1.5 to even


# ------------------------------------------------------------------------- layout, refusals
@pytest.mark.parametrize("cls,ctype", [(B.HraPlanParams, "hra_plan_params"), (B.HraAppendParams, "hra_append_params"),
                                       (B.HraLoadParams, "hra_load_params")])
def test_params_layout_matches_c(tmp_path, cls, ctype):
    fields = [f[0] for f in cls._fields_]
    prog = tmp_path / "layout.c"
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "hra.h"', 'int main(void) {',
             f'  printf("size %zu\\n", sizeof({ctype}));']
    lines += [f'  printf("{f} %zu\\n", offsetof({ctype}, {f}));' for f in fields]
    prog.write_text("\n".join(lines + ['  return 0;', '}']))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", f"-I{ROOT / 'include'}", str(prog), "-o", str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(out[f]) == getattr(cls, f).offset, f


def _plan(**over):
    """Well-formed parameters with fake device pointers that nothing reads."""
    p = B.HraPlanParams()
    p.batch, p.page_size, p.max_pages, p.num_pages, p.max_tokens = 4, 64, 16, 64, 32
    for k, name in enumerate(("seq_lens", "new_tokens", "block_table", "free_pages", "free_range", "seq_lens_out",
                              "free_range_out", "query_start", "slots", "positions", "status")):
        setattr(p, name, 0x10000 * (k + 1))
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), B.HRA_ERR_UNSUPPORTED), (dict(batch=1025), B.HRA_ERR_UNSUPPORTED),
    (dict(page_size=0), B.HRA_ERR_UNSUPPORTED), (dict(page_size=48), B.HRA_ERR_UNSUPPORTED),
    (dict(max_pages=0), B.HRA_ERR_INVALID_ARG), (dict(num_pages=0), B.HRA_ERR_INVALID_ARG),
    (dict(max_tokens=0), B.HRA_ERR_INVALID_ARG), (dict(max_tokens=2**30 + 1), B.HRA_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 26), B.HRA_ERR_UNSUPPORTED), (dict(num_pages=1 << 26), B.HRA_ERR_UNSUPPORTED),
    (dict(batch=1024, max_pages=1 << 21), B.HRA_ERR_UNSUPPORTED),
    (dict(seq_lens=0), B.HRA_ERR_INVALID_ARG), (dict(slots=0), B.HRA_ERR_INVALID_ARG),
    (dict(status=0), B.HRA_ERR_INVALID_ARG), (dict(free_range=0x10004), B.HRA_ERR_INVALID_ARG),
    (dict(positions=0x10002), B.HRA_ERR_INVALID_ARG),
])
def test_plan_rejects_before_launch(over, status):
    assert hra.load_library().hra_page_plan(ctypes.byref(_plan(**over)), None) == status
    assert hra.last_error() != ""


def _append(**over):
    p = B.HraAppendParams()
    p.n_tokens, p.d_c, p.d_rope = 8, 512, 64
    p.latent, p.krope_in, p.slots, p.positions = 0x10000, 0x20000, 0x30000, 0x40000
    p.latent_stride, p.krope_in_stride, p.rope_theta = 576, 576, 10000.0
    p.ckv, p.krope, p.ckv_stride, p.krope_stride, p.cache_rows = 0x50000, 0x60000, 512, 64, 1024
    p.cache_dtype, p.ckv_scale, p.ckv_scale_stride, p.scale_block = B.HRA_INT8, 0x70000, 4, 64
    for k, v in over.items():
        setattr(p, k, v)
    return p


CACHE_REFUSALS = [
    (dict(d_c=384), B.HRA_ERR_UNSUPPORTED), (dict(d_rope=32), B.HRA_ERR_UNSUPPORTED),
    (dict(ckv=0), B.HRA_ERR_INVALID_ARG), (dict(ckv=0x50008), B.HRA_ERR_INVALID_ARG),
    (dict(krope=0x60008), B.HRA_ERR_INVALID_ARG),
    (dict(ckv_stride=504), B.HRA_ERR_INVALID_ARG), (dict(ckv_stride=520), B.HRA_ERR_INVALID_ARG),
    (dict(krope_stride=60), B.HRA_ERR_INVALID_ARG), (dict(krope_stride=68), B.HRA_ERR_INVALID_ARG),
    (dict(cache_rows=0), B.HRA_ERR_INVALID_ARG), (dict(cache_rows=1 << 31), B.HRA_ERR_INVALID_ARG),
    (dict(cache_dtype=B.HRA_F32), B.HRA_ERR_INVALID_ARG),
    (dict(cache_dtype=B.HRA_BF16), B.HRA_ERR_INVALID_ARG),                     # scale_block without scales
    (dict(ckv_scale=0), B.HRA_ERR_INVALID_ARG), (dict(ckv_scale=0x70002), B.HRA_ERR_INVALID_ARG),
    (dict(ckv_scale_stride=3), B.HRA_ERR_INVALID_ARG),
    (dict(scale_block=48), B.HRA_ERR_UNSUPPORTED), (dict(scale_block=2048), B.HRA_ERR_UNSUPPORTED),
    (dict(scale_block=-1), B.HRA_ERR_UNSUPPORTED),
    (dict(cache_dtype=B.HRA_E4M3, scale_block=1), B.HRA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", CACHE_REFUSALS + [
    (dict(n_tokens=0), B.HRA_ERR_INVALID_ARG), (dict(n_tokens=2**31 - 1), B.HRA_ERR_UNSUPPORTED),
    (dict(latent=0), B.HRA_ERR_INVALID_ARG), (dict(krope_in=0x20008), B.HRA_ERR_INVALID_ARG),
    (dict(slots=0), B.HRA_ERR_INVALID_ARG), (dict(positions=0), B.HRA_ERR_INVALID_ARG),
    (dict(latent_stride=508), B.HRA_ERR_INVALID_ARG), (dict(krope_in_stride=60), B.HRA_ERR_INVALID_ARG),
    (dict(rows_out=0x80008, rows_out_stride=576), B.HRA_ERR_INVALID_ARG),
    (dict(rows_out=0x80000, rows_out_stride=568), B.HRA_ERR_INVALID_ARG),
    (dict(rope_theta=0.0), B.HRA_ERR_INVALID_ARG), (dict(rope_theta=math.inf), B.HRA_ERR_INVALID_ARG),
])
def test_append_rejects_before_launch(over, status):
    assert hra.load_library().hra_cache_append(ctypes.byref(_append(**over)), None) == status
    assert hra.last_error() != ""


def _load(**over):
    p = B.HraLoadParams()
    p.batch, p.max_tokens, p.d_c, p.d_rope = 2, 128, 512, 64
    p.ckv, p.krope, p.ckv_stride, p.krope_stride, p.cache_rows = 0x50000, 0x60000, 512, 64, 1024
    p.cache_dtype, p.ckv_scale, p.ckv_scale_stride, p.scale_block = B.HRA_INT8, 0x70000, 4, 64
    p.seq_lens, p.block_table, p.max_pages, p.page_size = 0x10000, 0x20000, 4, 64
    p.out, p.out_stride, p.out_seq_stride = 0x90000, 576, 576 * 128
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status", CACHE_REFUSALS + [
    (dict(batch=0), B.HRA_ERR_UNSUPPORTED), (dict(batch=1025), B.HRA_ERR_UNSUPPORTED),
    (dict(max_tokens=0), B.HRA_ERR_INVALID_ARG), (dict(max_tokens=2**31 - 1), B.HRA_ERR_UNSUPPORTED),
    (dict(seq_lens=0), B.HRA_ERR_INVALID_ARG),
    (dict(out=0), B.HRA_ERR_INVALID_ARG), (dict(out=0x90008), B.HRA_ERR_INVALID_ARG),
    (dict(page_size=40), B.HRA_ERR_UNSUPPORTED), (dict(max_pages=0), B.HRA_ERR_INVALID_ARG),
    (dict(block_table=0, seq_stride=-1), B.HRA_ERR_INVALID_ARG),
    (dict(out_stride=512), B.HRA_ERR_INVALID_ARG), (dict(out_stride=580), B.HRA_ERR_INVALID_ARG),
    (dict(out_seq_stride=-8), B.HRA_ERR_INVALID_ARG), (dict(out_seq_stride=4), B.HRA_ERR_INVALID_ARG),
])
def test_load_rejects_before_launch(over, status):
    assert hra.load_library().hra_cache_load(ctypes.byref(_load(**over)), None) == status
    assert hra.last_error() != ""


def _decode(**over):
    p = B.HraDecodeParams()
    p.batch, p.num_heads, p.n_branch = 2, 128, 4
    p.d_c, p.d_rope, p.d_nope, p.d_v = 512, 64, 128, 128
    p.q, p.ckv, p.krope, p.seq_lens = 0x10000, 0x20000, 0x30000, 0x40000
    p.w_uk, p.w_uv, p.out = 0x50000, 0x60000, 0x70000
    p.ckv_stride, p.krope_stride, p.cache_rows, p.seq_stride = 512, 64, 4096, 2048
    p.alpha_q = p.alpha_kv = 1.0
    p.branch_scale, p.rope_theta, p.out_dtype, p.num_splits = 0.5, 10000.0, B.HRA_F32, 37
    p.cache_dtype, p.ckv_scale, p.ckv_scale_stride, p.scale_block = B.HRA_INT8, 0x80000, 4, 64
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status", [
    (dict(scale_block=48), B.HRA_ERR_UNSUPPORTED), (dict(scale_block=2048), B.HRA_ERR_UNSUPPORTED),
    (dict(scale_block=-1), B.HRA_ERR_UNSUPPORTED),
    (dict(cache_dtype=B.HRA_E4M3, scale_block=0), B.HRA_ERR_UNSUPPORTED),
    (dict(cache_dtype=B.HRA_BF16), B.HRA_ERR_INVALID_ARG),
    (dict(n_branch=1), B.HRA_ERR_UNSUPPORTED), (dict(n_branch=2), B.HRA_ERR_UNSUPPORTED),  # wider branches
    (dict(seq_stride=2000), B.HRA_ERR_INVALID_ARG),                          # a block of two sequences' rows
    (dict(block_table=0x90000, max_pages=4, page_size=32), B.HRA_ERR_INVALID_ARG),
    (dict(block_table=0x90000, max_pages=4, page_size=96), B.HRA_ERR_INVALID_ARG),
    (dict(ckv_scale=0), B.HRA_ERR_INVALID_ARG), (dict(ckv_scale_stride=3), B.HRA_ERR_INVALID_ARG),
    (dict(ckv_stride=520), B.HRA_ERR_INVALID_ARG),
    (dict(), B.HRA_ERR_WORKSPACE),                                             # well formed but for the workspace
    (dict(cache_dtype=B.HRA_E4M3), B.HRA_ERR_WORKSPACE),
    (dict(batch=1, seq_stride=1000), B.HRA_ERR_WORKSPACE),
])
def test_block_scaled_decode_rejects_before_launch(over, status):
    p = _decode(**over)
    for entry in ("mlra_decode",):
        assert getattr(hra.load_library(), entry)(ctypes.byref(p), None) == status, hra.last_error()
        assert hra.last_error() != ""


def test_binding_checks_tensors():
    """Shapes, types and strides that a pointer cannot show are refused in the binding."""
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    good = dict(seq_lens=i32(2), new_tokens=i32(2), block_table=i32(2, 4), free_pages=i32(8),
                free_range=torch.zeros(2, dtype=torch.int64), seq_lens_out=i32(2),
                free_range_out=torch.zeros(2, dtype=torch.int64), query_start=i32(3), slots=i32(5), status=i32(4),
                page_size=64)
    hra.make_plan_params(**good)
    for bad in (dict(new_tokens=i32(3)), dict(seq_lens=torch.zeros(2, dtype=torch.int64)), dict(block_table=i32(4, 2).t()),
                dict(free_range=i32(2)), dict(query_start=i32(2)), dict(positions=i32(4)), dict(status=i32(2))):
        with pytest.raises(ValueError):
            hra.make_plan_params(**{**good, **bad})
    bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    ap = dict(latent=bf(5, 256), krope_in=bf(5, 64), slots=i32(5), positions=i32(5),
              ckv=torch.zeros(64, 256, dtype=torch.int8), krope=bf(64, 64), ckv_scale=torch.zeros(2, 2), scale_block=32)
    hra.make_append_params(**ap)
    for bad in (dict(latent=bf(5, 512)), dict(krope_in=bf(4, 64)), dict(slots=i32(4)), dict(positions=i32(6)),
                dict(ckv=torch.zeros(64, 256)), dict(krope=bf(63, 64)), dict(ckv_scale=None),
                dict(ckv_scale=torch.zeros(1, 2)), dict(ckv_scale=torch.zeros(2, 1)), dict(rows_out=bf(5, 256)),
                dict(ckv_scale=torch.zeros(2, 2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            hra.make_append_params(**{**ap, **bad})
    ld = dict(ckv=ap["ckv"], krope=ap["krope"], seq_lens=i32(2), out=bf(2, 7, 320), ckv_scale=ap["ckv_scale"], scale_block=32)
    hra.make_load_params(**ld)
    for bad in (dict(out=bf(2, 7, 256)), dict(out=bf(1, 7, 320)), dict(out=bf(14, 320)), dict(block_table=i32(1, 4)),
                dict(seq_lens=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            hra.make_load_params(**{**ld, **bad})


def test_launches_need_their_tensors_on_the_current_device():
    """Tensors in host memory, or on several devices, are refused before any launch."""
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    i64 = torch.zeros(2, dtype=torch.int64)
    plan = hra.make_plan_params(i32(2), i32(2), i32(2, 4), i32(8), i64, i32(2), i64.clone(), i32(3), i32(5), i32(4), page_size=64)
    put = hra.make_append_params(bf(5, 128), bf(5, 64), i32(5), i32(5), bf(64, 128), bf(64, 64))
    load = hra.make_load_params(bf(64, 128), bf(64, 64), i32(1), bf(1, 7, 192), seq_stride=64)
    for call, p in ((hra.page_plan, plan), (hra.check_plan_status, plan), (hra.cache_append, put), (hra.cache_load, load)):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call(p)
    with pytest.raises(ValueError, match="several devices"):
        hra.make_append_params(bf(5, 128), bf(5, 64), i32(5), i32(5), bf(64, 128).to("meta"), bf(64, 64))
