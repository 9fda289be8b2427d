"""CPU tests of the paged cache's edges: buffers that are too small for what a call would read or
write are refused in the binding, pages that are none of the pool in the plan, and a library of
another version's structs on loading."""
import pathlib
import re
import subprocess

import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
from head_rank_attention_b200 import _binding as B
from oracle import paged

BAD_SCALES = {
    "short": torch.zeros(63, 2), "block_sized": torch.zeros(2, 2), "narrow": torch.zeros(64, 1), "half": torch.zeros(64, 2).half(),
    "double": torch.zeros(64, 2).double(), "transposed": torch.zeros(2, 64).t(), "flat": torch.zeros(128),
    "deep": torch.zeros(64, 2, 1), "none": None,
}


def _bf(*n):
    return torch.zeros(*n, dtype=torch.bfloat16)


def _i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


@pytest.mark.parametrize("block", [0, 1])
@pytest.mark.parametrize("name", BAD_SCALES)
def test_scales_per_row_must_cover_the_cache(name, block):
    """A scale tensor that the append would write past, or that is not what the pointer would say."""
    ckv, krope, kw = torch.zeros(64, 256, dtype=torch.int8), _bf(64, 64), dict(ckv_scale=BAD_SCALES[name], scale_block=block)
    with pytest.raises(ValueError, match="ckv_scale"):
        hra.make_append_params(_bf(5, 256), _bf(5, 64), _i32(5), _i32(5), ckv, krope, **kw)
    with pytest.raises(ValueError, match="ckv_scale"):
        hra.make_load_params(ckv, krope, _i32(1), _bf(1, 7, 320), seq_stride=64, **kw)
    w = _bf(8, 256, 128)
    with pytest.raises(ValueError, match="ckv_scale"):
        hra.make_params(_bf(1, 8, 192), ckv, krope, _i32(1), w, w, _bf(1, 8, 128), n_branch=2, seq_stride=64, **kw)


@pytest.mark.parametrize("scale", [torch.zeros(64, 2), torch.zeros(70, 4)[:, 1:3], torch.zeros(64, 8)])
def test_scales_per_row_that_cover_it(scale):
    ckv, krope = torch.zeros(64, 256, dtype=torch.int8), _bf(64, 64)
    p = hra.make_append_params(_bf(5, 256), _bf(5, 64), _i32(5), _i32(5), ckv, krope, ckv_scale=scale)
    assert p.ckv_scale == scale.data_ptr() and p.ckv_scale_stride == scale.stride(0)
    p = hra.make_load_params(ckv, krope, _i32(1), _bf(1, 7, 320), seq_stride=64, ckv_scale=scale, scale_block=1)
    assert p.ckv_scale_stride == scale.stride(0)


def test_scales_of_a_branch_and_of_a_part_of_the_rows():
    """One branch's column, as a view or by itself; a decode that addresses fewer rows than the tensor has."""
    w, ckv = _bf(8, 128, 128), torch.zeros(64, 128, dtype=torch.int8)
    for scale in (torch.zeros(64, 4)[:, 2:3], torch.zeros(64)):
        hra.make_params(_bf(1, 8, 192), ckv, _bf(64, 64), _i32(1), w, w, _bf(1, 8, 128), n_branch=1, seq_stride=64, ckv_scale=scale)
    short = torch.zeros(40, 1)
    hra.make_params(_bf(1, 8, 192), ckv, _bf(64, 64), _i32(1), w, w, _bf(1, 8, 128), n_branch=1, seq_stride=64, ckv_scale=short,
                    cache_rows=40)
    with pytest.raises(ValueError, match="ckv_scale"):
        hra.make_params(_bf(1, 8, 192), ckv, _bf(64, 64), _i32(1), w, w, _bf(1, 8, 128), n_branch=1, seq_stride=64, ckv_scale=short)


@pytest.mark.parametrize("ring,status", [
    ([2, -1, 3, 0], [6, 0, 1, -1]), ([4, 0, 1, 2], [6, 0, 0, 4]), ([0, 1, 2, -9], [0, 0, 0, 0])])
def test_a_page_to_be_taken_that_is_none_of_the_pool(ring, status):
    """Three pages are taken of the four: a step that met a bad one is refused as a whole."""
    p = paged.page_plan([0, 31], [33, 2], np.array([[-1, -1], [7, -1]]), np.array(ring), [0, 4], 32, 64)
    assert p["status"] == status
    if status[0]:
        assert (p["slots"] == -1).all() and p["free"] == [0, 4] and p["lens"].tolist() == [0, 31]
        assert p["table"].tolist() == [[-1, -1], [7, -1]] and p["ring"].tolist() == ring


def test_versions_of_header_library_and_binding_agree(tmp_path, monkeypatch):
    header = (pathlib.Path(__file__).resolve().parents[1] / "include" / "hra.h").read_text()
    declared = re.search(r'#define HRA_VERSION "([^"]+)"', header).group(1)
    assert declared == B.HRA_VERSION and hra.version() == f"hra {declared} (sm_100a)"
    src, lib = tmp_path / "other.c", tmp_path / "libother.so"
    src.write_text('const char* hra_version(void) { return "hra 0.1.0 (sm_100a)"; }\n')
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    monkeypatch.setattr(B, "LIB_PATH", lib)
    monkeypatch.setattr(B, "_lib", None)
    with pytest.raises(ImportError, match="0.1.0"):
        B.load_library()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("growth", [0.0, 0.01, 0.3, 1.0])
def test_how_far_a_growing_block_takes_its_values(fmt, growth):
    """A block filled token by token, whose scale grows with nearly every token or not at all.  Every
    growth rounds the earlier codes again: an int8 value moves by half a step of the scale of the
    time, an e4m3 value by 2^-4 of itself or half a step of 2^-9 scales.  After g growths an int8
    value is within (g + 1) / 2 of the scale from its latent."""
    r = np.random.default_rng(17)
    n = 64
    x = r.standard_normal((n, 128)) * (1 + growth) ** np.arange(n)[:, None]
    codes, s, off, grown = np.zeros((n, 128)), np.float32(0), np.zeros((n, 128)), np.zeros(n)
    for t in range(n):
        before = s
        codes, s = paged.append_block(codes, s, x[t:t + 1], [t], fmt)
        rounded = slice(0, t + 1) if s > before else slice(t, t + 1)
        if s > before:
            grown[:t] += 1
        half = np.full_like(off[rounded], s / 2.0) if fmt == "int8" else np.maximum(
            2.0 ** -4 * (np.abs(x[rounded]) + off[rounded]), 2.0 ** -10 * s)
        off[rounded] += half
    err = np.abs(codes * np.float64(s) - x)
    # a scale is fl32(amax / top): the largest value may sit 2^-24 beyond the last code
    assert (err <= off + 2.0 ** -23 * np.abs(x)).all()
    assert grown.max() > (30 if growth >= 0.3 else 0)
    if fmt == "int8":
        assert (err <= ((grown + 1) / 2)[:, None] * s * (1 + 2.0 ** -20)).all()
