"""Block-scaled decode where its scales are no numbers: the outputs of the sequences that read
them are no numbers on every path behind the decode kernel, and the others' are untouched."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
import synth
from gpu_cases import assert_parity
from test_block_scaled_decode_gpu import _case, _oracle, _quantize, _run

pytestmark = pytest.mark.gpu


# Batch and heads choose the kernels that merge: up to 4 sequences with few heads the fused one,
# below 16 and from 16 sequences the two forms of the merge kernel.
@pytest.mark.parametrize("B,heads", [(2, 16), (4, 37), (2, 128), (5, 16), (16, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("length,block_at", [(300, 1), (40, 0), (64, 0), (1, 0)])
def test_a_bad_scale_reaches_its_sequence(B, heads, bad, length, block_at):
    """One bad block between good ones, or the only one of its sequence."""
    wl = _case("bad", (length,) + (200,) * (B - 1), heads=heads, page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    ref = _oracle(inp, wl, codes, scale, 64)
    scale[int(inp.block_table[0, block_at]), 2] = bad
    got = _run(inp, wl, codes, scale, 64)
    assert np.isnan(got[0]).all()
    assert_parity(got[1:], ref[1:], "the other sequences")


@pytest.mark.parametrize("heads", [16, 128])
def test_a_bad_scale_per_row_reaches_its_sequence(heads):
    """The same where every row has its own scale, for a row among good ones and for a sequence of one row."""
    wl = _case("bad_row", (200, 1, 90), heads=heads, page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 1, "int8")
    ref = _oracle(inp, wl, codes, scale, 1)
    table = inp.block_table
    scale[int(table[0, 2]) * 64 + 7, 1] = float("nan")
    scale[int(table[1, 0]) * 64, 3] = float("nan")
    got = _run(inp, wl, codes, scale, 0)
    assert np.isnan(got[:2]).all()
    assert_parity(got[2:], ref[2:], "the other sequence")


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("where", [0, 1])
def test_a_bad_scale_passes_the_combination_of_ranges(heads, where):
    """A sequence in two token ranges, one of them a bad block and nothing else: its state says so
    (an empty range's is -inf) and the combined output is no number; the second sequence's is right."""
    wl = _case("bad_range", (112, 112), heads=heads, page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "e4m3")
    ref = _oracle(inp, wl, codes, scale, 64)
    scale[int(inp.block_table[0, where]), 0] = float("nan")
    dev = synth.to_device(inp)
    cd, sd, krope = codes.cuda(), scale.cuda(), inp.cache[:, 512:].contiguous().cuda()
    pos = torch.full((2,), 111, dtype=torch.int32, device="cuda")
    po = torch.empty(3, 2, heads, 512, device="cuda")
    pl = torch.empty(3, 2, heads, 4, device="cuda")
    out = torch.empty(2, heads, 128, device="cuda")
    kw = dict(n_branch=4, branch_scale=wl.sigma_o, page_size=64, ckv_scale=sd, scale_block=64)
    keep = []
    for k, n in enumerate((64, 48, 0)):
        table = dev.block_table[:, min(k, 1):].contiguous()
        lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
        p = hra.make_params(dev.q, cd, krope, lens, dev.w_uk, dev.w_uv, None, block_table=table, q_positions=pos,
                            part_o=po[k], part_lse=pl[k], **kw)
        keep += [table, lens, hra.alloc_workspace(p)]
        hra.mlra_decode(p)
        hra.check_device_status(p)
    lse = pl.cpu().numpy()
    assert np.isnan(lse[where, 0, :, 0]).all() and np.isfinite(lse[where, 0, :, 1:]).all()
    assert np.isfinite(lse[1 - where]).all() and (lse[2] == -np.inf).all()
    p = hra.make_params(dev.q, cd, krope, lens, dev.w_uk, dev.w_uv, out, block_table=table, **kw)
    keep.append(hra.alloc_workspace(p))
    hra.combine_partials(p, po, pl)
    hra.check_device_status(p)
    got = out.cpu().numpy()
    assert np.isnan(got[0]).all()
    assert_parity(got[1:], ref[1:], "the other sequence")
    hra.combine_partials(p, po[2:], pl[2:])  # nothing but the empty range
    hra.check_device_status(p)
    assert (out == 0).all()
