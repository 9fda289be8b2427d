"""Block-scaled decode at the edges of its scales: scales that are no numbers (the outputs of the
sequences that read them are no numbers on every path behind the decode kernel, and the others'
are untouched) and neighbouring blocks whose scales are far apart."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
import oracle
import synth
from gpu_cases import assert_parity
from oracle import paged
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


@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_zero_scales(zero):
    """Blocks of scale 0 of either sign, beside others and as all that a sequence has: their codes stand for 0."""
    wl = _case("zero", (300, 60), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    for s, c, b in ((0, 1, 2), (0, 4, 0), (1, 0, 3)):
        scale[int(inp.block_table[s, c]), b] = zero
    assert_parity(_run(inp, wl, codes, scale, 64), _oracle(inp, wl, codes, scale, 64), "zero scales")


# --------------------------------------------------------------------- scales far apart
def _far_blocks(B, L, apart, high):
    """A paged case of 32-row blocks whose latents are 2^high, 2^(high - apart), 2^high, ... in size."""
    wl = _case("far", (L,) * B, page_size=32)
    inp = synth.make_inputs(wl)
    block = torch.zeros(inp.cache.shape[0], dtype=torch.bool)  # rows of small blocks
    for s in range(B):
        for c in range(1, -(-L // 32), 2):
            page = int(inp.block_table[s, c])
            block[32 * page:32 * page + 32] = True
    size = torch.where(block, 2.0 ** (high - apart), 2.0 ** high)[:, None]
    inp.cache[:, :512] = (inp.cache[:, :512].double() * size).to(torch.bfloat16)
    return wl, inp, block


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("apart,high", [(12, 0), (20, 4), (28, 10), (28, 13)])
def test_weight_on_small_blocks_beside_large_ones(fmt, apart, high):
    """The large blocks' RoPE keys point away from every head's query (scores of -60), so the
    output is made of the small blocks' values, 2^-apart of their neighbours'."""
    wl, inp, small = _far_blocks(3, 333, apart, high)
    inp.q[..., :128] = (inp.q[..., :128].double() * 2.0 ** -high).to(torch.bfloat16)  # scores stay in the usual range
    for s in range(wl.batch):
        inp.q[s, :, 128:] = inp.q[s, :1, 128:]
        u = torch.tensor(oracle.rope_rotate(inp.q[s, 0, 128:].double().numpy(), 332, wl.rope_theta))
        at = torch.tensor(paged.cache_rows_of(333, s, inp.block_table.numpy(), 32, 0))
        at = at[~small[at]]
        inp.cache[at, 512:] = (-60 / wl.softmax_scale * u / (u @ u)).to(torch.bfloat16)
    codes, scale = _quantize(inp.cache[:, :512], 32, fmt)
    assert_parity(_run(inp, wl, codes, scale, 32), _oracle(inp, wl, codes, scale, 32), f"{fmt} 2^{apart} apart")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("apart", [6, 12, 17])
def test_resolution_beside_large_blocks(fmt, apart):
    """Equal weights on blocks 2^apart from one another, the small ones' values in columns that the
    large ones leave at zero: a weight times its block's unit sigma (f 2^E, the scale where that is
    at least 2^-8) is off by 2^-11 of itself or 2^-25 of the largest, and so is what it adds."""
    wl, inp, small = _far_blocks(2, 320, apart, 10)
    inp.q[:] = 0
    cols = torch.arange(512) % 128 < 64
    inp.cache[:, :512] = torch.where(small[:, None] == cols[None], 0.0, inp.cache[:, :512].float()).to(torch.bfloat16)
    codes, scale = _quantize(inp.cache[:, :512], 32, fmt)
    got, ref = _run(inp, wl, codes, scale, 32), _oracle(inp, wl, codes, scale, 32)
    w = np.abs(inp.w_uv.double().numpy())
    for s in range(wl.batch):
        at = paged.cache_rows_of(320, s, inp.block_table.numpy(), 32, 0)
        x = np.abs(paged.values(codes.float().double().numpy(), scale.numpy(), 32)[at])
        sigma = np.maximum(scale.double().numpy()[at // 32], 2.0 ** -8)
        off = 2.0 ** -11 * x + 2.0 ** -25 * x / np.repeat(sigma, 128, axis=1) * np.repeat(sigma.max(axis=0), 128)[None]
        # sums, exponentials and their arguments are in fp32, o_lat is hi + lo bf16: 2^-16 covers them
        bound = np.einsum("c,hcv->hv", off.mean(axis=0) + 2.0 ** -16 * x.mean(axis=0), w) * wl.alpha_kv * wl.sigma_o
        assert (np.abs(got[s] - ref[s]) <= bound).all()
