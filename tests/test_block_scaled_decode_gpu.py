"""GPU parity of the decode over a cache held in 8 bits (int8 or e4m3) with one scale for each
block of tokens and 128-wide latent head, against the fp64 oracle on the values that the
cache stands for, and a serving loop that plans, appends, loads, prefills and decodes."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
import oracle
import synth
from gpu_cases import MAX_REL, MEAN_REL, assert_parity, parity
from oracle import paged

pytestmark = pytest.mark.gpu

DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _case(name, lengths, heads=128, page_size=0, **kw):
    return synth.Workload(name, 4, len(lengths), heads, max(lengths), page_size=page_size, lengths=tuple(lengths), **kw)


def _quantize(latent, block, fmt):
    """bf16 latents [rows, d_c] -> the format's tensor and fp32 scales [ceil(rows / block), d_c / 128]."""
    x = latent.double().numpy()
    rows, d_c = x.shape
    n = -(-rows // block)
    padded = np.zeros((n * block, d_c))
    padded[:rows] = x
    xb = padded.reshape(n, block, d_c // 128, 128)
    scale = paged.block_scale(np.abs(xb).max(axis=(1, 3)), fmt)
    s = np.where(scale > 0, scale, 1).astype(np.float64)[:, None, :, None]
    codes = paged.nearest(xb / s, fmt).reshape(n * block, d_c)[:rows]
    return torch.tensor(codes, dtype=torch.float32).to(DTYPE[fmt]), torch.tensor(scale)


def _poison(inp, wl, krope, codes, scale, block):
    """Rows that no sequence owns: RoPE part NaN, codes at their largest; blocks without an owned row: scale NaN."""
    used = np.zeros(krope.shape[0], dtype=bool)
    for s in range(wl.batch):
        used[paged.cache_rows_of(int(inp.seq_lens[s]), s, None if inp.block_table is None else inp.block_table.numpy(),
                                 wl.page_size or 1, inp.seq_stride)] = True
    u = torch.tensor(used)
    krope, scale = krope.clone(), scale.clone()
    krope[~u] = float("nan")
    codes.view(torch.uint8)[~u] = 0x7E  # 126, or 448
    touched = np.zeros(scale.shape[0], dtype=bool)
    touched[np.nonzero(used)[0] // block] = True
    scale[~torch.tensor(touched)] = float("nan")
    return krope, codes, scale


def _run(inp, wl, codes, scale, block, *, n_branch=4, cols=slice(0, 512), num_splits=0, out_dtype=torch.float32, krope=None,
         check=True, **kw):
    dev = synth.to_device(inp)
    krope = (inp.cache[:, 512:] if krope is None else krope).contiguous().cuda()
    g = slice(cols.start // 128, cols.stop // 128)
    ckv = codes.view(torch.uint8)[:, cols].contiguous().view(codes.dtype).cuda()
    w_uk, w_uv = dev.w_uk[:, cols].contiguous(), dev.w_uv[:, cols].contiguous()
    out = torch.empty(wl.batch, wl.heads, synth.D_V, dtype=out_dtype, device="cuda")
    p = hra.make_params(dev.q, ckv, krope, dev.seq_lens, w_uk, w_uv, out, n_branch=n_branch, alpha_q=wl.alpha_q,
                        alpha_kv=wl.alpha_kv, branch_scale=wl.sigma_o, softmax_scale=wl.softmax_scale, rope_theta=wl.rope_theta,
                        block_table=dev.block_table, page_size=wl.page_size, seq_stride=dev.seq_stride, num_splits=num_splits,
                        ckv_scale=scale.cuda()[:, g], scale_block=block, **kw)
    keep = (dev, krope, ckv, w_uk, w_uv, p.ckv_scale)
    sc = scale.cuda()
    p.ckv_scale = sc.data_ptr() + 4 * g.start
    ws = hra.alloc_workspace(p)
    ws.fill_(0xFF)
    hra.mlra_decode(p)
    if check:
        hra.check_device_status(p)
    torch.cuda.synchronize()
    del keep
    return out.float().cpu().numpy()


def _oracle(inp, wl, codes, scale, block):
    per_row = np.repeat(scale.numpy(), block, axis=0)[:codes.shape[0]]
    return oracle.decode_batch_int8(inp, wl, codes.float().double().numpy(), per_row)


CASES = [
    (_case("tails", (1, 31, 32, 33, 95, 96, 97, 127, 128, 129, 191, 192, 193, 1000)), 32),
    (_case("paged64", (5, 64, 65, 700), page_size=64), 64),
    (_case("paged64_b32", (96, 64, 257, 700), page_size=64), 32),
    (_case("paged32", (5, 64, 65, 700), page_size=32), 32),
    (_case("paged128", (300, 1, 256), page_size=128), 128),
    (_case("b1024", (1500,)), 1024),
    (_case("h16", (2048,), heads=16, alpha_q=2048 ** 0.5 / 1536 ** 0.5, alpha_kv=2.0, branch_scale=0.5), 64),
    (_case("h1", (70, 3), heads=1, page_size=64), 64),
    (_case("h40", (600, 97), heads=40, page_size=64), 64),
    (_case("h33", (3000,), heads=33), 96),
    (_case("stress", (3000, 17), alpha_q=synth.A_Q_V3, alpha_kv=synth.A_KV_V3, page_size=64), 64),
    (_case("outliers", (5000,), outlier_frac=0.01), 64),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("wl,block", CASES, ids=[c[0].name for c in CASES])
def test_block_scaled_decode_matches_the_oracle(wl, block, fmt):
    if wl.page_size == 0 and wl.batch > 1:  # contiguous sequences start on a block's first row
        wl = synth.Workload(**{**wl.__dict__, "seq_len": -(-wl.seq_len // block) * block})
    inp = synth.make_inputs(wl)
    if wl.page_size == 0 and wl.batch > 1 and inp.seq_stride % block:
        pad = -(-inp.seq_stride // block) * block
        cache = torch.zeros(wl.batch * pad, 576, dtype=torch.bfloat16)
        for s in range(wl.batch):
            cache[s * pad:s * pad + inp.seq_stride] = inp.cache[s * inp.seq_stride:(s + 1) * inp.seq_stride]
        inp.cache, inp.seq_stride = cache, pad
    codes, scale = _quantize(inp.cache[:, :512], block, fmt)
    ref = _oracle(inp, wl, codes, scale, block)
    krope, codes, scale = _poison(inp, wl, inp.cache[:, 512:], codes, scale, block)
    got = _run(inp, wl, codes, scale, block, krope=krope)
    assert_parity(got, ref, wl.name)


@pytest.mark.parametrize("num_splits", [1, 3, 200])
def test_split_counts(num_splits):
    wl = _case("splits", (1, 130, 2000, 64, 96, 97), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    assert_parity(_run(inp, wl, codes, scale, 64, num_splits=num_splits), _oracle(inp, wl, codes, scale, 64), f"splits={num_splits}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("world", [2, 4])
def test_branch_shards_sum_to_mlra4(fmt, world):
    """A rank holds its branches' columns and its columns of the scales (a strided view)."""
    wl = _case("shards", (1, 129, 1000), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 32, fmt)
    w = 512 // world
    total = sum(_run(inp, wl, codes, scale, 32, n_branch=4 // world, cols=slice(w * r, w * (r + 1))) for r in range(world))
    assert_parity(total, _oracle(inp, wl, codes, scale, 32), "shards")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 1.999, 2.0 ** 6])
def test_scales_of_any_size(fmt, size):
    """Blocks whose scales differ by powers of two and in every bit of their mantissa: the
    latents of a block are size * 2^k apart from its neighbours'; one block is zero."""
    wl = _case("sizes", (700, 333), page_size=64)
    inp = synth.make_inputs(wl)
    r = np.random.default_rng(7)
    factor = size * 2.0 ** r.integers(-4, 2, (inp.cache.shape[0] // 32, 1)) * r.uniform(1, 2, (inp.cache.shape[0] // 32, 1))
    factor[int(inp.block_table[0, 2]) * 2] = 0.0
    inp.cache[:, :512] = (inp.cache[:, :512].double() * torch.tensor(np.repeat(factor, 32, axis=0))).to(torch.bfloat16)
    codes, scale = _quantize(inp.cache[:, :512], 32, fmt)
    got, ref = _run(inp, wl, codes, scale, 32), _oracle(inp, wl, codes, scale, 32)
    max_rel, mean_rel = parity(got, ref)
    assert np.isfinite(got).all() and mean_rel <= MEAN_REL
    if size < 64:
        assert max_rel <= MAX_REL
    else:  # scores in the hundreds: what an fp16 query can move them by is no longer small
        assert (np.abs(got - ref) <= _fp16_bound(inp, wl, codes, scale, 32)).all()


def _fp16_bound(inp, wl, codes, scale, block):
    """How far rounding the query (and the RoPE key) to fp16, half a step of 2^-11 each, may
    move the output: a score moves by at most D = tau (2^-11 sum|q~||x| + 2^-10 sum|qr||kr|), so a
    softmax weight by a factor within e^(+-2D), and the output by at most (e^(2D) - 1) sum p|x||W|; P
    is rounded to fp16 as well."""
    tau, half = wl.softmax_scale, 2.0 ** -11
    w_uk, w_uv = inp.w_uk.double().numpy(), np.abs(inp.w_uv.double().numpy())
    bound = np.zeros((wl.batch, wl.heads, 128))
    for s in range(wl.batch):
        L = int(inp.seq_lens[s])
        at = paged.cache_rows_of(L, s, inp.block_table.numpy(), wl.page_size, 0)
        x = paged.values(codes.float().double().numpy(), scale.numpy(), block)[at]
        kr = inp.cache[:, 512:].double().numpy()[at]
        q = inp.q[s].double().numpy()
        qr = np.stack([oracle.rope_rotate(v, L - 1, wl.rope_theta) for v in q[:, 128:]])
        for b in range(4):
            c = slice(128 * b, 128 * b + 128)
            qt = np.einsum("hcn,hn->hc", w_uk[:, c], q[:, :128]) * wl.alpha_q * wl.alpha_kv
            D = tau * (half * np.abs(qt) @ np.abs(x[:, c]).T + 2 * half * np.abs(qr) @ np.abs(kr).T).max(axis=1)
            score = tau * (qt @ x[:, c].T + qr @ kr.T)
            pr = np.exp(score - score.max(axis=1, keepdims=True))
            pr /= pr.sum(axis=1, keepdims=True)
            mass = np.einsum("hc,hcv->hv", pr @ np.abs(x[:, c]), w_uv[:, c]) * wl.alpha_kv * wl.sigma_o
            bound[s] += (np.expm1(2 * D) + 2 * half)[:, None] * mass
    return bound


def test_empty_sequences_and_bf16_out():
    wl = _case("empty", (1, 200, 1, 65), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "e4m3")
    ref = _oracle(inp, wl, codes, scale, 64)
    inp.seq_lens[0] = inp.seq_lens[2] = 0
    got = _run(inp, wl, codes, scale, 64, out_dtype=torch.bfloat16)
    assert (got[[0, 2]] == 0).all()
    max_rel, mean_rel = parity(got[[1, 3]], ref[[1, 3]])
    assert max_rel <= MAX_REL and mean_rel <= MEAN_REL + 2.0 ** -8 / 2  # a uniform rounding averages half of its bound


def test_all_sequences_empty():
    wl = _case("none", (64, 64), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    inp.seq_lens[:] = 0
    assert (_run(inp, wl, codes, scale, 64) == 0).all()


def test_largest_batch():
    """1024 sequences of 1 to 130 tokens, few heads."""
    r = np.random.default_rng(9)
    wl = _case("b1024", tuple(int(n) for n in r.integers(1, 131, 1024)), heads=4, page_size=32)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 32, "e4m3")
    assert_parity(_run(inp, wl, codes, scale, 32), _oracle(inp, wl, codes, scale, 32), "1024 sequences")


def test_large_rope_keys_and_queries():
    """RoPE keys in the hundreds against small latents, and the reverse: the one divided by the
    tile's scale, the other times it, within fp16."""
    wl = _case("rope", (500, 97), page_size=64)
    for k_size, q_size, c_size in ((500.0, 2.0 ** -9, 2.0 ** -7), (2.0 ** -6, 4.0, 2.0 ** 4), (3000.0, 2.0 ** -12, 2.0 ** -9)):
        inp = synth.make_inputs(wl)
        inp.cache[:, 512:] = (inp.cache[:, 512:].float() / 4.5 * k_size).to(torch.bfloat16)
        inp.cache[:, :512] = (inp.cache[:, :512].float() * c_size).to(torch.bfloat16)
        inp.q[..., 128:] = (inp.q[..., 128:].float() * q_size).to(torch.bfloat16)
        codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
        assert_parity(_run(inp, wl, codes, scale, 64), _oracle(inp, wl, codes, scale, 64), f"{k_size} {q_size} {c_size}")


def test_a_scale_that_is_no_number_stays_in_its_sequence():
    wl = _case("nan", (300, 300), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    ref = _oracle(inp, wl, codes, scale, 64)
    scale[int(inp.block_table[0, 1]), 2] = float("nan")
    got = _run(inp, wl, codes, scale, 64)
    assert np.isnan(got[0]).any()
    assert_parity(got[1:], ref[1:], "the other sequence")


def test_token_ranges_combine():
    """Context parallelism over a block-scaled cache: two ranges' states combine to the whole."""
    wl = _case("ranges", (900,), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "int8")
    ref = _oracle(inp, wl, codes, scale, 64)
    dev = synth.to_device(inp)
    cd, sd, krope = codes.cuda(), scale.cuda(), inp.cache[:, 512:].contiguous().cuda()
    pos = torch.tensor([899], dtype=torch.int32, device="cuda")
    po = torch.empty(2, 1, 128, 512, device="cuda")
    pl = torch.empty(2, 1, 128, 4, device="cuda")
    out = torch.empty(1, 128, 128, device="cuda")
    for k, (a, n) in enumerate(((0, 448), (448, 452))):
        bt = dev.block_table[:, a // 64:].contiguous()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        p = hra.make_params(dev.q, cd, krope, lens, dev.w_uk, dev.w_uv, None, n_branch=4, branch_scale=wl.sigma_o,
                            block_table=bt, page_size=64, ckv_scale=sd, scale_block=64, q_positions=pos, part_o=po[k], part_lse=pl[k])
        ws = hra.alloc_workspace(p)
        hra.mlra_decode(p)
        hra.check_device_status(p)
    p = hra.make_params(dev.q, cd, krope, lens, dev.w_uk, dev.w_uv, out, n_branch=4, branch_scale=wl.sigma_o, block_table=bt,
                        page_size=64, ckv_scale=sd, scale_block=64)
    ws = hra.alloc_workspace(p)
    hra.combine_partials(p, po, pl)
    hra.check_device_status(p)
    assert_parity(out.cpu().numpy(), ref, "two ranges")
    del ws


def test_static_entry_point():
    wl = _case("static", (300, 77), page_size=64)
    inp = synth.make_inputs(wl)
    codes, scale = _quantize(inp.cache[:, :512], 64, "e4m3")
    dev = synth.to_device(inp)
    cd, sd, krope = codes.cuda(), scale.cuda(), inp.cache[:, 512:].contiguous().cuda()
    out = torch.empty(2, 128, 128, device="cuda")
    p = hra.make_params(dev.q, cd, krope, dev.seq_lens, dev.w_uk, dev.w_uv, out, n_branch=4, branch_scale=wl.sigma_o,
                        block_table=dev.block_table, page_size=64, ckv_scale=sd, scale_block=64)
    hra.mlra_decode_static(p)
    torch.cuda.synchronize()
    assert_parity(out.cpu().numpy(), _oracle(inp, wl, codes, scale, 64), "static")


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,block", [("int8", 64), ("e4m3", 32)])
def test_serving_loop(fmt, block):
    """Two prompts are planned, appended, loaded and prefilled; then single-token steps, in
    which one captured graph plans, appends and decodes, with a request that ends and one that
    starts on the way.  Every step's output against the oracle on the cache's own values."""
    r = np.random.default_rng(31)
    B, page, wide, pages, h, chunk = 3, 64, 6, 14, 16, 256
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, new, table, ring = i32(B), i32(B), i32(B, wide) - 1, torch.tensor(r.permutation(pages), dtype=torch.int32, device="cuda")
    free = torch.tensor([3, 3 + pages], dtype=torch.int64, device="cuda")
    start, slots, positions, status = i32(B + 1), i32(chunk), i32(chunk), i32(4)
    codes = torch.zeros(pages * page, 512, dtype=DTYPE[fmt], device="cuda")
    scale = torch.full((pages * page // block, 4), float("nan"), device="cuda")
    krope = torch.full((pages * page, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(chunk, 576, dtype=torch.bfloat16, device="cuda")
    seen = torch.zeros(chunk, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, h, 192, dtype=torch.bfloat16, device="cuda")
    w_uk, w_uv = (torch.tensor(r.standard_normal((h, 512, 128)) / 128 ** 0.5, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.zeros(B, h, 128, device="cuda")
    plan = hra.make_plan_params(lens, new, table, ring, free, lens, free, start, slots, status, positions=positions, page_size=page)
    put = hra.make_append_params(rows[:, :512], rows[:, 512:], slots, positions, codes, krope, ckv_scale=scale, scale_block=block,
                                 rows_out=seen)
    dec = hra.make_params(q, codes, krope, lens, w_uk, w_uv, out, n_branch=4, branch_scale=0.5, block_table=table, page_size=page,
                          ckv_scale=scale, scale_block=block)
    ws = hra.alloc_workspace(dec)

    def fill(t):
        t.copy_(torch.tensor(r.standard_normal(t.shape), dtype=torch.bfloat16))

    def cache_of(b):
        """The values and RoPE keys of sequence b's cached rows."""
        at = paged.cache_rows_of(int(lens[b]), b, table.cpu().numpy(), page, 0)
        s = scale.cpu().numpy()
        c = codes.float().double().cpu().numpy()[at] * np.repeat(s[at // block], 128, axis=1)
        return c, krope.double().cpu().numpy()[at]

    # prompts
    fill(rows)
    new.copy_(torch.tensor([150, 0, 97]))
    hra.page_plan(plan)
    hra.check_plan_status(plan)
    hra.cache_append(put)
    loaded = torch.zeros(B, 150, 576, dtype=torch.bfloat16, device="cuda")
    hra.cache_load(hra.make_load_params(codes, krope, lens, loaded, block_table=table, page_size=page, ckv_scale=scale,
                                        scale_block=block))
    torch.cuda.synchronize()
    assert torch.equal(loaded[0], seen[:150]) and torch.equal(loaded[2, :97], seen[150:247])
    qp = torch.tensor(r.standard_normal((150, h, 192)), dtype=torch.bfloat16, device="cuda")
    po = torch.zeros(150, h, 128, device="cuda")
    pre = hra.make_prefill_params(qp, loaded[0, :, :512], loaded[0, :, 512:], w_uk, w_uv, po, n_branch=4, branch_scale=0.5)
    pws = hra.alloc_prefill_workspace(pre)
    hra.mlra_prefill(pre)
    hra.check_prefill_status(pre)
    seen0 = loaded[0].double().cpu().numpy()
    ref = oracle.mlra_prefill_expanded(qp.cpu(), seen0[:, :512], seen0[:, 512:], w_uk.cpu(), w_uv.cpu(), 4, branch_scale=0.5)
    assert_parity(po.cpu().numpy(), ref, "prefill over loaded rows")
    # one graph for every step; the buffers' contents are put back after the warm-up
    new.fill_(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hra.page_plan(plan)
        hra.cache_append(put)
        hra.mlra_decode(dec)
    for step, asks in enumerate([[1, 0, 1], [1, 0, 1], [1, 33, 1], [1, 1, -1], [1, 1, 0], [1, 1, 70]] + [[1, 1, 1]] * 3):
        before = lens.tolist()
        new.copy_(torch.tensor(asks))
        fill(rows)
        fill(q)
        graph.replay()
        hra.check_plan_status(plan)
        hra.check_device_status(dec)
        assert lens.tolist() == [0 if a < 0 else n + a for n, a in zip(before, asks)]
        got = out.cpu().numpy()
        for b in range(B):
            n = int(lens[b])
            if n == 0:
                assert (got[b] == 0).all()
                continue
            c, k = cache_of(b)
            ref = oracle.mlra_decode_absorbed(q[b].cpu(), c, k, w_uk.cpu(), w_uv.cpu(), 4, branch_scale=0.5)
            assert_parity(got[b][None], ref[None], f"step {step} sequence {b}")
    used = sum(-(-int(n) // page) for n in lens.tolist())
    assert int(free[1] - free[0]) == pages - used
    del ws, pws


def test_two_captured_graphs_share_a_workspace():
    """Two graphs of different cases on one workspace, replayed in turn."""
    wls = [_case("ga", (700, 33), page_size=64), _case("gb", (64, 1200), page_size=64, heads=16)]
    kept, need = [], 0
    for wl, fmt in zip(wls, ("int8", "e4m3")):
        inp = synth.make_inputs(wl)
        codes, scale = _quantize(inp.cache[:, :512], 64, fmt)
        dev = synth.to_device(inp)
        out = torch.zeros(wl.batch, wl.heads, 128, device="cuda")
        bufs = [dev, codes.cuda(), scale.cuda(), inp.cache[:, 512:].contiguous().cuda(), out]
        p = hra.make_params(dev.q, bufs[1], bufs[3], dev.seq_lens, dev.w_uk, dev.w_uv, out, n_branch=4, branch_scale=wl.sigma_o,
                            block_table=dev.block_table, page_size=64, ckv_scale=bufs[2], scale_block=64)
        need = max(need, hra.workspace_size(p))
        kept.append((p, bufs, _oracle(inp, wl, codes, scale, 64)))
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:]
    graphs = []
    for p, _, _ in kept:
        p.workspace, p.workspace_bytes = ws.data_ptr(), need
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hra.mlra_decode(p)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for p, bufs, ref in kept:
        hra.check_device_status(p)
        assert_parity(bufs[4].cpu().numpy(), ref, "replayed")


def test_two_decodes_at_once():
    """Two calls on two streams, each with its own workspace, queued several times over."""
    wls = [_case("sa", (900, 33, 2000), page_size=64), _case("sb", (64, 1200), page_size=64)]
    kept = []
    for wl, fmt in zip(wls, ("int8", "e4m3")):
        inp = synth.make_inputs(wl)
        codes, scale = _quantize(inp.cache[:, :512], 64, fmt)
        dev = synth.to_device(inp)
        out = torch.zeros(wl.batch, wl.heads, 128, device="cuda")
        bufs = [dev, codes.cuda(), scale.cuda(), inp.cache[:, 512:].contiguous().cuda(), out]
        p = hra.make_params(dev.q, bufs[1], bufs[3], dev.seq_lens, dev.w_uk, dev.w_uv, out, n_branch=4, branch_scale=wl.sigma_o,
                            block_table=dev.block_table, page_size=64, ckv_scale=bufs[2], scale_block=64)
        kept.append((p, bufs, hra.alloc_workspace(p), _oracle(inp, wl, codes, scale, 64), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for p, _, _, _, stream in kept:
            hra.mlra_decode(p, stream)
    for p, bufs, _, ref, stream in kept:
        hra.check_device_status(p, stream)
        assert_parity(bufs[4].cpu().numpy(), ref, "two streams")


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
def test_steps_queued_back_to_back(fmt, graph):
    """Plan, append and decode of two steps in turn on the same buffers, with nothing between the
    calls: each decode sees its own step's lengths, pages and rows, bit for bit what it sees when every call
    is waited for (no sum's order depends on timing).  Few heads and long appends leave SMs to kernels
    that start early."""
    r = np.random.default_rng(5)
    page, wide, h, most = 64, 200, 16, 12000
    fmt_t = {**DTYPE, "bf16": torch.bfloat16}[fmt]
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    block = 0 if fmt == "bf16" else 64
    pages = 2 * wide
    codes = torch.zeros(pages * page, 512, dtype=fmt_t, device="cuda")
    scale = torch.zeros(pages * page // 64, 4, device="cuda") if block else None
    krope = torch.zeros(pages * page, 64, dtype=torch.bfloat16, device="cuda")
    lens, table, lens_out, start, status = i32(2), i32(2, wide), i32(2), i32(3), i32(4)
    slots, positions = i32(most), i32(most)
    ring = torch.arange(pages, dtype=torch.int32, device="cuda")
    free, free_out = (torch.tensor([0, pages], dtype=torch.int64, device="cuda") for _ in range(2))
    q = torch.tensor(r.standard_normal((2, h, 192)), dtype=torch.bfloat16, device="cuda")
    w_uk, w_uv = (torch.tensor(r.standard_normal((h, 512, 128)) / 128 ** 0.5, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    steps = []
    for asks in ((5000, 7000), (9, 11900), (7000, 1)):
        rows = torch.tensor(r.standard_normal((most, 576)), dtype=torch.bfloat16, device="cuda")
        new = torch.tensor(asks, dtype=torch.int32, device="cuda")
        steps.append((
            hra.make_plan_params(lens, new, table, ring, free, lens_out, free_out, start, slots, status, positions=positions, page_size=page),
            hra.make_append_params(rows[:, :512], rows[:, 512:], slots, positions, codes, krope, ckv_scale=scale, scale_block=block),
            [torch.zeros(2, h, 128, device="cuda") for _ in range(5)], (rows, new)))
    ws = None

    def queue(k, turn, wait):
        nonlocal ws
        plan, put, outs, _ = steps[k]
        dec = hra.make_params(q, codes, krope, lens_out, w_uk, w_uv, outs[turn], n_branch=4, branch_scale=0.5, block_table=table,
                              page_size=page, ckv_scale=scale, scale_block=block)
        if ws is None:
            ws = hra.alloc_workspace(dec)
        else:
            dec.workspace, dec.workspace_bytes = ws.data_ptr(), ws.numel()
        for call, p in ((hra.page_plan, plan), (hra.cache_append, put), (hra.mlra_decode, dec)):
            call(p)
            if wait:
                torch.cuda.synchronize()
        return dec

    for k in range(3):
        hra.check_device_status(queue(k, 0, True))
        hra.check_plan_status(steps[k][0])
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for turn in range(1, 5):
                for k in range(3):
                    queue(k, turn, False)
        g.replay()
    else:
        for turn in range(1, 5):
            for k in range(3):
                queue(k, turn, False)
    torch.cuda.synchronize()
    for k, (_, _, outs, _) in enumerate(steps):
        assert outs[0].abs().max() > 0 and torch.isfinite(outs[0]).all()
        for turn in range(1, 5):
            assert torch.equal(outs[turn], outs[0]), (k, turn)


def test_load_then_prefill_queued_back_to_back():
    """Two caches loaded in turn into one buffer, each followed at once by the prefill that reads it."""
    r = np.random.default_rng(6)
    L, n, h = 4000, 64, 16
    w_uk, w_uv = (torch.tensor(r.standard_normal((h, 512, 128)) / 128 ** 0.5, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.tensor(r.standard_normal((n, h, 192)), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    loaded = torch.zeros(1, L, 576, dtype=torch.bfloat16, device="cuda")
    loads, ws, outs = [], None, [[torch.zeros(n, h, 128, device="cuda") for _ in range(5)] for _ in range(2)]
    for _ in range(2):
        codes = torch.tensor(r.integers(-127, 128, (L, 512)), dtype=torch.int8, device="cuda")
        scale = torch.tensor(r.random((-(-L // 64), 4)) / 64 + 1e-3, dtype=torch.float32, device="cuda")
        krope = torch.tensor(r.standard_normal((L, 64)), dtype=torch.bfloat16, device="cuda")
        loads.append((hra.make_load_params(codes, krope, lens, loaded, seq_stride=L, ckv_scale=scale, scale_block=64), codes, scale, krope))
    for turn in range(5):
        for k in range(2):
            pre = hra.make_prefill_params(q, loaded[0, :, :512], loaded[0, :, 512:], w_uk, w_uv, outs[k][turn], n_branch=4, branch_scale=0.5)
            if ws is None:
                ws = hra.alloc_prefill_workspace(pre)
            else:
                pre.workspace, pre.workspace_bytes = ws.data_ptr(), ws.numel()
            hra.cache_load(loads[k][0])
            if turn == 0:
                torch.cuda.synchronize()
            hra.mlra_prefill(pre)
            if turn == 0:
                hra.check_prefill_status(pre)
    torch.cuda.synchronize()
    for k in range(2):
        assert outs[k][0].abs().max() > 0
        for turn in range(1, 5):
            assert torch.equal(outs[k][turn], outs[k][0]), (k, turn)
