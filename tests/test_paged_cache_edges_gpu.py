"""GPU tests of the paged cache's edges: page pools that hold what is no page, calls that overlap,
and chains of calls with nothing between them."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
from oracle import paged
from test_paged_cache_gpu import Plan, _plan_case

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- page plan
@pytest.mark.parametrize("B,page,wide,chunk,max_tokens,head", [
    (1, 32, 3, 90, 90, 0), (64, 64, 40, 1, 64, 77), (257, 96, 30, 50, 5000, 123456), (1024, 32, 16, 90, 65536, 1 << 33)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_refuses_pages_that_are_none_of_the_pool(B, page, wide, chunk, max_tokens, head, in_place):
    """The last page to be taken is -1, or one past the pool; behind the pages to be taken it does not matter."""
    lens, new, table, ring, free = _plan_case(B, B, page, wide, chunk, max_tokens, head=head)
    good = paged.page_plan(lens, new, table, ring, free, page, max_tokens)
    taken = good["free"][0] - free[0]
    assert good["status"] == [0, 0, 0, 0] and (taken > 0 or B == 64)
    for at, bad, code in ((taken - 1, -1, 6), (taken - 1, len(ring), 6), (0, -2 ** 31, 6), (taken, -1, 0)):
        if code and taken == 0:
            continue
        other = ring.copy()
        other[(free[0] + at) % len(ring)] = bad
        want = paged.page_plan(lens, new, table, other, free, page, max_tokens)
        assert want["status"][0] == code
        plan = Plan(lens, new, table, other, free, page, max_tokens, in_place=in_place)
        hra.page_plan(plan.p)
        plan.check(want)
        if code:
            with pytest.raises(hra.HraError, match="no page of the pool") as e:
                hra.check_plan_status(plan.p)
            assert e.value.status == hra._binding.HRA_ERR_PLAN


def test_a_bad_page_given_back_is_not_handed_out():
    """Request 0 ends with a page that is none of the pool in its row; the page goes to the ring, and
    the step that would hand it to request 1 is refused, lengths and pool as they were."""
    case = ([40, 0], [-1, 32], np.array([[0, 9], [-1, -1]]), np.array([2, 3, -7, -7]), [0, 2])
    plan = Plan(*case, 32, 64, in_place=True)
    hra.page_plan(plan.p)
    hra.check_plan_status(plan.p)
    assert plan.free.tolist() == [1, 4] and plan.ring.tolist() == [2, 3, 0, 9] and plan.table.tolist()[1] == [2, -1]
    plan.new.copy_(torch.tensor([0, 32]))
    hra.page_plan(plan.p)
    plan.new.copy_(torch.tensor([64, 0]))
    hra.page_plan(plan.p)
    assert plan.status.tolist() == [6, 0, 3, 9] and plan.free.tolist() == [2, 4] and plan.lens.tolist() == [0, 64]


# ------------------------------------------------- chains of calls with nothing between them
def _bf16(r, *shape, std=1.0):
    return torch.tensor(r.standard_normal(shape) * std, dtype=torch.bfloat16, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Chain:
    """Steps that write the same buffers in turn, each ending in an output of its own: queued with
    nothing between the calls, in a stream or a captured graph, they give bit for bit what they give when
    every call is waited for (no sum's order depends on timing)."""

    def __init__(self):
        self.steps = []  # (calls, output)

    def add(self, calls, out):
        self.steps.append((calls, out))

    def queue(self, wait):
        outs = []
        for calls, out in self.steps:
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            outs.append(out.clone())
        return outs

    def check(self, graph):
        want = self.queue(True)
        assert all(torch.isfinite(w).all() and w.abs().max() > 0 for w in want)
        assert not torch.equal(want[0], want[1])
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                turns = [self.queue(False) for _ in range(4)]
            g.replay()
        else:
            torch.cuda.synchronize()
            turns = [self.queue(False) for _ in range(4)]
        torch.cuda.synchronize()
        for got in turns:
            for k, (g, w) in enumerate(zip(got, want)):
                assert torch.equal(g, w), k


def _plain_decode(r, rows, lens, n_branch, h=16):
    """A bf16 decode over rows [B, L, 576] as they lie; returns its call and its output."""
    B, L = rows.shape[:2]
    q, w_uk, w_uv = _bf16(r, B, h, 192), _bf16(r, h, 512, 128, std=128 ** -0.5), _bf16(r, h, 512, 128, std=128 ** -0.5)
    out = torch.zeros(B, h, 128, device="cuda")
    flat = rows.view(B * L, 576)
    p = hra.make_params(q, flat[:, :512], flat[:, 512:], lens, w_uk, w_uv, out, n_branch=n_branch, seq_stride=L)
    keep = (q, w_uk, w_uv, rows, lens, hra.alloc_workspace(p))
    return lambda: (hra.mlra_decode(p), keep)[0], out


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("n_branch", [1, 2, 4])
def test_load_then_plain_decode(n_branch, graph):
    """Rows of two 8-bit caches loaded in turn into one buffer, each read at once by a bf16 decode."""
    r = np.random.default_rng(n_branch)
    L, chain = 3000, Chain()
    lens = _i32([L, 1777])
    loaded = torch.zeros(2, L, 576, dtype=torch.bfloat16, device="cuda")
    decode, out = _plain_decode(r, loaded, lens, n_branch)
    for _ in range(2):
        codes = torch.tensor(r.integers(-127, 128, (2 * L, 512)), dtype=torch.int8, device="cuda")
        scale = torch.tensor(r.random((-(-2 * L // 32), 4)) / 64 + 1e-3, dtype=torch.float32, device="cuda")
        krope = _bf16(r, 2 * L, 64)
        p = hra.make_load_params(codes, krope, lens, loaded, seq_stride=L, ckv_scale=scale, scale_block=32)
        p.keep = (codes, scale, krope)
        chain.add([lambda p=p: hra.cache_load(p), decode], out)
    chain.check(graph)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_of_an_append_then_plain_decode(fmt, graph):
    """The rows that a block-scaled append leaves, read at once by a bf16 decode."""
    r = np.random.default_rng(11)
    L, chain = 4096, Chain()
    seen = torch.zeros(1, L, 576, dtype=torch.bfloat16, device="cuda")
    decode, out = _plain_decode(r, seen, _i32([L]), 4)
    codes = torch.zeros(L, 512, dtype={"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt], device="cuda")
    krope, scale, slots = _bf16(r, L, 64), torch.zeros(L // 64, 4, device="cuda"), torch.arange(L, dtype=torch.int32, device="cuda")
    for _ in range(2):
        rows = _bf16(r, L, 576)
        p = hra.make_append_params(rows[:, :512], rows[:, 512:], slots, slots, codes, krope, ckv_scale=scale, scale_block=64,
                                   rows_out=seen[0])
        p.keep = rows
        chain.add([lambda p=p: hra.cache_append(p), decode], out)
    chain.check(graph)


@pytest.mark.parametrize("graph", [False, True])
def test_plan_append_decode_with_a_scale_per_row(graph):
    r = np.random.default_rng(12)
    page, wide, h, most, chain = 64, 100, 16, 9000, Chain()
    zeros = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    codes = torch.zeros(2 * wide * page, 512, dtype=torch.int8, device="cuda")
    krope, scale = _bf16(r, 2 * wide * page, 64), torch.zeros(2 * wide * page, 4, device="cuda")
    lens, lens_out, table, start, status, slots, positions = (zeros(2), zeros(2), zeros(2, wide), zeros(3), zeros(4), zeros(most),
                                                              zeros(most))
    ring = torch.arange(2 * wide, dtype=torch.int32, device="cuda")
    free, free_out = (torch.tensor([0, 2 * wide], dtype=torch.int64, device="cuda") for _ in range(2))
    q, w_uk, w_uv = _bf16(r, 2, h, 192), _bf16(r, h, 512, 128, std=128 ** -0.5), _bf16(r, h, 512, 128, std=128 ** -0.5)
    out = torch.zeros(2, h, 128, device="cuda")
    dec = hra.make_params(q, codes, krope, lens_out, w_uk, w_uv, out, n_branch=4, block_table=table, page_size=page, ckv_scale=scale)
    keep = hra.alloc_workspace(dec)
    for asks in ((4000, 5000), (6000, 3), (7, 6400)):
        rows, new = _bf16(r, most, 576), _i32(asks)
        plan = hra.make_plan_params(lens, new, table, ring, free, lens_out, free_out, start, slots, status, positions=positions,
                                    page_size=page)
        put = hra.make_append_params(rows[:, :512], rows[:, 512:], slots, positions, codes, krope, ckv_scale=scale)
        plan.keep, put.keep = new, rows
        chain.add([lambda p=plan: hra.page_plan(p), lambda p=put: hra.cache_append(p), lambda: hra.mlra_decode(dec)], out)
    chain.check(graph)
    del keep


@pytest.mark.parametrize("graph", [False, True])
def test_inputs_written_just_before_a_call(graph):
    """A decode whose query, lengths, table and cache a copy has only just written."""
    r = np.random.default_rng(13)
    chain, h, page = Chain(), 16, 64
    sets = [dict(q=_bf16(r, 3, h, 192), lens=_i32(n), table=_i32(r.permutation(96).reshape(3, 32)),
                 cache=_bf16(r, 96 * page, 576)) for n in ([2000, 1, 640], [65, 2048, 1500])]
    live = {k: torch.zeros_like(v) for k, v in sets[0].items()}
    w_uk, w_uv, out = _bf16(r, h, 512, 128, std=128 ** -0.5), _bf16(r, h, 512, 128, std=128 ** -0.5), torch.zeros(3, h, 128, device="cuda")
    p = hra.make_params(live["q"], live["cache"][:, :512], live["cache"][:, 512:], live["lens"], w_uk, w_uv, out, n_branch=4,
                        block_table=live["table"], page_size=page)
    keep = hra.alloc_workspace(p)
    for s in sets:
        chain.add([lambda s=s: [live[k].copy_(v) for k, v in s.items()], lambda: hra.mlra_decode(p)], out)
    chain.check(graph)
    del keep


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("rows", [1, 20])
def test_quotients_by_a_scale_that_is_not_the_rows_own(fmt, rows):
    """Open blocks of any scale: the nearest code to the exact quotient, for values on a border
    between two codes, the neighbours of such values in bf16, and any others.  A quotient is a
    border or 2^-33 of itself away from it, so its rounding to 64 bits keeps the side."""
    r = np.random.default_rng(rows)
    blocks, block = 600, 32
    scale = np.ldexp(r.uniform(1, 2, blocks), r.integers(-85, 90, blocks))
    scale[::3] = np.ldexp(r.integers(1, 128, len(scale[::3])), r.integers(-85, 84, len(scale[::3])))  # borders that are bf16
    scale = scale.astype(np.float32)
    grid = np.arange(128.0) if fmt == "int8" else paged.e4m3_values()
    borders = (grid[1:] + grid[:-1]) / 2
    borders = borders[borders * (1 + 2.0 ** -6) < paged.TOP[fmt]]  # the scale stays the block's
    x = r.choice(borders, (blocks * rows, 128)) * r.choice([-1, 1], (blocks * rows, 128))
    x[:, 96:] = r.uniform(-0.98, 0.98, (blocks * rows, 32)) * paged.TOP[fmt]
    x = torch.tensor(x * np.repeat(scale.astype(np.float64), rows)[:, None], dtype=torch.bfloat16)
    step = torch.tensor(r.integers(-1, 2, x.shape), dtype=torch.int16)
    x = (x.view(torch.int16) + step).view(torch.bfloat16)  # the bf16 number itself, or a neighbour
    want = paged.nearest(x.double().numpy() / np.repeat(scale.astype(np.float64), rows)[:, None], fmt)
    slots = (np.arange(blocks)[:, None] * block + 1 + np.arange(rows)).reshape(-1)
    codes = torch.zeros(blocks * block, 128, dtype={"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt], device="cuda")
    krope, sd, s = torch.zeros(blocks * block, 64, dtype=torch.bfloat16, device="cuda"), torch.tensor(scale[:, None], device="cuda"), _i32(slots)
    hra.cache_append(hra.make_append_params(x.cuda(), torch.zeros(len(slots), 64, dtype=torch.bfloat16, device="cuda"), s, s, codes,
                                            krope, ckv_scale=sd, scale_block=block))
    assert np.array_equal(sd.cpu().numpy()[:, 0], scale)
    assert np.array_equal(codes.float().double().cpu().numpy()[slots], want)


# --------------------------------------------------------------------------- two streams
def test_appends_and_loads_of_two_streams_overlap():
    """Two caches, a stream each: appends that start every block anew and loads of what they wrote,
    queued in turn on both streams with no wait between them."""
    r = np.random.default_rng(21)
    sides = []
    for fmt, block, n in (("int8", 64, 12000), ("e4m3", 32, 9000)):
        rows = -(-n // 64) * 64
        codes = torch.zeros(rows, 512, dtype={"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt], device="cuda")
        scale, krope = torch.zeros(rows // block, 4, device="cuda"), torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
        slots, lens = torch.arange(n, dtype=torch.int32, device="cuda"), _i32([n])
        stream, steps = torch.cuda.Stream(), []
        for _ in range(6):
            x = _bf16(r, n, 576)
            seen, back = (torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            steps.append((hra.make_append_params(x[:, :512], x[:, 512:], slots, slots, codes, krope, ckv_scale=scale,
                                                 scale_block=block, rows_out=seen),
                          hra.make_load_params(codes, krope, lens, back[None], seq_stride=rows, ckv_scale=scale, scale_block=block),
                          x, seen, back))
        sides.append((stream, steps, (codes, scale, krope, slots, lens), fmt, block))
    torch.cuda.synchronize()
    for k in range(6):
        for stream, steps, _, _, _ in sides:
            hra.cache_append(steps[k][0], stream)
            hra.cache_load(steps[k][1], stream)
    torch.cuda.synchronize()
    for _, steps, keep, fmt, block in sides:
        for _, _, x, seen, back in steps:
            assert torch.equal(seen, back)
        # the last step's cache against the definition, and every step's rows near its own tokens
        n = len(keep[3])
        for _, _, x, seen, _ in steps:
            top, eps = (127.0, 0.5 / 127) if fmt == "int8" else (448.0, 2.0 ** -4)
            amax = torch.nn.functional.pad(x[:, :512].float().abs(), (0, 0, 0, -n % block)).view(-1, block, 4, 128).amax((1, 3))
            a = amax.repeat_interleave(block, 0)[:n].repeat_interleave(128, 1)
            # int8: half a step of amax / 127; e4m3: 2^-4 of the value or half a step of 2^-9 amax / 448; and bf16
            off = a * eps if fmt == "int8" else torch.maximum(x[:, :512].float().abs() * eps, a * 2.0 ** -10 / 448)
            assert ((seen[:, :512].float() - x[:, :512].float()).abs() <= off * 1.001 + 2.0 ** -8 * seen[:, :512].float().abs()).all()
        want = paged.append(np.zeros((len(keep[0]), 512)), np.zeros(keep[1].shape, np.float32), np.zeros((len(keep[0]), 64)),
                            steps[-1][2][:, :512].double().cpu().numpy(), steps[-1][2][:, 512:].double().cpu().numpy(),
                            range(n), range(n), block, fmt)
        assert np.array_equal(keep[0].float().double().cpu().numpy(), want[0]) and np.array_equal(keep[1].cpu().numpy(), want[1])
