"""GPU tests of the paged cache (page plan, append, load) through the C ABI against the fp64
definitions of oracle.paged: whole numbers, codes and scales are equal; RoPE keys and loaded
values are within one bf16 rounding of the definition."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
from oracle import paged

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative to the value
DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------- page plan
def _plan_case(seed, B, page, wide, chunk, max_tokens, kinds=(0.1, 0.85, 0.95), head=0):
    r = np.random.default_rng(seed)
    cached, new, left = [], [], max_tokens
    for _ in range(B):
        u = r.random()
        cached.append(0 if u < kinds[0] else int(r.integers(0, wide * page - chunk + 1)))
        n = -1 if u > kinds[2] else 0 if u > kinds[1] else int(r.integers(1, chunk + 1))
        new.append(min(n, left))
        left -= max(new[-1], 0)
    pages = [-(-c // page) for c in cached]
    total = sum(pages) + max_tokens // page + B + 3
    order = r.permutation(total)
    table = np.full((B, wide), -1)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    ring = np.full(total, -7)
    free = [head, head + total - at]
    for k, p in enumerate(order[at:]):
        ring[(head + k) % total] = p
    return cached, new, table, ring, free


class Plan:
    """Device buffers and parameters of one plan; outputs start as garbage."""

    def __init__(self, lens, new, table, ring, free, page, max_tokens, in_place=False, positions=True):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        B = len(lens)
        self.lens, self.new, self.table, self.ring = i32(lens), i32(new), i32(table), i32(ring)
        self.free = torch.tensor(free, dtype=torch.int64, device="cuda")
        self.lens_out = self.lens if in_place else torch.full_like(self.lens, 99)
        self.free_out = self.free if in_place else torch.full_like(self.free, 99)
        self.start, self.status = i32(np.full(B + 1, 99)), i32([99] * 4)
        self.slots = i32(np.full(max_tokens, 99))
        self.positions = i32(np.full(max_tokens, 99)) if positions else None
        self.p = hra.make_plan_params(self.lens, self.new, self.table, self.ring, self.free, self.lens_out, self.free_out,
                                      self.start, self.slots, self.status, positions=self.positions, page_size=page)

    def check(self, want):
        got = dict(lens=self.lens_out, table=self.table, ring=self.ring, free=self.free_out, start=self.start,
                   slots=self.slots, positions=self.positions, status=self.status)
        for k, v in got.items():
            if v is not None:
                assert v.tolist() == np.asarray(want[k]).tolist(), k


@pytest.mark.parametrize("B,page,wide,chunk,max_tokens,head", [
    (1, 32, 1, 1, 1, 0), (1, 64, 3, 150, 200, 5), (3, 32, 9, 70, 40, 1 << 40), (64, 64, 40, 1, 64, 77),
    (257, 96, 30, 50, 5000, 123456), (1000, 64, 8, 33, 20000, 3), (1024, 32, 16, 90, 65536, 1 << 33),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, page, wide, chunk, max_tokens, head, in_place):
    case = _plan_case(B + page, B, page, wide, chunk, max_tokens, head=head)
    want = paged.page_plan(*case, page, max_tokens)
    assert want["status"] == [0, 0, 0, 0]
    plan = Plan(*case, page, max_tokens, in_place=in_place, positions=not in_place or B % 2 == 0)
    hra.page_plan(plan.p)
    hra.check_plan_status(plan.p)
    plan.check(want)
    if not in_place:  # the same call again: the same plan
        hra.page_plan(plan.p)
        plan.check(want)


def test_plan_without_tokens_and_all_ended():
    for new in ([0, 0, 0], [-1, -5, -1]):
        case = ([70, 0, 64], new, np.array([[4, 5], [-1, -1], [1, -1]]), np.array([0, 2, 3, -1, -1, -1, 9, 9]), [8, 11])
        plan = Plan(*case, 64, 7)
        hra.page_plan(plan.p)
        plan.check(paged.page_plan(*case, 64, 7))


@pytest.mark.parametrize("case", [
    dict(lens=[5, -1, -3]), dict(lens=[5, 129, 0]), dict(lens=[5, 120, 128], new=[1, 9, 1]),
    dict(lens=[5, 120, 128], new=[-1, 1, 2 ** 31 - 1]), dict(new=[10, 10, 13]),
    dict(new=[2 ** 31 - 1] * 3, lens=[0, 0, 0]), dict(lens=[64, 0, 0], new=[1, 1, 1], free=[6, 8]),
    dict(free=[3, 2]), dict(free=[-1, 2]), dict(free=[0, 9]), dict(lens=[128, 0, 0], new=[-1, 1, 1], free=[0, 7]),
])
def test_plan_refuses_as_a_whole(case):
    a = dict(lens=[5, 64, 0], new=[1, 1, 1], free=[2, 8])
    a.update(case)
    args = (a["lens"], a["new"], np.arange(6).reshape(3, 2), np.arange(8), a["free"])
    want = paged.page_plan(*args, 64, 32)
    assert want["status"][0] > 0
    plan = Plan(*args, 64, 32)
    hra.page_plan(plan.p)
    with pytest.raises(hra.HraError) as e:
        hra.check_plan_status(plan.p)
    assert e.value.status == hra._binding.HRA_ERR_PLAN
    plan.check(want)


def test_plan_skips_table_entries_that_are_no_page():
    """A cached page outside the pool: its tokens have no slot."""
    case = ([10, 40], [2, 2], np.array([[99, -1], [0, -5]]), np.array([1, 2, 3, 4]), [0, 2])
    plan = Plan(*case, 32, 4)
    hra.page_plan(plan.p)
    plan.check(paged.page_plan(*case, 32, 4))
    assert plan.slots.tolist()[:2] == [-1, -1]


# ------------------------------------------------------------------------------- append
def _codes_of(t):
    return t.float().double().cpu().numpy()


def _random_cache(r, rows, d_c, block, fmt):
    krope = torch.tensor(r.standard_normal((rows, 64)), dtype=torch.bfloat16)
    if fmt == "bf16":
        return torch.tensor(r.standard_normal((rows, d_c)), dtype=torch.bfloat16), None, krope
    codes = torch.tensor(r.integers(-127, 128, (rows, d_c)), dtype=torch.int8)
    if fmt == "e4m3":
        codes = (codes.float() * 3).to(torch.float8_e4m3fn)
    scale = torch.tensor(r.uniform(0.5, 1.5, (-(-rows // block), d_c // 128)) / paged.TOP[fmt] * 3.0, dtype=torch.float32)
    return codes, scale, krope


def _append(r, slots, positions, *, rows, d_c, block, fmt, x=None, rows_out=True, theta=10000.0, stream=None, extra=0):
    """Run the append on a random cache; returns (cache before, got, want)."""
    n = len(slots)
    codes, scale, krope = _random_cache(r, rows, d_c, block, fmt)
    fused = torch.tensor(r.standard_normal((n, d_c + 64 + extra)) * np.exp(r.standard_normal((n, 1))), dtype=torch.bfloat16)
    if x is not None:
        fused[:, :d_c] = x
    dev = [None if t is None else t.cuda() for t in (codes, scale, krope, fused)]
    s, pos = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (slots, positions))
    out = torch.full((n, d_c + 64 + extra), 7.0, dtype=torch.bfloat16, device="cuda")[:, :d_c + 64] if rows_out else None
    p = hra.make_append_params(dev[3][:, :d_c], dev[3][:, d_c:d_c + 64], s, pos, dev[0], dev[2], ckv_scale=dev[1],
                               scale_block=block, rows_out=out, rope_theta=theta)
    torch.cuda.synchronize()
    hra.cache_append(p, stream)
    torch.cuda.synchronize()
    want = paged.append(_codes_of(codes), None if scale is None else scale.numpy(), krope.double().numpy(),
                        fused[:, :d_c].double().numpy(), fused[:, d_c:d_c + 64].double().numpy(), slots, positions,
                        block, fmt, theta)
    return (codes, scale, krope, fused), (dev[0], dev[1], dev[2], out), want


def _check_append(before, got, want, slots, *, block, fmt, d_c):
    codes, scale, krope = want
    assert np.array_equal(_codes_of(got[0]), codes)
    if scale is not None:
        assert np.array_equal(got[1].cpu().numpy(), scale)
    # one bf16 rounding of a rotation in fp32: its products and its angle are off by a few
    # 2^-24 of the pair's size
    size = np.abs(before[3][:, -64:].double().numpy()).max() if before[3].shape[1] else 1.0
    live = [i for i in range(len(slots)) if 0 <= slots[i] < codes.shape[0]]
    written = [slots[i] for i in live]
    k = _codes_of(got[2])
    size = np.abs(before[3][:, d_c:d_c + 64].double().numpy())[live].max(initial=0.0)
    assert (np.abs(k - krope) <= HALF_BF16 * np.abs(krope) + 16 * 2.0 ** -24 * size).all()
    others = np.setdiff1d(np.arange(codes.shape[0]), written)
    assert np.array_equal(k[others], krope[others])
    if got[3] is not None:
        out = _codes_of(got[3])
        v = codes if fmt == "bf16" else paged.values(codes, scale, block)
        skipped = np.setdiff1d(np.arange(len(slots)), live)
        assert (out[skipped] == 7.0).all()
        # fl32(code * s), then bf16
        assert (np.abs(out[live, :d_c] - v[written]) <= HALF_BF16 * 1.001 * np.abs(v[written])).all()
        assert np.array_equal(out[live, d_c:], k[written])


RUNS = {  # name: (rows, block, slots)
    "one_token_fresh": (64, 32, [32]),
    "one_token_mid": (64, 64, [37]),
    "one_token_last_row": (96, 32, [95]),
    "decode_step": (640, 64, [5, 64, 191, 200, 256 + 63, 384, 450, 575, 600]),
    "prompt_across_blocks": (512, 64, list(range(130, 420))),
    "whole_blocks_1024": (2048, 1024, list(range(0, 2048))),
    "mid_of_1024": (2048, 1024, list(range(1000, 1500))),
    "eight_and_nine_rows": (256, 64, list(range(10, 18)) + list(range(64 + 10, 64 + 19)) + list(range(128, 137))),
    "padding_between": (256, 32, [-1, 3, 4, -1, 40, 41, -1, -1, 999, 64, 256, 255]),
    "backwards_in_a_block": (128, 64, list(range(63, 40, -1)) + [70, 66, 68]),
    "all_padding": (64, 32, [-1, -1, 64, 70]),
    "three_windows": (192, 96, list(range(50, 96)) + list(range(96, 130))),
}


@pytest.mark.parametrize("name", RUNS)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d_c", [128, 512])
def test_append_blocks(name, fmt, d_c):
    rows, block, slots = RUNS[name]
    r = np.random.default_rng(len(name) + d_c)
    positions = [int(p) for p in r.integers(0, 1 << 21, len(slots))]
    before, got, want = _append(r, slots, positions, rows=rows, d_c=d_c, block=block, fmt=fmt)
    _check_append(before, got, want, slots, block=block, fmt=fmt, d_c=d_c)


@pytest.mark.parametrize("fmt,block", [("bf16", 0), ("int8", 0), ("int8", 1)])
@pytest.mark.parametrize("d_c,n", [(128, 1), (256, 77), (512, 300)])
def test_append_per_token(fmt, block, d_c, n):
    """bf16, and int8 with one scale per token and 128 columns (the format without blocks)."""
    r = np.random.default_rng(n)
    slots = [int(s) for s in r.permutation(400)[:n]]
    slots[n // 2] = -1 if n > 1 else slots[0]
    before, got, want = _append(r, slots, list(range(n)), rows=400, d_c=d_c, block=block or 1, fmt=fmt) if fmt == "int8" else \
        _append(r, slots, list(range(n)), rows=400, d_c=d_c, block=0, fmt=fmt)
    _check_append(before, got, want, slots, block=1, fmt=fmt, d_c=d_c)


def test_append_strides_theta_and_no_rows():
    r = np.random.default_rng(5)
    slots = list(range(20, 60))
    before, got, want = _append(r, slots, [1000003 + i for i in range(40)], rows=128, d_c=256, block=32, fmt="int8", extra=24,
                                theta=500000.0)
    _check_append(before, got, want, slots, block=32, fmt="int8", d_c=256)
    before, got, want = _append(r, slots, [0] * 40, rows=128, d_c=256, block=32, fmt="e4m3", rows_out=False)
    _check_append(before, got, want, slots, block=32, fmt="e4m3", d_c=256)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -95, 1e-8, 1e6, 2.0 ** 110])
def test_append_ties_and_far_scales(fmt, scale):
    """Values that sit on, and one step of bf16 beside, the borders between codes, under
    scales from the smallest to the largest."""
    r = np.random.default_rng(3)
    x = np.zeros((40, 128))
    steps = np.arange(128) + 0.5 if fmt == "int8" else np.resize((paged.e4m3_values()[1:] + paged.e4m3_values()[:-1]) / 2, 128)
    for i in range(40):
        x[i] = steps * r.choice([-1, 1], 128) * (1 + (i % 5 - 2) * 2.0 ** -8)
    x[:, 0] = paged.TOP[fmt]  # the scale is a power of two where the others allow
    slots = list(range(40))
    before, got, want = _append(r, slots, [0] * 40, rows=64, d_c=128, block=32, fmt=fmt,
                                x=torch.tensor(x * scale, dtype=torch.bfloat16))
    _check_append(before, got, want, slots, block=32, fmt=fmt, d_c=128)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_zeros_and_values_that_are_no_numbers(fmt):
    """A zero block has scale 0; Inf or NaN make their own block's scale no finite number and
    leave the other blocks and heads alone."""
    r = np.random.default_rng(4)
    x = torch.tensor(r.standard_normal((96, 256)), dtype=torch.bfloat16)
    x[:32] = 0
    x[40, 5], x[70, 200] = float("nan"), float("inf")
    slots = list(range(96))
    _, got, want = _append(r, slots, slots, rows=96, d_c=256, block=32, fmt=fmt, x=torch.nan_to_num(x))
    sane_codes, sane_scale = _codes_of(got[0]), got[1].cpu().numpy()
    assert np.array_equal(sane_codes, want[0]) and (sane_scale[0] == 0).all() and (sane_codes[:32] == 0).all()
    r = np.random.default_rng(4)
    x2 = torch.tensor(r.standard_normal((96, 256)), dtype=torch.bfloat16)
    codes, scale, krope = _random_cache(r, 96, 256, 32, fmt)
    dev = [codes.cuda(), scale.cuda(), krope.cuda()]
    p = hra.make_append_params(x.cuda(), torch.zeros(96, 64, dtype=torch.bfloat16, device="cuda"),
                               torch.arange(96, dtype=torch.int32, device="cuda"),
                               torch.arange(96, dtype=torch.int32, device="cuda"), dev[0], dev[2], ckv_scale=dev[1], scale_block=32)
    hra.cache_append(p)
    s = dev[1].cpu().numpy()
    finite = np.isfinite(s)
    assert finite.tolist() == [[True, True], [False, True], [True, False]]
    assert np.array_equal(s[finite], sane_scale[finite])
    got_codes = _codes_of(dev[0])
    for b, g in np.argwhere(finite):
        rows, cols = slice(32 * b, 32 * b + 32), slice(128 * g, 128 * g + 128)
        assert np.array_equal(got_codes[rows, cols], sane_codes[rows, cols])
    del x2


def test_append_token_by_token_equals_its_definition():
    """A sequence appended one token at a time over three blocks; the scale grows in between."""
    r = np.random.default_rng(8)
    codes, scale, krope = _random_cache(r, 96, 512, 32, "int8")
    dev = [codes.cuda(), scale.cuda(), krope.cuda()]
    want = (_codes_of(codes), scale.numpy(), krope.double().numpy())
    for t in range(70):
        x = torch.tensor(r.standard_normal((1, 576)) * (1 + t / 10), dtype=torch.bfloat16)
        s = torch.tensor([t], dtype=torch.int32, device="cuda")
        xd = x.cuda()
        hra.cache_append(hra.make_append_params(xd[:, :512], xd[:, 512:], s, s, dev[0], dev[2], ckv_scale=dev[1],
                                                scale_block=32))
        want = paged.append(*want, x[:, :512].double().numpy(), x[:, 512:].double().numpy(), [t], [t], 32, "int8")
        torch.cuda.synchronize()
    assert np.array_equal(_codes_of(dev[0]), want[0]) and np.array_equal(dev[1].cpu().numpy(), want[1])


# --------------------------------------------------------------------------------- load
@pytest.mark.parametrize("fmt,block", [("bf16", 0), ("int8", 0), ("int8", 32), ("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("d_c", [128, 256, 512])
@pytest.mark.parametrize("page", [0, 128])
def test_load(fmt, block, d_c, page):
    r = np.random.default_rng(d_c + page)
    lens = [0, 1, 37, 128, 129, 300]
    width = 260                      # the last sequence is longer than out
    B = len(lens)
    wide = 3
    rows = B * wide * 128
    codes, scale, krope = _random_cache(r, rows, d_c, max(1, block), fmt)
    table = r.permutation(B * wide).reshape(B, wide).astype(np.int32)
    out = torch.full((B, width, d_c + 64 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    keep = [t if t is None else t.cuda() for t in (codes, scale, krope)] + [torch.tensor(lens, dtype=torch.int32, device="cuda")]
    td = torch.tensor(table, device="cuda") if page else None
    p = hra.make_load_params(keep[0], keep[2], keep[3], out[:, :, :d_c + 64], block_table=td, page_size=page,
                             seq_stride=wide * 128, ckv_scale=keep[1], scale_block=block)
    hra.cache_load(p)
    got = out.double().cpu().numpy()
    v = codes.double().numpy() if fmt == "bf16" else paged.values(_codes_of(codes), scale.numpy(), max(1, block))
    for b, n in enumerate(lens):
        m = min(n, width)
        at = paged.cache_rows_of(m, b, table if page else None, 128, wide * 128)
        assert (np.abs(got[b, :m, :d_c] - v[at]) <= (0 if fmt == "bf16" else HALF_BF16 * 1.001) * np.abs(v[at])).all()
        assert np.array_equal(got[b, :m, d_c:d_c + 64], krope.double().numpy()[at])
        assert (got[b, m:] == 7.0).all() and (got[b, :, d_c + 64:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_offsets_past_32_bits(fmt):
    """Append and load at the end of a cache of more than 2^31 bytes (and, for bf16, elements)."""
    rows = (4_400_000 // 64) * 64
    ckv = torch.zeros(rows, 512, dtype=DTYPE[fmt], device="cuda")
    krope = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    scale = torch.zeros(rows // 64, 4, device="cuda") if fmt == "int8" else None
    block = 64 if fmt == "int8" else 0
    r = np.random.default_rng(2)
    x = torch.tensor(r.standard_normal((70, 576)), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(rows - 70, rows, dtype=torch.int32, device="cuda")
    seen = torch.zeros(70, 576, dtype=torch.bfloat16, device="cuda")
    hra.cache_append(hra.make_append_params(x[:, :512], x[:, 512:], slots, slots, ckv, krope, ckv_scale=scale, scale_block=block,
                                            rows_out=seen))
    page = rows // 64
    table = torch.tensor([[page - 2, page - 1]], dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 128, 576, dtype=torch.bfloat16, device="cuda")
    hra.cache_load(hra.make_load_params(ckv, krope, torch.tensor([128], dtype=torch.int32, device="cuda"), out, block_table=table,
                                        page_size=64, ckv_scale=scale, scale_block=block))
    assert torch.equal(out[0, 58:], seen) and (out[0, :58] == 0).all()
    assert int((ckv[:rows - 70].view(torch.int8) != 0).sum()) == 0
    if fmt == "bf16":
        assert torch.equal(seen[:, :512], x[:, :512])


def test_load_pages_outside_the_cache_are_zero():
    r = np.random.default_rng(1)
    codes, scale, krope = _random_cache(r, 128, 128, 32, "int8")
    keep = [codes.cuda(), scale.cuda(), krope.cuda(), torch.tensor([200], dtype=torch.int32, device="cuda"),
            torch.tensor([[1, -3, 2 ** 30]], dtype=torch.int32, device="cuda")]
    out = torch.full((1, 200, 192), 7.0, dtype=torch.bfloat16, device="cuda")
    hra.cache_load(hra.make_load_params(keep[0], keep[2], keep[3], out, block_table=keep[4], page_size=64, ckv_scale=keep[1],
                                        scale_block=32))
    got = out[0].double().cpu().numpy()
    assert (got[64:] == 0).all() and np.array_equal(got[:64, 128:], krope[64:].double().numpy())


def test_operators_on_another_stream_and_twice_at_once():
    """Two appends and two loads on two streams at once, each on buffers of its own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for k, st in enumerate(streams):
        r = np.random.default_rng(20 + k)
        slots = list(range(7, 700))
        before, got, want = _append(r, slots, slots, rows=768, d_c=512, block=64, fmt="int8", stream=st)
        results.append((before, got, want, slots))
    for before, got, want, slots in results:
        _check_append(before, got, want, slots, block=64, fmt="int8", d_c=512)
