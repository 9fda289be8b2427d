"""The paged 8-bit latent cache, from request lengths to attention, as it is measured.

Four operators: the page plan of one step (block tables, slot map), the append of new tokens
into the cache (int8 or e4m3 with one scale per block of tokens and 128-wide latent head),
the load of cached rows back to bf16 rows (what prefill reads), and the decode over that
cache.  ``run`` computes each in its plain form, elementary torch operations in 32 bits (64
where a value next to a rounding border or a far position's angle needs it), or, where
``own`` is true, through this repository's entry points.  ``exact`` computes the same from
the definitions in 64 bits.
"""
import math
import random

import torch

own = False

ROPE = 64       # width of the shared RoPE key
NOPE = 128      # no-position width of a query head, and width of a value head
HEAD = 128      # latent columns that share a scale (one MLRA-4 branch)
THETA = 10000.0
TOP = {"int8": 127.0, "e4m3": 448.0}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a serving batch: 64 requests, one token each, 64-token pages.
        dict(name="plan_step_b64", op="plan", batch=64, page=64, max_pages=512, chunk=1, max_tokens=64),
        # A scheduling step at the largest batch: prompt chunks, single tokens, idle and finished requests.
        dict(name="plan_mixed_b1024", op="plan", batch=1024, page=64, max_pages=256, chunk=96, max_tokens=65536),
        # The cache write of that decode step (64 open blocks).
        dict(name="append_step_b64", op="append", batch=64, new=1, cached=500, page=64, block=64, d_c=512, fmt="int8",
             pad=0),
        # A prompt's cache write: 8 requests of about 1000 tokens into e4m3.
        dict(name="append_prompt_8k", op="append", batch=8, new=1024, cached=0, page=64, block=64, d_c=512,
             fmt="e4m3", pad=37),
        # Chunked prompts of a rank that holds one branch: ragged chunks that open and end inside blocks of 32.
        dict(name="append_shard_32k", op="append", batch=33, new=1000, cached=77, page=128, block=32, d_c=128,
             fmt="int8", pad=0),
        # A 2048-token prefix back to bf16 rows for prefill (the h = 16 model's context).
        dict(name="load_prefix_2k", op="load", batch=1, tokens=2048, page=64, block=64, d_c=512, fmt="int8"),
        # Long prefixes of a ragged batch.
        dict(name="load_ragged_128k", op="load", batch=6, tokens=40000, page=64, block=64, d_c=512, fmt="e4m3"),
        # The smallest decode: one sequence of the h = 16 model.
        dict(name="decode_h16_2k", op="decode", batch=1, heads=16, low=2048, high=2048, page=0, block=64, d_c=512,
             fmt="int8"),
        # Short ragged requests, one of them with a single token.
        dict(name="decode_ragged_b32", op="decode", batch=32, heads=128, low=1, high=4096, page=64, block=64, d_c=512,
             fmt="e4m3"),
        # The paged serving batch: 64 requests at 32k tokens.
        dict(name="decode_paged_b64_32k", op="decode", batch=64, heads=128, low=32768, high=32768, page=64, block=64,
             d_c=512, fmt="int8"),
        # One branch of four (4-way tensor parallelism), ragged lengths.
        dict(name="decode_shard_b32_16k", op="decode", batch=32, heads=128, low=12000, high=16384, page=64, block=64,
             d_c=128, fmt="int8"),
        # One long sequence, contiguous, half of the heads.
        dict(name="decode_long_100k", op="decode", batch=1, heads=64, low=100003, high=100003, page=0, block=128,
             d_c=512, fmt="e4m3"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("plan", "append", "load", "decode", "decode"))
    if op == "plan":
        batch, chunk = _spread(rng, 1, 1024), _spread(rng, 1, 96)
        return dict(op=op, batch=batch, page=rng.choice((32, 64, 128)), max_pages=rng.randint(64, 512), chunk=chunk,
                    max_tokens=max(batch, min(65536, batch * chunk + rng.randint(0, 64))))
    fmt, d_c = rng.choice(("int8", "e4m3")), rng.choice((128, 256, 512, 512))
    page = rng.choice((32, 64, 128))
    block = rng.choice([b for b in (32, 64, 128) if b <= page])
    if op == "append":
        batch = _spread(rng, 1, 64)
        return dict(op=op, batch=batch, new=_spread(rng, 1, max(1, 16384 // batch)), cached=rng.randint(0, 700),
                    page=page, block=block, d_c=d_c, fmt=fmt, pad=rng.randint(0, 9))
    if op == "load":
        batch = _spread(rng, 1, 16)
        return dict(op=op, batch=batch, tokens=_spread(rng, 1, 200000 // batch), page=page, block=block, d_c=d_c, fmt=fmt)
    batch = _spread(rng, 1, 64)
    high = _spread(rng, 16, 2000000 // batch)
    return dict(op=op, batch=batch, heads=rng.choice((1, 8, 16, 40, 64, 128, 128)), low=rng.choice((1, high)), high=high,
                page=rng.choice((0, page)), block=block, d_c=d_c, fmt=fmt)


def _lengths(case, low, high):
    """The case's lengths, the same for every seed (they decide the work): uniform in [low, high], both ends met."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = [r.randint(low, high) for _ in range(case["batch"])]
    n[0] = high
    if len(n) > 1:
        n[1] = low
    return n


def _plan_lengths(case):
    """Cached lengths and new tokens of a plan's requests: mostly running ones, some new, idle or finished."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    room, left = case["max_pages"] * case["page"] - case["chunk"], case["max_tokens"]
    cached, new = [], []
    for _ in range(case["batch"]):
        kind = r.random() if case["chunk"] > 1 else 0.5
        cached.append(0 if kind < 0.1 else r.randint(1, room))
        n = 1 if case["chunk"] == 1 else -1 if kind > 0.95 else 0 if kind > 0.85 else r.randint(1, case["chunk"])
        new.append(min(n, left))
        left -= max(new[-1], 0)
    return cached, new


def _append_lengths(case):
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b = case["batch"]
    new = [case["new"]] * b if case["new"] == 1 else [r.randint(max(1, case["new"] // 2), case["new"]) for _ in range(b)]
    return [r.randint(case["cached"] // 2, case["cached"]) for _ in range(b)], new


def work(case):
    """What one pass reads, writes and computes at the least."""
    d_c = case.get("d_c", 0)
    row8, row16, scales = d_c + 2 * ROPE, 2 * (d_c + ROPE), 4 * (d_c // HEAD)
    if case["op"] == "plan":
        cached, new = _plan_lengths(case)
        ceil = lambda n: -(-n // case["page"])  # noqa: E731
        pages = sum(ceil(c) if n < 0 else ceil(c + n) - ceil(c) for c, n in zip(cached, new))
        # lengths and new tokens in, lengths and starts out, a page number read and written, slots and positions out
        return {"bytes": 16 * case["batch"] + 8 * pages + 8 * case["max_tokens"], "flops": 0}
    if case["op"] == "append":
        cached, new = _append_lengths(case)
        n = sum(new)
        blocks = sum((c + m - 1) // case["block"] - c // case["block"] + 1 for c, m in zip(cached, new))
        return {"bytes": n * (row16 + 8 + row8 + row16) + blocks * 2 * scales, "flops": n * (2 * d_c + 4 * ROPE)}
    if case["op"] == "load":
        n = sum(_lengths(case, max(1, case["tokens"] // 2), case["tokens"]))
        return {"bytes": n * (row8 + row16) + -(-n // case["block"]) * scales, "flops": n * d_c}
    lens, h = _lengths(case, case["low"], case["high"]), case["heads"]
    n, b = sum(lens), case["batch"]
    return {"bytes": n * row8 + -(-n // case["block"]) * scales + 4 * h * d_c * NOPE + 2 * b * h * (NOPE + ROPE + NOPE),
            "flops": 2 * n * h * (2 * d_c + ROPE) + 4 * b * h * d_c * NOPE}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _to_codes(y, fmt):
    """Quotients x / s (64 bits) to the nearest value of the 8-bit format, ties to even, in 64 bits."""
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    step = torch.exp2(torch.frexp(y.abs())[1].to(torch.float64).sub(1).clamp(min=-6) - 3)  # e4m3's spacing at y
    return ((y / step).round() * step).clamp(-448, 448)


def _quantize(x, block, fmt):
    """Rows x [R, d_c] (R a multiple of the block) to codes and scales [R / block, d_c / 128]."""
    xb = x.float().view(-1, block, x.shape[1] // HEAD, HEAD)
    scale = (xb.abs().amax(dim=(1, 3)).double() / TOP[fmt]).float()
    s = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None, :, None]
    codes = _to_codes(xb.double().div_(s.double()), fmt)
    return codes.to(torch.float32).to(STORE[fmt]).view(x.shape), scale


def _cache(g, rows, case):
    """A filled cache of `rows` rows, in pieces so that the 64-bit quotients stay small."""
    block, fmt, d_c = case["block"], case["fmt"], case["d_c"]
    codes = torch.empty(rows, d_c, dtype=STORE[fmt], device="cuda")
    scale = torch.empty(rows // block, d_c // HEAD, device="cuda")
    piece = 32768
    for r in range(0, rows, piece):
        n = min(piece, rows - r)
        # tokens differ in size, as latents do
        x = (_normal(g, n, d_c) * torch.exp(0.25 * _normal(g, n, 1))).to(torch.bfloat16)
        codes[r:r + n], scale[r // block:(r + n) // block] = _quantize(x, block, fmt)
    return codes, scale, _normal(g, rows, ROPE).to(torch.bfloat16)


def _table(g, lens, page):
    """Pages of each sequence, in random order over the pool; entries past a sequence's pages are -1."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "plan":
        cached, new = _plan_lengths(case)
        page, wide = case["page"], case["max_pages"]
        have = torch.tensor([-(-c // page) for c in cached], device="cuda")
        used = int(have.sum())
        pages = used + case["max_tokens"] // page + 2 * case["batch"]
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        cols = torch.arange(wide, device="cuda")[None]
        mine = (have.cumsum(0) - have)[:, None] + cols
        table = torch.where(cols < have[:, None], order[mine.clamp(max=pages - 1)], -1).to(torch.int32)
        # the free pages lie in a ring, from a place that differs from run to run
        head = int(torch.randint(0, 1 << 20, (1,), generator=g, device="cuda"))
        ring = torch.empty(pages, dtype=torch.int32, device="cuda")
        at = (head + torch.arange(pages, device="cuda")) % pages
        ring[at] = order.roll(-used)
        n = case["max_tokens"]
        return dict(case=case, lens=_ints(cached), new=_ints(new), table=table, ring=ring,
                    free=torch.tensor([head, head + pages - used], dtype=torch.int64, device="cuda"),
                    lens_out=torch.zeros(case["batch"], dtype=torch.int32, device="cuda"),
                    free_out=torch.zeros(2, dtype=torch.int64, device="cuda"),
                    start=torch.zeros(case["batch"] + 1, dtype=torch.int32, device="cuda"),
                    slots=torch.zeros(n, dtype=torch.int32, device="cuda"),
                    positions=torch.zeros(n, dtype=torch.int32, device="cuda"),
                    status=torch.zeros(4, dtype=torch.int32, device="cuda"))
    if op == "append":
        cached, new = _append_lengths(case)
        page, d_c = case["page"], case["d_c"]
        table, pages = _table(g, [c + n for c, n in zip(cached, new)], page)
        codes, scale, krope = _cache(g, pages * page, case)
        count = sum(new) + case["pad"]
        rows = (_normal(g, count, d_c + ROPE) * torch.exp(0.25 * _normal(g, count, 1))).to(torch.bfloat16)
        c, n = torch.tensor(cached, device="cuda"), torch.tensor(new, device="cuda")
        seq = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), n)
        pos = torch.arange(sum(new), device="cuda") - (n.cumsum(0) - n)[seq] + c[seq]
        slots = torch.full((count,), -1, dtype=torch.int32, device="cuda")
        positions = torch.full((count,), -1, dtype=torch.int32, device="cuda")
        slots[:sum(new)] = table[seq, pos // page] * page + (pos % page).to(torch.int32)
        positions[:sum(new)] = pos.to(torch.int32)
        # the projection's output holds latent and RoPE key side by side
        return dict(case=case, rows=rows, slots=slots, positions=positions, codes=codes, scale=scale, krope=krope,
                    out=torch.zeros(count, d_c + ROPE, dtype=torch.bfloat16, device="cuda"))
    if op == "load":
        lens = _lengths(case, max(1, case["tokens"] // 2), case["tokens"])
        table, pages = _table(g, lens, case["page"])
        codes, scale, krope = _cache(g, pages * case["page"], case)
        return dict(case=case, lens=_ints(lens), table=table, codes=codes, scale=scale, krope=krope,
                    out=torch.zeros(case["batch"], case["tokens"], case["d_c"] + ROPE, dtype=torch.bfloat16, device="cuda"))
    lens, d_c, h, b = _lengths(case, case["low"], case["high"]), case["d_c"], case["heads"], case["batch"]
    if case["page"]:
        table, pages = _table(g, lens, case["page"])
        rows, stride = pages * case["page"], 0
    else:
        table, stride = None, -(-max(lens) // case["block"]) * case["block"]
        rows = b * stride
    codes, scale, krope = _cache(g, rows, case)
    std = 1.0 / math.sqrt(HEAD)
    return dict(case=case, lens=_ints(lens), table=table, stride=stride, codes=codes, scale=scale, krope=krope,
                q=_normal(g, b, h, NOPE + ROPE).to(torch.bfloat16),
                w_uk=(_normal(g, h, d_c, NOPE) * std).to(torch.bfloat16),
                w_uv=(_normal(g, h, d_c, NOPE) * std).to(torch.bfloat16),
                out=torch.zeros(b, h, NOPE, dtype=torch.bfloat16, device="cuda"))


# --------------------------------------------------------------------------- the passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "load": _own_load, "decode": _own_decode}[op](state)
    return {"plan": _plan, "append": _append, "load": _load, "decode": _decode}[op](state)


def _own_plan(s):
    import head_rank_attention_b200 as hra
    if "params" not in s:  # filled once for a program's buffers, like every parameter block below
        s["params"] = hra.make_plan_params(s["lens"], s["new"], s["table"], s["ring"], s["free"], s["lens_out"],
                                           s["free_out"], s["start"], s["slots"], s["status"],
                                           positions=s["positions"], page_size=s["case"]["page"])
    hra.page_plan(s["params"])
    return {"lens": s["lens_out"], "table": s["table"], "ring": s["ring"], "free": s["free_out"], "start": s["start"],
            "slots": s["slots"], "positions": s["positions"], "status": s["status"]}


def _own_append(s):
    import head_rank_attention_b200 as hra
    if "params" not in s:
        d_c = s["case"]["d_c"]
        s["params"] = hra.make_append_params(s["rows"][:, :d_c], s["rows"][:, d_c:], s["slots"], s["positions"],
                                             s["codes"], s["krope"], ckv_scale=s["scale"],
                                             scale_block=s["case"]["block"], rows_out=s["out"], rope_theta=THETA)
    hra.cache_append(s["params"])
    return {"rows": s["out"], "codes": s["codes"], "scale": s["scale"], "krope": s["krope"]}


def _own_load(s):
    import head_rank_attention_b200 as hra
    if "params" not in s:
        s["params"] = hra.make_load_params(s["codes"], s["krope"], s["lens"], s["out"], block_table=s["table"],
                                           page_size=s["case"]["page"], ckv_scale=s["scale"],
                                           scale_block=s["case"]["block"])
    hra.cache_load(s["params"])
    return s["out"]


def _own_decode(s):
    import head_rank_attention_b200 as hra
    if "params" not in s:
        c = s["case"]
        s["params"] = hra.make_params(s["q"], s["codes"], s["krope"], s["lens"], s["w_uk"], s["w_uv"], s["out"],
                                      n_branch=c["d_c"] // HEAD, branch_scale=0.5, rope_theta=THETA,
                                      block_table=s["table"], page_size=c["page"], seq_stride=s["stride"],
                                      ckv_scale=s["scale"], scale_block=c["block"])
        s["workspace"] = hra.alloc_workspace(s["params"])
    hra.mlra_decode(s["params"])
    return s["out"]


def _plan(s):
    c = s["case"]
    page, wide, n = c["page"], c["max_pages"], s["ring"].numel()
    lens, new = s["lens"].long(), s["new"].long()
    gone = new < 0
    add = new.clamp(min=0)
    after = torch.where(gone, 0, lens + add)
    have, want = (lens + page - 1) // page, (after + page - 1) // page
    need, freed = torch.where(gone, 0, want - have), torch.where(gone, have, 0)
    cols = torch.arange(wide, device=lens.device)[None]
    # the call's pages come off the ring's head in the order of the sequences
    taken = (s["free"][0] + (need.cumsum(0) - need)[:, None] + cols - have[:, None]) % n
    fresh = (cols >= have[:, None]) & (cols < want[:, None])
    table = torch.where(fresh, s["ring"][taken], s["table"])
    # finished requests' pages go to its tail
    back = (s["free"][1] + (freed.cumsum(0) - freed)[:, None] + cols) % n
    back = torch.where(gone[:, None] & (cols < have[:, None]), back, n)
    ring = torch.cat([s["ring"], s["ring"][:1]]).scatter(0, back.view(-1), s["table"].view(-1))[:n]
    start = torch.cat([add.new_zeros(1), add.cumsum(0)])
    t = torch.arange(c["max_tokens"], device=lens.device)
    seq = torch.searchsorted(start[1:], t, right=True).clamp(max=c["batch"] - 1)
    pos = lens[seq] + t - start[seq]
    slot = table[seq, (pos // page).clamp(0, wide - 1)].long() * page + pos % page
    live = t < start[-1]
    free = s["free"] + torch.stack([need.sum(), freed.sum()])
    i32 = torch.int32
    return {"lens": after.to(i32), "table": table, "ring": ring, "free": free, "start": start.to(i32),
            "slots": torch.where(live, slot, -1).to(i32), "positions": torch.where(live, pos, -1).to(i32),
            "status": torch.zeros_like(s["status"])}


def _turned(k, positions):
    """RoPE of k [..., 64] at positions: pairs (j, j + 32), the angle in 64 bits."""
    inv = THETA ** (-torch.arange(0, ROPE, 2, device=k.device, dtype=torch.float64) / ROPE)
    angle = positions.double()[:, None] * inv
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = k[..., :ROPE // 2].float(), k[..., ROPE // 2:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _append(s):
    c = s["case"]
    block, fmt, d_c = c["block"], c["fmt"], c["d_c"]
    rows, groups = s["codes"].shape[0], d_c // HEAD
    count = rows // block
    x, k = s["rows"][:, :d_c].float().view(-1, groups, HEAD), s["rows"][:, d_c:]
    slot = s["slots"].long()
    live = slot >= 0
    at = torch.where(live, slot, rows)                         # padding goes to a row that is dropped
    blk, off = at // block, at % block
    # per block: the new rows' largest magnitude, the first of them, and the scale
    peak = x.new_zeros(count + 1, groups).scatter_reduce(0, blk[:, None].expand(-1, groups), x.abs().amax(-1), "amax")[:count]
    first = off.new_full((count + 1,), block).scatter_reduce(0, blk, off, "amin")[:count]
    touched = (first < block)[:, None]
    old = torch.where((first > 0)[:, None], s["scale"], 0.0)
    scale = torch.where(touched, torch.maximum(old, (peak.double() / TOP[fmt]).float()), s["scale"])
    # rows written before the call are brought to the block's new scale where it grew
    grew = touched & (first > 0)[:, None] & (scale > s["scale"])
    grown = grew[:, None, :] & (torch.arange(block, device=x.device)[None] < first[:, None])[:, :, None]
    codes = s["codes"].view(count, block, groups, HEAD).float()
    over = torch.where(scale > 0, scale, 1.0).double()[:, None, :, None]
    again = _to_codes(codes.double() * s["scale"].double()[:, None, :, None] / over, fmt).float()
    codes = torch.where(grown[..., None], again, codes).view(rows, d_c)
    mine = torch.cat([scale, scale[:1]])[blk]                     # each token's scales
    safe = torch.where(mine > 0, mine, 1.0)
    new = _to_codes(x.double() / safe.double()[:, :, None], fmt).float()
    codes = torch.cat([codes, codes[:1]]).index_copy(0, at, new.view(-1, d_c))[:rows]
    turned = _turned(k, s["positions"]).to(torch.bfloat16)
    krope = torch.cat([s["krope"], s["krope"][:1]]).index_copy(0, at, turned)[:rows]
    out = torch.cat([(new * mine[:, :, None]).view(-1, d_c).to(torch.bfloat16), turned], dim=1)
    return {"rows": torch.where(live[:, None], out, s["out"]), "codes": codes.to(STORE[fmt]), "scale": scale, "krope": krope}


def _rows_of(s, width):
    """Each sequence's cache rows [B, width], and which of them it has."""
    c = s["case"]
    t = torch.arange(width, device=s["lens"].device)
    if s["table"] is None:
        row = torch.arange(c["batch"], device=t.device)[:, None] * s["stride"] + t[None]
    else:
        row = s["table"][:, t // c["page"]].long() * c["page"] + t % c["page"]
    return row.clamp(0, s["codes"].shape[0] - 1), t[None] < s["lens"][:, None]


def _dequantized(s, row):
    """The latents [B, T, groups, 128] that the cache stands for, in 32 bits."""
    c = s["case"]
    codes = s["codes"].view(torch.int8)[row].view(s["codes"].dtype).float()  # gathered as bytes
    return codes.view(*row.shape, c["d_c"] // HEAD, HEAD) * s["scale"][row // c["block"]][..., None]


def _load(s):
    c = s["case"]
    row, live = _rows_of(s, c["tokens"])
    x = _dequantized(s, row).view(*row.shape, c["d_c"])
    out = torch.cat([x.to(torch.bfloat16), s["krope"][row]], dim=2)
    return torch.where(live[:, :, None], out, s["out"])


def _decode(s):
    c = s["case"]
    groups, b, h = c["d_c"] // HEAD, c["batch"], c["heads"]
    row, live = _rows_of(s, c["high"])
    x = _dequantized(s, row)                                                # [B, T, g, 128]
    q = s["q"].float()
    absorbed = torch.einsum("bhn,hcn->bhc", q[..., :NOPE], s["w_uk"].float()).view(b, h, groups, HEAD).transpose(1, 2)
    turned = _turned(q[..., NOPE:].transpose(0, 1), s["lens"] - 1).transpose(0, 1)   # [B, h, 64]
    score = absorbed @ x.permute(0, 2, 3, 1)                                # [B, g, h, T]
    score += (turned @ s["krope"][row].float().transpose(1, 2))[:, None]
    score *= 1.0 / math.sqrt(NOPE + ROPE)
    score.masked_fill_(~live[:, None, None, :], -math.inf)
    score -= score.amax(dim=-1, keepdim=True)
    score.exp_()
    total = score.sum(dim=-1, keepdim=True)
    latent = (score @ x.transpose(1, 2)) / total                            # [B, g, h, 128]
    out = torch.einsum("bghc,hgcv->bhv", latent, s["w_uv"].float().view(h, groups, HEAD, NOPE))
    return (0.5 * out).to(torch.bfloat16)


# ------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    """The outputs from the definitions in 64 bits, sequence by sequence; a plan has whole numbers only."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "load": _exact_load, "decode": _exact_decode}[case["op"]](s)


def _values(codes, scale, block):
    """Codes [n, d_c] whose rows lie in the blocks that `block` names, times their scales."""
    return codes.float().double() * scale.double()[block].repeat_interleave(HEAD, dim=1)


def _complex_turn(k, positions):
    j = torch.arange(ROPE // 2, device=k.device, dtype=torch.float64)
    turn = torch.polar(torch.ones_like(j)[None].expand(len(positions), -1).contiguous(),
                       positions.double()[:, None] * torch.exp(j * (-2.0 / ROPE) * math.log(THETA)))
    k = k.double()
    z = torch.complex(k[..., :ROPE // 2], k[..., ROPE // 2:]) * turn
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_append(s):
    """Block by block: scales are 32-bit numbers by the format's definition, codes the nearest values, ties to even."""
    c = s["case"]
    block, d_c, top = c["block"], c["d_c"], TOP[c["fmt"]]
    slots = s["slots"].cpu()
    n = int((slots >= 0).sum())
    where = slots[:n].long().cuda()
    values = s["rows"][:, :d_c].double()
    codes, scale = s["codes"].float().double(), s["scale"].clone()
    runs, begin = [], 0
    for i in range(1, n + 1):
        if i == n or int(slots[i]) // block != int(slots[i - 1]) // block:
            runs.append((begin, i))
            begin = i
    out = torch.zeros(len(slots), d_c, dtype=torch.float64, device="cuda")
    for a, e in runs:
        blk, first = int(slots[a]) // block, int(slots[a]) % block
        x = values[a:e].view(e - a, -1, HEAD)
        s32 = (x.abs().amax(dim=(0, 2)) / top).float()
        if first:
            s32 = torch.maximum(s32, scale[blk])
            before = codes[blk * block:blk * block + first].view(first, -1, HEAD)
            again = _nearest(before * scale[blk].double()[None, :, None] / s32.double()[None, :, None], c["fmt"])
            grown = (s32 > scale[blk])[None, :, None]
            codes[blk * block:blk * block + first] = torch.where(grown, again, before).view(first, d_c)
        scale[blk] = s32
        new = _nearest(x / s32.double()[None, :, None], c["fmt"])
        codes[where[a:e]] = new.view(e - a, d_c)
        out[a:e] = (new * s32.double()[None, :, None]).view(e - a, d_c)
    turned = _complex_turn(s["rows"][:n, d_c:], s["positions"][:n])
    krope = s["krope"].double()
    krope[where] = turned
    rows = torch.zeros(len(slots), d_c + ROPE, dtype=torch.float64, device="cuda")
    rows[:n] = torch.cat([out[:n], turned], dim=1)
    # int8 codes are whole numbers: they have no other value to be near to
    return {"rows": rows, "codes": None if c["fmt"] == "int8" else codes, "scale": scale.double(), "krope": krope}


def _nearest(y, fmt):
    """The nearest value of the format by distance, an even code on a tie."""
    if fmt == "int8":
        low = y.floor()
        high_wins = (y - low > 0.5) | ((y - low == 0.5) & (low.remainder(2) == 1))
        return (low + high_wins).clamp(-127, 127)
    size = y.abs()
    grid = torch.arange(127, dtype=torch.uint8, device=y.device).view(torch.float8_e4m3fn).double()  # codes 0 .. 126
    high = torch.searchsorted(grid, size.contiguous()).clamp(max=126)
    low = (high - 1).clamp(min=0)
    up, down = grid[high] - size, size - grid[low]
    code = torch.where((up < down) | ((up == down) & (high % 2 == 0)), high, low)
    return torch.copysign(grid[code], y)


def _exact_load(s):
    c = s["case"]
    out = s["out"].double()
    for b, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device="cuda")
        row = s["table"][b, t // c["page"]].long() * c["page"] + t % c["page"]
        out[b, :n, :c["d_c"]] = _values(s["codes"].view(torch.int8)[row].view(s["codes"].dtype), s["scale"], row // c["block"])
        out[b, :n, c["d_c"]:] = s["krope"][row].double()
    return out


def _exact_decode(s):
    c = s["case"]
    out = torch.zeros(c["batch"], c["heads"], NOPE, dtype=torch.float64, device="cuda")
    w_uk, w_uv = s["w_uk"].double(), s["w_uv"].double()
    for b, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device="cuda")
        row = b * s["stride"] + t if s["table"] is None else s["table"][b, t // c["page"]].long() * c["page"] + t % c["page"]
        latent = _values(s["codes"].view(torch.int8)[row].view(s["codes"].dtype), s["scale"], row // c["block"])
        q = s["q"][b].double()
        rope = _complex_turn(q[None, :, NOPE:].transpose(0, 1), torch.full((1,), n - 1, device="cuda"))[:, 0]
        shared = s["krope"][row].double() @ rope.T                          # [n, h]
        for g in range(c["d_c"] // HEAD):
            cols = slice(HEAD * g, HEAD * (g + 1))
            side = (w_uk[:, cols] @ q[:, :NOPE, None])[..., 0]              # [h, 128]
            p = torch.softmax((latent[:, cols] @ side.T + shared) / math.sqrt(NOPE + ROPE), dim=0)
            mixed = p.T @ latent[:, cols]                                   # [h, 128]
            out[b] += 0.5 * (mixed[:, None, :] @ w_uv[:, cols])[:, 0]
    return out
