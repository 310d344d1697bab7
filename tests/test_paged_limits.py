"""Paged 8-bit KV cache at its limits: lengths that disagree with the free ring, value scales far apart, the smallest
and the largest magnitudes, skipped and misplaced tokens, bad pointers, and batches of many hundred requests."""
import random

import numpy as np
import pytest

import rank_gemm_svdq_b200 as sv
from oracle import pagedkv as pk
from tests.test_paged import UNIT, Pool, call_append, call_attend, call_plan, dev, dtype_of, make_table, raw_batch, raw_cache


def both(P, q, new, lens, table, causal=True, dtype="bf16", scale=None, max_new=None):
    """Attention of q (tokens x heads d, 16-bit values held in float32) over the pool, by the kernels and the oracle:
    the 16-bit result, its values, the oracle's and how far a value may be off."""
    import torch
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(cu[-1])
    want, tol = pk.attend(q.double().numpy().reshape(n, P.heads, P.d), cu, lens, table, P.codes[0], P.scale[0], P.codes[1], P.scale[1],
                          P.fmt, causal, P.d ** -0.5 if scale is None else scale, UNIT[dtype])
    c = P.to_device()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(cu), None, n_tokens=n, max_new=max_new or max(new), max_len=max(lens))
    ws = torch.full((sv.paged_attention_workspace_bytes(c, b),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((n, P.heads * P.d), 7.0, dtype=dtype_of(dtype), device="cuda")
    sv.paged_attention(c, b, q.to(dtype_of(dtype)).cuda(), out, ws, causal=causal, scale=scale)
    return out.cpu(), out.double().cpu().numpy().reshape(n, P.heads, P.d), want, tol


def normal(rng, n, cols, dtype="bf16", power=0):
    """Random 16-bit values times a power of two."""
    import torch
    x = torch.from_numpy(rng.normal(size=(n, cols)).astype(np.float32)).to(dtype_of(dtype)).float() * 2.0 ** power
    return x.to(dtype_of(dtype)).float()


def within(got, want, tol):
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(np.argmax(off), off.shape))


# A shape for each kernel and each way of sharing the work out: heads, kv, d, bs, new, lens.  The last block of every
# request holds a few tokens of its own, so that some of its new rows do not see that block.
PATHS = [
    (4, 4, 64, 16, [8], [101]),                            # a CTA a cell
    (4, 2, 128, 16, [4, 3], [2003, 402]),                  # clusters
    (8, 2, 64, 32, [3], [514]),                            # clusters, 9 to 16 rows
    (2, 2, 128, 32, [7], [8996]),                          # one long request over the whole chip, cut and joined
    (8, 1, 64, 64, [2], [6017]),                           # the same, 9 to 16 rows
    (4, 4, 64, 16, [6] * 45, [85 + 16 * (i % 40) for i in range(45)]),   # many cells: shares cut inside requests
    (16, 4, 128, 64, [4] * 50, [66] * 50),                 # 16 rows, whole items
    (2, 1, 64, 16, [40, 33], [101, 340]),                  # tensor-core rows
    (4, 2, 128, 64, [300], [1064]),                        # the same, cut and joined
]
BOTH_FORMATS = [("int8", "bf16"), ("e4m3", "fp16")]


def pool(seed, heads, kv, d, bs, lens, fmt, dtype):
    P = Pool(seed, heads, kv, d, bs, sum(-(-L // bs) for L in lens) + 2, fmt, dtype)
    return P, make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens) + 1, fill=-1)


# -------------------------------------------- the plan: what is given back has to fit the ring
# One request takes 3 blocks, another gives 4 back: the ring would hold 8 - 3 + 4 = 9 of 10, but the four entries
# from head + count on are 8, 9, 0, 1, and 0 and 1 are also read as blocks to take.
OVERFULL = dict(prev=[0, 64], target=[48, 0], state=(0, 8), n_blocks=10, bs=16)


def test_plan_never_writes_a_ring_entry_that_it_reads():
    r = random.Random(5)
    accepted = 0
    for k in range(4000):
        n, bs, B = r.randint(1, 12), 16, r.randint(1, 4)
        prev, target = [r.randint(0, 6 * bs) for _ in range(B)], [r.randint(0, 6 * bs) for _ in range(B)]
        head, count = r.randrange(n), r.randint(0, n)
        if k == 0:
            prev, target, (head, count), n = OVERFULL["prev"], OVERFULL["target"], OVERFULL["state"], OVERFULL["n_blocks"]
            B = 2
        got = pk.plan(prev, target, np.zeros((B, 8), np.int32), np.arange(n, dtype=np.int32), head, count, bs, 10 ** 4, 10 ** 4, 8 * bs)
        if got["state"][2] != 0:
            continue
        accepted += 1
        blocks = lambda t: -(-t // bs)  # noqa: E731
        take = sum(max(0, blocks(t) - blocks(p)) for p, t in zip(prev, target))
        give = sum(max(0, blocks(p) - blocks(t)) for p, t in zip(prev, target))
        read, written = {(head + i) % n for i in range(take)}, [(head + count + i) % n for i in range(give)]
        assert len(set(written)) == give and not read & set(written), (k, prev, target, head, count, n)
    assert accepted > 100


@pytest.mark.gpu
def test_plan_refuses_more_blocks_than_the_ring_has_room_for(gpu):
    import torch
    c = OVERFULL
    table, ring = np.arange(16, dtype=np.int32).reshape(2, 8) % 10, np.arange(10, dtype=np.int32)[::-1].copy()
    want = pk.plan(c["prev"], c["target"], table, ring, *c["state"], c["bs"], 60, 60, 128)
    assert want["state"][2] == -1
    t = dict(table=dev(table), ring=dev(ring), lens=torch.zeros(2, dtype=torch.int32).cuda(), cu=torch.ones(3, dtype=torch.int32).cuda(),
             slots=torch.ones(60, dtype=torch.int32).cuda())
    b = sv.paged_batch(t["table"], t["lens"], t["cu"], t["slots"], max_new=60, max_len=128)
    out = torch.zeros(4, dtype=torch.int32).cuda()
    sv.paged_plan(b, c["bs"], dev(np.array(c["prev"], np.int32)), dev(np.array(c["target"], np.int32)), t["ring"],
                  dev(np.array([*c["state"], 0, 0], np.int32)), out)
    for name in t:
        assert np.array_equal(t[name].cpu().numpy(), want[name]), name
    assert np.array_equal(out.cpu().numpy(), want["state"])


# ------------------------------------------------- value scales far apart
@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt,dtype", BOTH_FORMATS)
def test_rows_do_not_depend_on_what_they_do_not_see(gpu, heads, kv, d, bs, new, lens, fmt, dtype):
    """Other keys and values, with scales 2^4 to 2^30 larger, in the blocks that only later rows see: the same bits."""
    import torch
    P, table = pool(sum(lens), heads, kv, d, bs, lens, fmt, dtype)
    q = normal(P.rng, sum(new), heads * d, dtype)
    base, got, want, tol = both(P, q, new, lens, table, dtype=dtype)
    within(got, want, tol)
    starts, blind = np.concatenate([[0], np.cumsum(new)]), []
    for i, (m, L) in enumerate(zip(new, lens)):
        lead = (L - 1) // bs * bs                          # the last block's first token
        blind += [starts[i] + j for j in range(m) if L - m + j + 1 <= lead]
    assert len(blind) >= len(new)
    P2, _ = pool(77, heads, kv, d, bs, lens, fmt, dtype)
    for power in (4, 30):
        if dtype == "fp16" and power > 4:
            continue                                       # the later rows' results would not be fp16 numbers
        for i, L in enumerate(lens):
            blk = int(table[i, (L - 1) // bs])
            P.codes[:, blk] = P2.codes[:, blk]
            P.scale[:, blk] = P2.scale[:, blk] * np.array([[1.0], [2.0 ** power]], np.float32)
        bits, got, want, tol = both(P, q, new, lens, table, dtype=dtype)
        assert torch.equal(bits[blind], base[blind])
        within(got, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt,dtype", BOTH_FORMATS)
@pytest.mark.parametrize("causal", [True, False])
def test_large_values_of_no_weight(gpu, heads, kv, d, bs, new, lens, fmt, dtype, causal):
    """Every third block holds values 2^40 larger at scores 60 below the others': weights of e^-60 leave nothing of them,
    and what the others add keeps its bits.  Every fifth holds values 2^30 smaller."""
    P, table = pool(sum(lens) + 1, heads, kv, d, bs, lens, fmt, dtype)
    n = sum(new)
    q = normal(P.rng, n, heads * d, dtype).abs() * 0.25 + 0.75
    q = q.to(dtype_of(dtype)).float()
    low = np.zeros(P.n, bool)
    for i in range(len(lens)):
        low[table[i, 1::3]] = True
        P.scale[1, table[i, 2::5]] *= np.float32(2.0 ** -30)
    low[table[:, 0]] = False                               # every row sees a block of ordinary scores
    P.codes[0, low] = pk.to_codes(np.full((1,), -127.0), fmt)[0]
    P.scale[0, low] = 60.0 / (d ** 0.5 * 127.0 * 0.75)     # q >= 0.75: scores of -60 or less
    P.scale[1, low] *= np.float32(2.0 ** 40)
    P.scale[0, ~low] *= np.float32(0.25)
    _, got, want, tol = both(P, q, new, lens, table, causal, dtype)
    within(got, want, tol)
    assert np.abs(got).max() < 1000


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt,dtype", BOTH_FORMATS)
def test_small_weights_of_many_tokens(gpu, heads, kv, d, bs, new, lens, fmt, dtype):
    """The first token takes nearly all of the weight and has a value of 0: what is left are the others, at weights
    of 2^-27 of its own and ordinary values."""
    P, table = pool(sum(lens) + 8, heads, kv, d, bs, lens, fmt, dtype)
    q = normal(P.rng, sum(new), heads * d, dtype) * 0 + 1
    P.codes[0] = pk.to_codes(np.full((1,), 1.0), fmt)[0]
    P.codes[0, table[:, 0], :, 0] = pk.to_codes(np.full((1,), 15.0), fmt)[0]
    P.scale[0] = 27.0 * np.log(2.0) / 14.0 / d ** 0.5      # a step of 14 codes in all values is 27 in log2
    P.codes[1, table[:, 0], :, 0] = 0
    P.codes[1] = P.codes[1] & 0x7F if fmt == "e4m3" else np.abs(P.codes[1].view(np.int8)).view(np.uint8)
    P.scale[1] = np.float32(256.0 if dtype == "fp16" else 1.0)
    _, got, want, tol = both(P, q, new, lens, table, dtype=dtype)
    within(got, want, tol)
    assert (tol < 0.5 * np.abs(want)).mean() > 0.8         # the bound tells a lost tail from a kept one


# ---------------------------------------------------- the smallest and the largest numbers
@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [125, 116, 100, -100, -120])
def test_queries_of_extreme_size(gpu, heads, kv, d, bs, new, lens, fmt, power):
    """Queries near 2^power over keys near 2^-power: the scores are ordinary ones."""
    P, table = pool(sum(lens) + 3, heads, kv, d, bs, lens, fmt, "bf16")
    P.scale[0] = (P.scale[0].astype(np.float64) * 2.0 ** (-power if power > 0 else min(-power, 112))).astype(np.float32)
    _, got, want, tol = both(P, normal(P.rng, sum(new), heads * d, power=power), new, lens, table)
    within(got, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("where", ["first", "all", "last"])
def test_values_of_subnormal_size(gpu, heads, kv, d, bs, new, lens, fmt, where):
    """Blocks as an append leaves them for values of 1 to 3 times 2^-133 (scales near 2^-140), before, without and behind
    ordinary ones."""
    P, table = pool(sum(lens) + 2, heads, kv, d, bs, lens, fmt, "bf16")
    for i, L in enumerate(lens):
        nb = -(-L // bs)
        for c in {"first": range(0, max(1, nb // 2)), "all": range(nb), "last": range(nb // 2, nb)}[where]:
            blk = int(table[i, c])
            x = (P.rng.integers(1, 4, size=(bs, kv, d)) * np.where(P.rng.random((bs, kv, d)) < 0.5, 1, -1)) * 2.0 ** -133
            P.codes[1], P.scale[1] = pk.append(x, np.arange(blk * bs, (blk + 1) * bs), [0, bs], P.codes[1], P.scale[1], fmt)
            assert 0 < P.scale[1, blk].max() < 2.0 ** -137
    _, got, want, tol = both(P, normal(P.rng, sum(new), heads * d), new, lens, table)
    within(got, want, tol)
    if where == "all":
        assert np.abs(got).max() <= 2.0 ** -131


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("largest,growing", [(2.0 ** 126, False), (2.0 ** 128 - 2.0 ** 120, False), (2.0 ** 128 - 2.0 ** 120, True)])
def test_values_near_the_largest(gpu, heads, kv, d, bs, new, lens, largest, growing):
    """Values up to the largest bf16 number: a mean of finite values is finite.  Uniform weights, or scores that
    grow by less than a reference may lag, to blocks of values 2^10 larger than the first ones."""
    P, table = pool(sum(lens) + 4, heads, kv, d, bs, lens, "int8", "bf16")
    P.codes[1] = np.abs(P.codes[1].view(np.int8)).view(np.uint8)
    P.scale[1] = np.float32(largest / 127)
    P.scale[0] *= np.float32(2.0 ** -20)
    q = normal(P.rng, sum(new), heads * d)
    if growing:                                            # scores of 0 in the first two blocks, then of 4 (5.8 in log2)
        q = q.abs() * 0 + 1
        P.codes[0] = 127
        P.scale[0] = 4.0 / (d ** 0.5 * 127.0)
        for i in range(len(lens)):
            P.scale[0, table[i, :2]] = 0.0
            P.scale[1, table[i, :2]] *= np.float32(2.0 ** -10)
    _, got, want, tol = both(P, q, new, lens, table)
    within(got, want, tol)
    # 2^126 / 8 at least; where a request has no third block, all values are 2^10 smaller
    assert np.abs(got).max() > (2.0 ** 115 if growing else 2.0 ** 123)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -70, 2.0 ** 70])
def test_append_keeps_the_sign_of_zero(gpu, fmt, size):
    """-0 is the code of -0 (E4M3: 0x80), whatever the block's scale."""
    import torch
    bs, d = 16, 64
    x = np.linspace(-1, 1, 2 * bs * d).reshape(2 * bs, 1, d) * size
    x[:, :, ::3], x[:, :, 1::3] = -0.0, 0.0
    x = torch.from_numpy(x).to(torch.bfloat16)
    P = Pool(1, 1, 1, d, bs, 3, fmt, "bf16")
    slots = np.arange(2 * bs, dtype=np.int32)
    want = pk.append(x.double().numpy(), slots, [0, 2 * bs], P.codes[0], P.scale[0], fmt)
    assert fmt == "int8" or (want[0][:2, :, :, ::3] == 0x80).all()
    c = P.to_device()
    b = sv.paged_batch(dev(np.array([[0, 1]], np.int32)), dev(np.array([32], np.int32)), dev(np.array([0, 32], np.int32)), dev(slots),
                       max_new=32, max_len=32)
    sv.paged_append(c, b, x.cuda(), x.cuda())
    assert np.array_equal(P.t[0].cpu().numpy(), want[0]) and np.array_equal(P.t[1].cpu().numpy(), want[1])


# ------------------------------------------------------ rows that see nothing
@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", [
    (64, 8, 128, 16, [1500] * 6, [20, 0, 1, 140, 7, 3]), (24, 8, 64, 64, [700] * 12, [0, 0, 50, 0, 0, 300, 0, 0, 0, 0, 0, 1]),
    (160, 8, 128, 128, [300, 17, 250] * 6, [20, 3, 11] * 6), (8, 8, 64, 16, [5000, 1, 5000], [0, 9, 0])])
@pytest.mark.parametrize("causal", [True, False])
def test_many_rows_that_see_nothing(gpu, heads, kv, d, bs, new, lens, causal):
    """Hundreds of 256-row items without a token in between others: zeros, and nobody waits."""
    P, table = pool(sum(lens) + 9, heads, kv, d, bs, lens, "int8", "bf16")
    _, got, want, tol = both(P, normal(P.rng, sum(new), heads * d), new, lens, table, causal)
    within(got, want, tol)
    assert sv.get_status() == sv.OK
    if causal or 0 in lens:                                # otherwise every row sees something
        assert (want == 0).all(axis=2).any()


# ------------------------------------------------------- NaN and infinities
@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt,dtype", BOTH_FORMATS)
@pytest.mark.parametrize("bad,where", [(float("nan"), 0), (float("nan"), 1), (float("-inf"), 0), (float("inf"), 1)])
def test_non_finite_values_are_seen(gpu, heads, kv, d, bs, new, lens, fmt, dtype, bad, where):
    """One NaN or infinity in a token's keys or values: recorded, and not finite for the rows that see its block in its
    head.  All other rows have the bits that they have with a finite value there."""
    import torch
    P, table = pool(sum(lens) + 6, heads, kv, d, bs, lens, fmt, dtype)
    n, G, L = sum(new), heads // kv, lens[0]
    q = normal(P.rng, n, heads * d, dtype).to(dtype_of(dtype)).cuda()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    blk = int(table[0, (L - 1) // bs])
    slot = dev(np.array([blk * bs + (L - 1) % bs], np.int32))
    one = sv.paged_batch(dev(table[:1]), dev(np.array([L], np.int32)), dev(np.array([0, 1], np.int32)), slot, max_new=1, max_len=L)
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(cu), None, n_tokens=n, max_new=max(new), max_len=max(lens))
    kv_new = normal(P.rng, 2, kv * d, dtype).to(dtype_of(dtype))
    out = []
    for value in (1.0, bad):
        c = P.to_device()
        kv_new[where, 5] = value                           # in head 0
        x = kv_new.cuda()
        sv.paged_append(c, one, x[:1], x[1:])
        assert sv.get_status() == (sv.OK if value == 1.0 else sv.ERR_INVALID_ARG)
        if value != 1.0:
            assert torch.isinf(P.t[2 * where + 1][blk, 0]) and torch.isfinite(P.t[2 * where + 1][blk, 1:]).all()
        ws = torch.empty(sv.paged_attention_workspace_bytes(c, b), dtype=torch.uint8, device="cuda")
        o = torch.zeros(n, heads * d, dtype=dtype_of(dtype), device="cuda")
        sv.paged_attention(c, b, q, o, ws)
        out.append(o.cpu().view(n, heads, d))
    sees = torch.zeros(n, heads, dtype=torch.bool)
    for j in range(new[0]):
        sees[j, :G] = L - new[0] + j + 1 > (L - 1) // bs * bs
    assert torch.isfinite(out[0].float()).all() and not torch.isfinite(out[1][sees].float()).any()
    assert torch.equal(out[0][~sees], out[1][~sees]) and sees.any() and (~sees).any()
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("fmt,dtype", BOTH_FORMATS)
def test_a_nan_in_a_query_stays_in_its_row(gpu, heads, kv, d, bs, new, lens, fmt, dtype):
    import torch
    P, table = pool(sum(lens) + 7, heads, kv, d, bs, lens, fmt, dtype)
    n = sum(new)
    q = normal(P.rng, n, heads * d, dtype)
    base, got, want, tol = both(P, q, new, lens, table, dtype=dtype)
    within(got, want, tol)
    q[n // 2, (heads - 1) * d + 3] = float("nan")
    bits = both(P, q, new, lens, table, dtype=dtype)[0].view(n, heads, d)
    assert torch.isnan(bits[n // 2, heads - 1].float()).all()
    bits[n // 2, heads - 1] = base.view(n, heads, d)[n // 2, heads - 1]
    assert torch.equal(bits, base.view(n, heads, d))


# --------------------------------------------------------------- bad pages
@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", PATHS)
@pytest.mark.parametrize("number", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_every_bad_block_number_is_recorded(gpu, heads, kv, d, bs, new, lens, number):
    """One bad number, in an even or an odd place of the table: left out and recorded."""
    for place in (0, 1):
        P, table = pool(sum(lens) + 5, heads, kv, d, bs, lens, "int8", "bf16")
        table[-1, place] = number
        _, got, want, tol = both(P, normal(P.rng, sum(new), heads * d), new, lens, table)
        within(got, want, tol)
        assert sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK
    P, table = pool(sum(lens) + 5, heads, kv, d, bs, lens, "int8", "bf16")
    for i, L in enumerate(lens):
        table[i, -(-L // bs):] = number                    # past the request's blocks: not read
    both(P, normal(P.rng, sum(new), heads * d), new, lens, table)
    assert sv.get_status() == sv.OK


# ------------------------------------------------------------ skipped tokens
def appended(x, slots, cu, codes, scale, fmt):
    """The rule for slot maps with tokens left out (-1): the block's new tokens, whatever lies between them, share one scale."""
    codes, scale = codes.copy(), scale.copy()
    bs = codes.shape[2]
    for a, e in zip(cu[:-1], cu[1:]):
        own = {}
        for t in range(a, e):
            if slots[t] >= 0:
                own.setdefault(int(slots[t]) // bs, {})[int(slots[t]) % bs] = t
        for blk, rows in own.items():
            lo, hi = min(rows), max(rows) + 1
            part = np.zeros((hi - lo, *x.shape[1:]))
            for r, t in rows.items():
                part[r - lo] = x[t]
            kept = codes[blk].copy()
            codes, scale = pk.append(part, np.arange(blk * bs + lo, blk * bs + hi), [0, hi - lo], codes, scale, fmt)
            for r in set(range(lo, hi)) - set(rows):
                codes[blk, :, r] = kept[:, r]
    return codes, scale


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (64, 128), (128, 64)])
@pytest.mark.parametrize("skip", ["leading", "block starts", "first blocks", "scattered", "all but the last", "all"])
def test_append_leaves_skipped_tokens_out(gpu, fmt, d, bs, skip):
    """Slots of -1 anywhere in a request (a prefix that is cached already, tokens of no interest): those tokens and no
    others are left out."""
    r, kv = random.Random(bs + d), 2
    olds, news = [0, 5, bs - 1, 2 * bs + 3], [3 * bs + 2, 2 * bs, bs + 4, 1]
    lens = [a + b for a, b in zip(olds, news)]
    P = Pool(bs + d, kv, kv, d, bs, sum(-(-L // bs) for L in lens) + 3, fmt, "bf16")
    table = make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens))
    slots, cu = [], [0]
    for i, (o, L) in enumerate(zip(olds, lens)):
        for t in range(o, L):
            out = {"leading": t < o + 3 and L > o + 1, "block starts": t % bs == 0, "first blocks": t < o + bs + 2, "scattered": r.random() < 0.4,
                   "all but the last": t < L - 1, "all": True}[skip]
            slots.append(-1 if out else int(table[i, t // bs]) * bs + t % bs)
        cu.append(len(slots))
    slots = np.array(slots, np.int32)
    x = (normal(P.rng, len(slots), 2 * kv * d) * 3).to(dtype_of("bf16"))
    x64 = x.double().numpy()
    want = [appended(x64[:, k * kv * d:(k + 1) * kv * d].reshape(-1, kv, d), slots, cu, P.codes[k], P.scale[k], fmt) for k in (0, 1)]
    c, xd = P.to_device(), x.cuda()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)), dev(slots), max_new=max(news), max_len=max(lens))
    sv.paged_append(c, b, xd[:, :kv * d], xd[:, kv * d:])
    for k in (0, 1):
        assert np.array_equal(P.t[2 * k + 1].cpu().numpy(), want[k][1])
        assert np.array_equal(P.t[2 * k].cpu().numpy(), want[k][0])
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("bs,d", [(16, 64), (128, 64), (128, 128)])
def test_append_behind_a_long_skipped_prefix(gpu, bs, d):
    """30000 tokens of which the first 29001 are cached already, and a request behind them."""
    olds, news, skip = [7, 3], [30000, 50], 29001
    lens = [a + b for a, b in zip(olds, news)]
    P = Pool(bs, 1, 1, d, bs, sum(-(-L // bs) for L in lens) + 3, "int8", "bf16")
    table = make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens))
    slots = [int(table[i, t // bs]) * bs + t % bs for i in (0, 1) for t in range(olds[i], lens[i])]
    slots[:skip] = [-1] * skip
    slots, cu = np.array(slots, np.int32), [0, news[0], sum(news)]
    x = normal(P.rng, len(slots), d).to(dtype_of("bf16"))
    want = appended(x.double().numpy().reshape(-1, 1, d), slots, cu, P.codes[0], P.scale[0], "int8")
    c, xd = P.to_device(), x.cuda()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)), dev(slots), max_new=max(news), max_len=max(lens))
    sv.paged_append(c, b, xd, xd)
    assert np.array_equal(P.t[1].cpu().numpy(), want[1]) and np.array_equal(P.t[0].cpu().numpy(), want[0])
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("slots", [[0, 1, 3, 2], [3, 3, 5, 6], [0, 1, 34, 3], [5, 6, 7, 20], [-1, 4, 9, 6]])
def test_append_records_tokens_astray(gpu, slots):
    """Slots of one request that do not follow one another in their block, the same slot twice, another block's slot:
    left out, recorded, and the tokens in place are written."""
    P = Pool(9, 2, 2, 64, 16, 4, "int8", "bf16")
    x = (normal(P.rng, 4, 128) * 30).to(dtype_of("bf16"))
    lead = next(k for k, v in enumerate(slots) if v >= 0)
    place = np.array([v if v == slots[lead] + k - lead else -1 for k, v in enumerate(slots)], np.int32)
    want = appended(x.double().numpy().reshape(4, 2, 64), place, [0, 4], P.codes[0], P.scale[0], "int8")
    c, xd = P.to_device(), x.cuda()
    b = sv.paged_batch(dev(np.zeros((1, 4), np.int32)), dev(np.zeros(1, np.int32)), dev(np.array([0, 4], np.int32)), dev(np.array(slots, np.int32)),
                       max_new=4, max_len=64)
    sv.paged_append(c, b, xd, xd)
    assert np.array_equal(P.t[1].cpu().numpy(), want[1]) and np.array_equal(P.t[0].cpu().numpy(), want[0])
    assert sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK


# -------------------------------------------------------------- bad pointers
def test_unaligned_int32_arrays_refused():
    """Addresses between two int32 words never reach a launch."""
    A, c = sv.ERR_ALIGNMENT, raw_cache()
    for name in ("table", "lens", "cu", "slots"):
        for off in (1, 2, 3):
            b = raw_batch(**{"lens": 12288, name: 20480 + off})
            assert call_plan(b) == A, name
            if name in ("cu", "slots"):
                assert call_append(c, b) == A, name
            if name != "slots":
                assert call_attend(c, b) == A, name
    for name in ("prev", "target", "ring", "sin", "sout"):
        assert call_plan(raw_batch(lens=12288), **{name: 20482}) == A, name


def test_scales_of_another_type_refused():
    """Scales are fp32; a buffer of another type with as many bytes would be read as something else."""
    import torch
    codes = torch.zeros(4 * 2 * 16 * 64, dtype=torch.uint8)
    ok = torch.zeros(8, dtype=torch.float32)
    for dtype, n in ((torch.float64, 8), (torch.float16, 16), (torch.bfloat16, 16), (torch.int32, 8), (torch.float32, 7)):
        bad = torch.zeros(n, dtype=dtype)
        for args in ((codes, bad, codes, ok), (codes, ok, codes, bad)):
            with pytest.raises(sv.SVDQError):
                sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", *args)
    sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", codes, ok, codes, ok)


def test_one_row_of_any_stride_is_taken():
    """The stride of a single row says nothing: a view of a wider, oddly sized row keeps its row."""
    import torch
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)  # noqa: E731
    codes, scale = z(4 * 2 * 16 * 64, t=torch.uint8), z(8, t=torch.float32)
    c = sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", codes, scale, codes, scale)
    for wide in (128, 131, 4099):
        x = z(3, wide, t=torch.bfloat16)
        for row in (x[:1, :128], x[:1, :128].unflatten(1, (2, 64)), torch.as_strided(x, (1, 128), (1, 1))):
            assert sv._rows16(row, 1, 128, c, "K") == (x.data_ptr(), 128)
    assert sv._rows16(z(3, 136, t=torch.bfloat16)[:, :128], 3, 128, c, "K")[1] == 136


# ---------------------------------------------------------- many requests
@pytest.mark.gpu
def test_plan_of_16384_requests(gpu):
    """The largest batch: 32 rounds of the scan, and all of the shared memory that it may take."""
    import torch
    B, bs, mb, cap = 16384, 16, 3, 40000
    r = random.Random(8)
    n_blocks = B * mb
    table, ring, head, count = np.zeros((B, mb), np.int32), np.arange(n_blocks, dtype=np.int32), 0, n_blocks
    lens = [0] * B
    t = dict(table=dev(table), ring=dev(ring), lens=torch.zeros(B, dtype=torch.int32).cuda(), cu=torch.zeros(B + 1, dtype=torch.int32).cuda(),
             slots=torch.zeros(cap, dtype=torch.int32).cuda())
    b = sv.paged_batch(t["table"], t["lens"], t["cu"], t["slots"], max_new=30, max_len=mb * bs)
    for step in range(3):
        target = [0 if r.random() < 0.1 else min(mb * bs, n + (r.randint(1, 30) if r.random() < 0.1 else 1)) for n in lens]
        want = pk.plan(lens, target, table, ring, head, count, bs, cap, 30, mb * bs)
        assert want["state"][2] == 0
        sout = torch.zeros(4, dtype=torch.int32).cuda()
        sv.paged_plan(b, bs, dev(np.array(lens, np.int32)), dev(np.array(target, np.int32)), t["ring"],
                      dev(np.array([head, count, 0, 0], np.int32)), sout)
        for name in t:
            assert np.array_equal(t[name].cpu().numpy(), want[name]), (step, name)
        assert np.array_equal(sout.cpu().numpy(), want["state"])
        table, ring, lens = want["table"], want["ring"], want["lens"].tolist()
        head, count = int(want["state"][0]), int(want["state"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("most", [1, 40])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 128)])
def test_append_of_many_requests(gpu, most, d, bs):
    """More requests than a pass of the search for a work item's request takes, some without a new token."""
    r, B, kv = random.Random(most), 700, 1
    news = [0 if r.random() < 0.2 else r.randint(1, most) for _ in range(B)]
    olds = [r.randint(0, 2 * bs) for _ in range(B)]
    lens = [a + b for a, b in zip(olds, news)]
    P = Pool(most + d, kv, kv, d, bs, sum(-(-L // bs) for L in lens) + 1, "int8", "bf16")
    table = make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens))
    slots, cu = [], [0]
    for i, (o, L) in enumerate(zip(olds, lens)):
        slots += [int(table[i, t // bs]) * bs + t % bs for t in range(o, L)]
        cu.append(len(slots))
    x = normal(P.rng, len(slots), 2 * kv * d).to(dtype_of("bf16"))
    want = [pk.append(x[:, k * d:(k + 1) * d].double().numpy().reshape(-1, 1, d), slots, cu, P.codes[k], P.scale[k], "int8") for k in (0, 1)]
    c, xd = P.to_device(), x.cuda()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)), dev(np.array(slots, np.int32)), max_new=most,
                       max_len=max(lens))
    sv.paged_append(c, b, xd[:, :d], xd[:, d:])
    for k in (0, 1):
        assert np.array_equal(P.t[2 * k + 1].cpu().numpy(), want[k][1]) and np.array_equal(P.t[2 * k].cpu().numpy(), want[k][0])
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,most", [(1, 1, 30), (2, 1, 1), (8, 2, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_many_requests(gpu, heads, kv, most, causal):
    """More requests than a pass of the schedule's scan takes (128 or 512 threads), some without a query."""
    r, B = random.Random(most), 1300
    new = [0 if r.random() < 0.2 else r.randint(1, most) for _ in range(B)]
    new[0] = most
    lens = [r.randint(1, 90) + m for m in new]
    P, table = pool(most, heads, kv, 64, 16, lens, "int8", "bf16")
    _, got, want, tol = both(P, normal(P.rng, sum(new), heads * 64), new, lens, table, causal)
    within(got, want, tol)
    assert sv.get_status() == sv.OK


# ------------------------------------------------------------- recorded failures
@pytest.mark.gpu
def test_two_recorded_failures_are_both_read(gpu):
    """A wait that ran out in the layer's kernels and a bad block number in the paged cache's: one after the other."""
    P, table = pool(3, 2, 2, 64, 16, [40], "int8", "bf16")
    table[0, 1] = -1
    assert sv.get_status() == sv.OK
    sv.probe_timeout(1_000_000)
    both(P, normal(P.rng, 1, 128), [1], [40], table)
    assert sv.get_status() == sv.ERR_TIMEOUT and sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK


# ------------------------------------------------------------- the schedule's size
def test_the_schedule_has_as_many_parts_as_are_resident():
    """9 to 16 rows of 64 values: three CTAs of the balanced schedule fit an SM (168 registers a thread of 128), not four."""
    import ctypes
    for d, G, per_sm in ((64, 8, 4), (64, 16, 3), (128, 8, 3), (128, 16, 2)):
        c = sv.svdq_paged_cache(4096, 4096, 4096, 4096, 4 * G, 4, d, 64, 1 << 16, 1, sv.BF16, 0)
        b = sv.svdq_paged_batch(4096, 4096, 4096, None, 100, 600, 100, 1, 30000, 0)
        got = sv.lib().svdq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b))
        assert got == 148 * per_sm * 2 * (32 + G * (d + 2) * 4), (d, G)
