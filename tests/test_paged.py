"""Paged 8-bit KV cache: the oracle's rules (CPU), the C ABI's refusals (CPU) and the kernels against the oracle
(GPU: plans and codes exactly, attention within the oracle's derived bound)."""
import ctypes
import math
import random

import numpy as np
import pytest

import rank_gemm_svdq_b200 as sv
from oracle import pagedkv as pk

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


# ------------------------------------------------------------------ the oracle
def test_e4m3_codes_are_the_nearest_values():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=4000) * np.exp(rng.normal(size=4000) * 3), pk.E4M3[np.isfinite(pk.E4M3)], [0.0, -0.0, 1e-9, 500.0, -449.0]])
    got = pk.E4M3[pk.to_codes(x, "e4m3")]
    grid = np.unique(pk.E4M3[np.isfinite(pk.E4M3)])
    best = np.abs(np.clip(x, -448, 448)[:, None] - grid[None, :]).min(axis=1)
    assert np.array_equal(np.abs(got - np.clip(x, -448, 448)), best)


def test_append_worked_by_hand():
    # one head, two values a token, blocks of 4: 127 -> scale 1; then 254 doubles the scale and halves the old codes
    codes, scale = np.zeros((2, 1, 4, 2), np.uint8), np.zeros((2, 1), np.float32)
    c, s = pk.append(np.array([[[127.0, -3.0]], [[5.0, 1.0]]]), [4, 5], [0, 2], codes, scale, "int8")
    assert s[1, 0] == 1.0 and c[1, 0, :2].view(np.int8).tolist() == [[127, -3], [5, 1]] and not c[0].any()
    c, s = pk.append(np.array([[[254.0, 10.0]]]), [6], [0, 1], c, s, "int8")
    # 127 / 2 = 63.5 -> 64 (even), -3 / 2 = -1.5 -> -2, 5 / 2 = 2.5 -> 2, 1 / 2 = 0.5 -> 0
    assert s[1, 0] == 2.0 and c[1, 0, :3].view(np.int8).tolist() == [[64, -2], [2, 0], [127, 5]]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_is_off_by_half_a_step(fmt):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(32, 3, 16)).astype(np.float32)
    c, s = pk.append(x, np.arange(32), [0, 32], np.zeros((2, 3, 16, 16), np.uint8), np.zeros((2, 3), np.float32), fmt)
    y = pk.gather(c, s, [0, 1], 32, fmt).transpose(1, 0, 2)
    step = np.repeat(s, 16, axis=0)[:, :, None]
    off = 0.5 * step if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)
    assert np.all(np.abs(y - x) <= off * (1 + 1e-6))


def random_walk(seed, steps, B, bs, n_blocks, max_blocks, max_new):
    """Steps of a server: (prev, target) pairs from empty requests."""
    r = random.Random(seed)
    lens = [0] * B
    for _ in range(steps):
        target = []
        for n in lens:
            u = r.random()
            if n == 0:
                t = r.randint(0, min(max_new, max_blocks * bs)) if u < 0.6 else 0
            elif u < 0.15:
                t = 0
            elif u < 0.25:
                t = r.randint(0, n)
            elif u < 0.4:
                t = n
            else:
                t = min(max_blocks * bs, n + r.randint(1, max_new if u > 0.9 else 1))
            target.append(t)
        yield lens, target
        lens = target


@pytest.mark.parametrize("seed,bs", [(1, 16), (2, 32), (3, 128)])
def test_plan_keeps_every_block_once(seed, bs):
    B, max_blocks, n_blocks = 7, 6, 14
    table, ring, head, count = np.full((B, max_blocks), -1, np.int32), np.arange(n_blocks, dtype=np.int32), 0, n_blocks
    lens = [0] * B
    refused = 0
    for _, target in random_walk(seed, 200, B, bs, n_blocks, max_blocks, 3 * bs):
        target = list(target)
        r = pk.plan(lens, target, table, ring, head, count, bs, B * 3 * bs, 10 ** 6, max_blocks * bs)
        refused += r["state"][2] != 0
        table, ring, lens = r["table"], r["ring"], r["lens"].tolist()
        head, count = int(r["state"][0]), int(r["state"][1])
        held = [int(table[i, c]) for i in range(B) for c in range(-(-lens[i] // bs))]
        free = [int(ring[(head + k) % n_blocks]) for k in range(count)]
        assert sorted(held + free) == list(range(n_blocks))
        live = r["slots"][r["slots"] >= 0]
        assert len(set(live.tolist())) == len(live) == r["state"][3]
    assert refused > 0


def test_attend_is_softmax():
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 256, size=(3, 2, 16, 64)).astype(np.uint8)
    scale = rng.uniform(0.01, 0.02, size=(3, 2)).astype(np.float32)
    q = rng.normal(size=(2, 4, 64))
    out, _ = pk.attend(q, [0, 2], [20], np.array([[2, 0]]), codes, scale, codes[::-1].copy(), scale, "int8", True, 0.125)
    K, V = pk.gather(codes, scale, [2, 0], 20, "int8"), pk.gather(codes[::-1].copy(), scale, [2, 0], 20, "int8")
    for h in range(4):
        w = [math.exp(0.125 * float(q[0, h] @ K[h // 2, t])) for t in range(19)]        # token 0 sees 19
        want = sum(wt * V[h // 2, t] for t, wt in enumerate(w)) / sum(w)
        assert np.allclose(out[0, h], want, rtol=1e-12)


# --------------------------------------------------------------- refusals (CPU)
def raw_cache(**kw):
    c = dict(heads=4, kv_heads=2, head_dim=64, block_size=16, n_blocks=8, fmt=1, dtype=sv.BF16, reserved=0,
             kcodes=4096, kscale=4096, vcodes=4096, vscale=4096)
    c.update(kw)
    return sv.svdq_paged_cache(**c)


def raw_batch(**kw):
    b = dict(table=4096, lens=4096, cu=4096, slots=4096, B=2, max_blocks=4, n_tokens=4, max_new=2, max_len=64, reserved=0)
    b.update(kw)
    return sv.svdq_paged_batch(**b)


BAD_CACHE = [(dict(heads=0), sv.ERR_INVALID_ARG), (dict(kv_heads=3), sv.ERR_INVALID_ARG), (dict(kv_heads=0), sv.ERR_INVALID_ARG),
             (dict(head_dim=80), sv.ERR_UNSUPPORTED), (dict(head_dim=256), sv.ERR_UNSUPPORTED), (dict(block_size=24), sv.ERR_UNSUPPORTED),
             (dict(block_size=256), sv.ERR_UNSUPPORTED), (dict(n_blocks=0), sv.ERR_INVALID_ARG), (dict(n_blocks=1 << 28), sv.ERR_UNSUPPORTED),
             (dict(fmt=0), sv.ERR_INVALID_ARG), (dict(fmt=3), sv.ERR_INVALID_ARG), (dict(dtype=3), sv.ERR_INVALID_ARG),
             (dict(reserved=1), sv.ERR_INVALID_ARG), (dict(kcodes=None), sv.ERR_INVALID_ARG), (dict(vscale=None), sv.ERR_INVALID_ARG),
             (dict(vcodes=4097), sv.ERR_ALIGNMENT), (dict(kscale=4100), sv.ERR_ALIGNMENT)]
BAD_BATCH = [(dict(B=0), sv.ERR_INVALID_ARG), (dict(B=16385), sv.ERR_INVALID_ARG), (dict(max_blocks=0), sv.ERR_INVALID_ARG),
             (dict(n_tokens=-1), sv.ERR_INVALID_ARG), (dict(max_new=0), sv.ERR_INVALID_ARG), (dict(max_len=65), sv.ERR_INVALID_ARG),
             (dict(max_len=-1), sv.ERR_INVALID_ARG), (dict(reserved=2), sv.ERR_INVALID_ARG), (dict(cu=None), sv.ERR_INVALID_ARG),
             (dict(max_blocks=1 << 30), sv.ERR_UNSUPPORTED)]


def call_plan(b, **kw):
    a = dict(bs=16, n=8, prev=4096, target=8192, ring=4096, sin=4096, sout=8192)
    a.update(kw)
    return sv.lib().svdq_paged_plan(ctypes.byref(b), a["bs"], a["n"], a["prev"], a["target"], a["ring"], a["sin"], a["sout"], None)


def call_append(c, b, K=4096, ks=128, V=4096, vs=128):
    return sv.lib().svdq_paged_append(ctypes.byref(c), ctypes.byref(b), K, ks, V, vs, None)


def call_attend(c, b, Q=4096, qs=256, causal=1, scale=0.1, out=4096, os=256, ws=4096, n=1 << 40):
    return sv.lib().svdq_paged_attention(ctypes.byref(c), ctypes.byref(b), Q, qs, causal, scale, out, os, ws, n, None)


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_bad_cache_refused(bad, status):
    c, b = raw_cache(**bad), raw_batch()
    assert call_append(c, b) == status and call_attend(c, b) == status
    assert sv.lib().svdq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b)) == 0


@pytest.mark.parametrize("bad,status", BAD_BATCH)
def test_bad_batch_refused(bad, status):
    c, b = raw_cache(), raw_batch(**bad)
    assert call_append(c, b) == status and call_attend(c, b) == status and call_plan(b) == status
    if "cu" not in bad:
        assert sv.lib().svdq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b)) == 0


def test_bad_arguments_refused():
    c, b = raw_cache(), raw_batch()
    E = sv.ERR_INVALID_ARG
    assert call_append(c, b, K=None) == E and call_append(c, b, vs=127) == E and call_append(c, raw_batch(slots=None)) == E
    assert call_append(c, b, K=4104) == sv.ERR_ALIGNMENT and call_append(c, b, ks=132) == sv.ERR_ALIGNMENT
    assert call_attend(c, b, Q=None) == E and call_attend(c, b, out=None) == E and call_attend(c, b, ws=None) == E
    assert call_attend(c, b, causal=2) == E and call_attend(c, b, scale=math.inf) == E and call_attend(c, b, scale=math.nan) == E
    assert call_attend(c, b, qs=255) == E and call_attend(c, b, os=255) == E
    assert call_attend(c, b, out=4104) == sv.ERR_ALIGNMENT and call_attend(c, b, qs=260) == sv.ERR_ALIGNMENT
    assert call_attend(c, b, n=0) == sv.ERR_WORKSPACE
    for kw in (dict(prev=None), dict(target=None), dict(ring=None), dict(sin=None), dict(n=0), dict(sout=4096),
               dict(sin=8192), ):
        bb = raw_batch(lens=12288)
        assert call_plan(bb, **kw) == E, kw
    assert call_plan(raw_batch(lens=4096)) == E and call_plan(raw_batch(lens=8192)) == E
    assert call_plan(raw_batch(lens=12288), bs=8) == sv.ERR_UNSUPPORTED
    # nothing to do: no device is needed
    none = raw_batch(n_tokens=0)
    assert call_append(c, none) == sv.OK and call_attend(c, none) == sv.OK


def test_binding_checks_tensors():
    import torch
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t)  # noqa: E731
    codes, scale = z(4 * 2 * 16 * 64, torch.uint8), z(8, torch.float32)
    with pytest.raises(sv.SVDQError):
        sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", codes[:-1], scale, codes, scale)
    c = sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", codes, scale, codes, scale)
    with pytest.raises(sv.SVDQError):
        sv.paged_batch(z((2, 2)), z(1), z(3), z(4), max_new=1, max_len=32)
    with pytest.raises(sv.SVDQError):
        sv.paged_batch(z((2, 2)), z(2, torch.int64), z(3), z(4), max_new=1, max_len=32)
    b = sv.paged_batch(z((2, 2)), z(2), z(3), z(4), max_new=2, max_len=32)
    K = z((4, 128), torch.bfloat16)
    for bad in (K[:3], K.half(), z((4, 120), torch.bfloat16), z((4, 256), torch.bfloat16)[:, ::2], z((4, 2, 128), torch.bfloat16)[:, :, :64]):
        with pytest.raises(sv.SVDQError):
            sv.paged_append(c, b, bad, K)
        with pytest.raises(sv.SVDQError):
            sv.paged_append(c, b, K, bad)


# ------------------------------------------------------------------------- GPU
def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


class Pool:
    """A cache with random content, on the host and on the device."""

    def __init__(self, seed, heads, kv, d, bs, n_blocks, fmt, dtype, spare=0xFF):
        rng = np.random.default_rng(seed)
        self.rng, self.heads, self.kv, self.d, self.bs, self.n, self.fmt, self.dtype = rng, heads, kv, d, bs, n_blocks, fmt, dtype
        x = rng.normal(size=(2, n_blocks, kv, bs, d)) * np.exp(rng.normal(size=(2, n_blocks, kv, 1, 1)))
        self.scale = (np.abs(x).max(axis=(3, 4)) / float(pk.QMAX[fmt])).astype(np.float32)
        self.codes = pk.to_codes(x / self.scale[..., None, None], fmt)

    def to_device(self):
        self.t = [dev(self.codes[0]), dev(self.scale[0]), dev(self.codes[1]), dev(self.scale[1])]
        self.c = sv.paged_cache(self.heads, self.kv, self.d, self.bs, self.n, self.fmt, self.dtype, *self.t)
        return self.c


def sixteen_bit(rng, shape, dtype, spread=1.0):
    """Random 16-bit values: a device tensor and the same numbers in float64."""
    import torch
    x = torch.from_numpy((rng.normal(size=shape) * spread).astype(np.float32)).to(dtype_of(dtype))
    return x.cuda(), x.double().numpy()


def make_table(rng, lens, bs, n_blocks, max_blocks, fill=0):
    ids = rng.permutation(n_blocks)
    table, at = np.full((len(lens), max_blocks), fill, np.int32), 0
    for i, L in enumerate(lens):
        nb = -(-int(L) // bs)
        table[i, :nb] = ids[at:at + nb]
        at += nb
    assert at <= n_blocks
    return table


@pytest.mark.gpu
@pytest.mark.parametrize("seed,B,bs,max_blocks,n_blocks,max_new", [
    (1, 1, 16, 4, 5, 40), (2, 7, 16, 6, 30, 50), (3, 33, 64, 5, 100, 100), (4, 600, 32, 4, 1500, 60), (5, 1500, 128, 3, 2600, 200)])
def test_plan_matches_oracle(gpu, seed, B, bs, max_blocks, n_blocks, max_new):
    import torch
    cap = min(B * max_new, 40000) + 5
    table, ring = np.full((B, max_blocks), -1, np.int32), np.arange(n_blocks, dtype=np.int32)
    head, count, lens = 0, n_blocks, [0] * B
    t = dict(table=dev(table), ring=dev(ring), lens=torch.zeros(B, dtype=torch.int32).cuda(),
             cu=torch.full((B + 1,), 7, dtype=torch.int32).cuda(), slots=torch.full((cap,), 9, dtype=torch.int32).cuda())
    sin, sout = dev(np.array([0, n_blocks, 5, 5], np.int32)), torch.zeros(4, dtype=torch.int32).cuda()
    b = sv.paged_batch(t["table"], t["lens"], t["cu"], t["slots"], max_new=max_new, max_len=max_blocks * bs - 1)
    seen = set()
    for k, (_, target) in enumerate(random_walk(seed, 25, B, bs, n_blocks, max_blocks, max_new)):
        want = pk.plan(lens, target, table, ring, head, count, bs, cap, max_new, max_blocks * bs - 1)
        prev = dev(np.array(lens, np.int32))
        for _ in range(1 + k % 2):                      # the same call twice gives the same
            sv.paged_plan(b, bs, prev, dev(np.array(target, np.int32)), t["ring"], sin, sout)
        for name in ("table", "lens", "cu", "slots", "ring"):
            assert np.array_equal(t[name].cpu().numpy(), want[name]), (k, name)
        assert np.array_equal(sout.cpu().numpy(), want["state"])
        seen.add(int(want["state"][2]))
        table, ring, lens = want["table"], want["ring"], want["lens"].tolist()
        head, count = int(want["state"][0]), int(want["state"][1])
        sin, sout = sout, sin
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
def test_plan_refuses_bad_lengths(gpu):
    import torch
    B, bs, n_blocks, max_blocks = 5, 16, 12, 4
    for bad_prev, bad_target, state, cap in [(-1, 4, (0, 12), 100), (3, -2, (0, 12), 100), (0, 61, (0, 12), 100), (0, 2 ** 31 - 1, (0, 12), 100),
                                             (2 ** 31 - 1, 0, (0, 12), 100), (0, 21, (0, 12), 100), (3, 4, (12, 0), 100), (3, 4, (-1, 3), 100),
                                             (3, 4, (0, 13), 100), (3, 4, (0, -1), 100), (0, 20, (0, 12), 23), (0, 20, (3, 1), 100), (64, 0, (2, 10), 100)]:
        prev, target = np.array([1, 2, bad_prev, 4, 5], np.int32), np.array([2, 3, bad_target, 5, 6], np.int32)
        table, ring = np.arange(B * max_blocks, dtype=np.int32).reshape(B, -1) % n_blocks, np.arange(n_blocks, dtype=np.int32)[::-1].copy()
        want = pk.plan(prev, target, table, ring, *state, bs, cap, 20, 60)
        assert want["state"][2] != 0
        t = dict(table=dev(table), ring=dev(ring), lens=torch.zeros(B, dtype=torch.int32).cuda(), cu=torch.ones(B + 1, dtype=torch.int32).cuda(),
                 slots=torch.ones(cap, dtype=torch.int32).cuda())
        b = sv.paged_batch(t["table"], t["lens"], t["cu"], t["slots"], max_new=20, max_len=60)
        out = torch.zeros(4, dtype=torch.int32).cuda()
        sv.paged_plan(b, bs, dev(prev), dev(target), t["ring"], dev(np.array([*state, 0, 0], np.int32)), out)
        for name in t:
            assert np.array_equal(t[name].cpu().numpy(), want[name]), (bad_prev, bad_target, state, name)
        assert np.array_equal(out.cpu().numpy(), want["state"])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,bs,kv,news,olds", [
    (128, 64, 2, [1], [0]), (64, 16, 1, [1, 1, 0, 1], [15, 16, 3, 40]), (128, 16, 3, [5, 0, 70, 1], [13, 9, 0, 31]),
    (64, 32, 4, [33, 200], [31, 7]), (128, 32, 2, [64, 31, 1], [0, 1, 32]), (64, 64, 2, [130, 1, 63], [62, 63, 1]),
    (128, 128, 2, [1, 300, 127], [127, 5, 1]), (64, 128, 1, [129], [127])])
def test_append_matches_oracle(gpu, fmt, dtype, d, bs, kv, news, olds):
    import torch
    lens = [n + o for n, o in zip(news, olds)]
    n, max_blocks = sum(news), max(-(-L // bs) for L in lens) + 1
    P = Pool(n + d + bs, kv, kv, d, bs, sum(-(-L // bs) for L in lens) + 3, fmt, dtype)
    P.scale[0, ::3] *= 0.25                                # small old scales: the new tokens make them grow
    table = make_table(P.rng, lens, bs, P.n, max_blocks)
    slots, cu = [], [0]
    for i, (o, L) in enumerate(zip(olds, lens)):
        slots += [int(table[i, t // bs]) * bs + t % bs for t in range(o, L)]
        cu.append(len(slots))
    pad = 4
    slots = np.array(slots + [-1] * pad, np.int32)
    row = 2 * kv * d + 16                                  # keys and values as views of a wider row
    x = P.rng.normal(size=(n + pad, row)) * np.exp(P.rng.normal(size=(n + pad, 1)))
    x[: n // 3, : kv * d // 2] = 0.0
    if n > 3:
        x[2] = 0.0
    x = torch.from_numpy(x.astype(np.float32)).to(dtype_of(dtype))
    want = [pk.append(x[:n, c:c + kv * d].double().numpy().reshape(n, kv, d), slots, cu, P.codes[k], P.scale[k], fmt)
            for k, c in ((0, 8), (1, 8 + kv * d))]
    c, xd = P.to_device(), x.cuda()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)), dev(slots), max_new=max(news), max_len=max(lens))
    K, V = xd[:, 8:8 + kv * d], xd[:, 8 + kv * d:8 + 2 * kv * d]
    sv.paged_append(c, b, K, V.unflatten(1, (kv, d)))
    for k in range(2):
        assert np.array_equal(P.t[2 * k + 1].cpu().numpy(), want[k][1])
        assert np.array_equal(P.t[2 * k].cpu().numpy(), want[k][0])
    sv.paged_append(c, b, K, V)                            # the same tokens again: nothing grows, nothing changes
    for k in range(2):
        assert np.array_equal(P.t[2 * k].cpu().numpy(), want[k][0])
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_extreme_scales(gpu, fmt):
    """All zeros, the smallest and the largest finite inputs; every bf16 magnitude between."""
    import torch
    bs, d = 16, 64
    x = np.zeros((6 * bs, 1, d))
    x[bs:2 * bs] = 2.0 ** -133                              # subnormal in bf16
    x[2 * bs:3 * bs] = 3.3e38
    x[3 * bs:4 * bs] = np.exp2(np.linspace(-126, 127, bs * d)).reshape(bs, 1, d)
    x[4 * bs:5 * bs] = np.linspace(-1, 1, bs * d).reshape(bs, 1, d) * 2.0 ** -70
    x[5 * bs:] = np.linspace(-1, 1, bs * d).reshape(bs, 1, d) * 2.0 ** 70
    x = torch.from_numpy(x).to(torch.bfloat16)
    P = Pool(1, 1, 1, d, bs, 8, fmt, "bf16")
    slots = np.arange(bs, 7 * bs, dtype=np.int32)
    want = pk.append(x.double().numpy(), slots, [0, 6 * bs], P.codes[0], P.scale[0], fmt)
    c = P.to_device()
    b = sv.paged_batch(dev(np.arange(8, dtype=np.int32)[None]), dev(np.array([96], np.int32)), dev(np.array([0, 96], np.int32)), dev(slots),
                       max_new=96, max_len=128)
    sv.paged_append(c, b, x.cuda(), x.cuda())
    assert np.array_equal(P.t[1].cpu().numpy(), want[1])
    assert np.array_equal(P.t[0].cpu().numpy(), want[0])
    assert P.t[1][1].item() == 0.0 and not P.t[0][1].any()


@pytest.mark.gpu
def test_append_bad_slots_are_left_out(gpu):
    """Slots of -1, past the pool, out of order within a block: those tokens are left out, nothing else changes."""
    P = Pool(9, 2, 2, 64, 16, 4, "int8", "bf16")
    x, x64 = sixteen_bit(P.rng, (9, 2, 64), "bf16", 30.0)
    slots = np.array([3, 4, 9, 6, -1, 16 * 4 + 2, 2 ** 31 - 1, 17, -7], np.int32)
    cu = np.array([0, 4, 5, 6, 7, 9], np.int32)
    keep = np.array([3, 4, -1, 6, -1, -1, -1, 17, -1], np.int32)   # 9 is not next to 4; 6 sits where 3 + 3 is
    codes, scale = P.codes[0].copy(), P.scale[0].copy()
    x1 = x64.copy()
    x1[2] = 0.0                                                    # the token left out inside the first block
    wc, ws = pk.append(x1, np.array([3, 4, 5, 6, -1, -1, -1, 17, -1], np.int32), cu, codes, scale, "int8")
    wc[0, :, 5] = codes[0, :, 5] if np.array_equal(ws[0], scale[0]) else P.codes[0][0, :, 5]
    c = P.to_device()
    b = sv.paged_batch(dev(np.zeros((5, 2), np.int32)), dev(np.zeros(5, np.int32)), dev(cu), dev(slots), max_new=4, max_len=32)
    sv.paged_append(c, b, x, x)
    got, gs = P.t[0].cpu().numpy(), P.t[1].cpu().numpy()
    assert np.array_equal(gs, ws) and np.array_equal(got, wc)
    assert keep[2] == -1 and sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK


ATTEND = [
    # heads, kv, d, bs, new, lens
    (1, 1, 64, 16, [1], [1]), (1, 1, 128, 16, [1], [17]), (4, 4, 128, 64, [1, 1, 1], [63, 64, 65]),
    (8, 2, 128, 32, [1, 1, 0, 1], [300, 0, 5, 129]), (7, 1, 64, 128, [1, 1], [1000, 3]), (32, 2, 64, 64, [1], [200]),
    (6, 2, 128, 16, [5, 1, 9], [33, 700, 9]), (4, 4, 64, 32, [40, 17, 1], [40, 100, 260]), (3, 3, 128, 128, [130], [400]),
    (16, 16, 64, 16, [3, 2], [513, 31]), (8, 1, 128, 64, [50, 33], [90, 33]), (2, 1, 64, 64, [300], [300]),
    (4, 2, 128, 16, [129, 0, 257], [1030, 4, 300]), (2, 2, 128, 64, [5, 6], [3, 6])]


def run_attend(P, new, lens, causal, dtype, table=None, pad=3, scale=None, max_len=None, max_new=None):
    import torch
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n, max_blocks = int(cu[-1]), max(1, max(-(-L // P.bs) for L in lens)) + 1
    table = make_table(P.rng, lens, P.bs, P.n, max_blocks, fill=-1) if table is None else table
    wide = P.heads * P.d + 24
    q, q64 = sixteen_bit(P.rng, (n + pad, wide), dtype)
    sc = P.d ** -0.5 if scale is None else scale
    want, tol = pk.attend(q64[:n, 8:8 + P.heads * P.d].reshape(n, P.heads, P.d), cu, lens, table, P.codes[0], P.scale[0], P.codes[1],
                          P.scale[1], P.fmt, causal, sc, UNIT[dtype])
    c = P.to_device()
    b = sv.paged_batch(dev(table), dev(np.array(lens, np.int32)), dev(cu), None, n_tokens=n + pad, max_new=max_new or max(max(new), 1),
                       max_len=max(lens) if max_len is None else max_len)
    ws = torch.full((sv.paged_attention_workspace_bytes(c, b),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((n + pad, wide), 7.0, dtype=dtype_of(dtype), device="cuda")
    view = out[:, 8:8 + P.heads * P.d]
    sv.paged_attention(c, b, q[:, 8:8 + P.heads * P.d], view, ws, causal=causal, scale=scale)
    first = out.clone()
    sv.paged_attention(c, b, q[:, 8:8 + P.heads * P.d], view, ws, causal=causal, scale=scale)
    assert torch.equal(first, out), "the same call gives the same bits"
    got = out.double().cpu().numpy()
    assert np.all(got[n:] == 7.0) and np.all(got[:, :8] == 7.0) and np.all(got[:, 8 + P.heads * P.d:] == 7.0)
    err = np.abs(got[:n, 8:8 + P.heads * P.d].reshape(n, P.heads, P.d) - want)
    worst = np.max(err - tol) if err.size else 0.0
    assert worst <= 0, (worst, float(err.max()), np.unravel_index(np.argmax(err - tol), err.shape))
    return want


def spoil(P, table, lens):
    """Everything that no request holds: codes of 0xFF, scales NaN."""
    held = np.zeros((P.n, P.bs), bool)
    for i, L in enumerate(lens):
        for t in range(L):
            held[table[i, t // P.bs], t % P.bs] = True
    P.codes[:, ~held.any(1)] = 0xFF
    P.scale[:, ~held.any(1)] = np.nan
    for blk in np.nonzero(held.any(1))[0]:
        P.codes[:, blk, :, ~held[blk]] = 0xFF


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", ATTEND)
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16"), ("int8", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_oracle(gpu, heads, kv, d, bs, new, lens, fmt, dtype, causal):
    P = Pool(sum(lens) + heads, heads, kv, d, bs, sum(-(-L // bs) for L in lens) + 2, fmt, dtype)
    table = make_table(P.rng, lens, bs, P.n, max(1, max(-(-L // bs) for L in lens)) + 1, fill=-1)
    spoil(P, table, lens)
    want = run_attend(P, new, lens, causal, dtype, table)
    if causal and new[0] > lens[0] and want.size:
        assert not want[: new[0] - lens[0]].any()          # rows that see nothing are zero
    assert sv.get_status() == sv.OK


# Shapes that reach each way of sharing the work out: (heads, kv, d, bs, new, lens)
def ragged(seed, B, lo, hi, new=1, idle=0.0):
    r = random.Random(seed)
    lens = [r.randint(lo, hi) for _ in range(B)]
    return [0 if r.random() < idle else min(new, L) if new == 1 else r.randint(1, min(new, max(L, 1))) for L in lens], lens


SCHEDULE = [
    (8, 4, 128, 64, *ragged(1, 48, 1, 900)),               # more cells than SMs: shares cut inside requests
    (16, 8, 64, 16, *ragged(2, 40, 1, 700, 4)),            # 8 rows of several tokens
    (64, 4, 128, 32, *ragged(3, 40, 1, 600)),              # 16 rows
    (5, 5, 64, 128, *ragged(4, 200, 1, 250)),              # short: whole items
    (4, 4, 128, 16, *ragged(5, 130, 1, 300, 1, 0.9)),      # most requests idle
    (2, 1, 128, 128, [1], [9000]),                         # one long request over the whole chip
    (1, 1, 64, 16, [3], [7000]),
    (20, 1, 128, 64, [1], [6000]),                         # 20 rows over the whole chip
    (3, 3, 64, 32, *ragged(6, 70, 1, 400, 90, 0.5)),       # tensor-core rows, half the requests idle
    (200, 1, 128, 16, [3, 1], [333, 40]),                  # many heads on one
    (7, 1, 64, 64, [90, 1, 200], [90, 64, 1500])]


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", SCHEDULE)
@pytest.mark.parametrize("fmt,dtype,causal", [("int8", "bf16", True), ("e4m3", "fp16", True), ("e4m3", "bf16", False)])
def test_attention_schedules(gpu, heads, kv, d, bs, new, lens, fmt, dtype, causal):
    P = Pool(sum(lens) + heads, heads, kv, d, bs, sum(-(-L // bs) for L in lens) + 2, fmt, dtype)
    table = make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens) + 1, fill=-1)
    spoil(P, table, lens)
    run_attend(P, new, lens, causal, dtype, table)
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", [
    (4, 2, 128, 64, [1, 1], [300, 90]), (4, 4, 64, 16, [1] * 40, [100] * 40), (8, 2, 64, 32, [40, 70], [200, 70])])
@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0, 1e-30])
def test_attention_scales(gpu, heads, kv, d, bs, new, lens, scale):
    """Softmax scales of any sign; key and value blocks of zeros (scale 0); value scales far apart."""
    P = Pool(7, heads, kv, d, bs, sum(-(-L // bs) for L in lens) + 2, "int8", "bf16")
    P.codes[0, ::3], P.scale[0, ::3] = 0, 0
    P.codes[1, 1::4], P.scale[1, 1::4] = 0, 0
    P.scale[1, 2::5] *= np.float32(2.0 ** -40)
    P.scale[1, 3::5] *= np.float32(2.0 ** 30)
    run_attend(P, new, lens, True, "bf16", scale=scale)
    P.codes[1], P.scale[1] = 0, 0                          # nothing but zeros
    assert not run_attend(P, new, lens, True, "bf16", scale=scale).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("heads,kv,d,bs,new,lens", [
    (4, 2, 128, 64, [1, 1], [300, 90]), (4, 4, 64, 16, [1] * 40, [100] * 40), (8, 2, 64, 16, [40, 70], [200, 300]), (2, 2, 128, 128, [200], [500])])
def test_attention_leaves_bad_blocks_out(gpu, fmt, heads, kv, d, bs, new, lens):
    P = Pool(3, heads, kv, d, bs, sum(-(-L // bs) for L in lens) + 2, fmt, "bf16")
    table = make_table(P.rng, lens, bs, P.n, max(-(-L // bs) for L in lens) + 1, fill=-1)
    table[0, 1], table[-1, 0] = P.n, -1                    # past the pool, negative
    if lens[0] > 3 * bs:
        table[0, 3], table[0, 2] = 2 ** 31 - 1, -2 ** 31
    run_attend(P, new, lens, True, "bf16", table)
    assert sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,new", [(4, 2, 1), (4, 4, 30)])
def test_attention_bounds_are_recorded(gpu, heads, kv, new):
    """A length above max_len, more new tokens than max_new: cut and recorded; nothing outside is written."""
    import torch
    P = Pool(5, heads, kv, 64, 16, 12, "int8", "bf16")
    c = P.to_device()
    for lens, cu, max_new, max_len in (([60, 40], [0, new, 2 * new], new, 50), ([60, 40], [0, 2 * new + 3, 2 * new + 4], new, 64)):
        b = sv.paged_batch(dev(np.arange(8, dtype=np.int32).reshape(2, 4)), dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)),
                           n_tokens=2 * new + 4, max_new=max_new, max_len=max_len)
        q = torch.ones(2 * new + 4, heads * 64, dtype=torch.bfloat16, device="cuda")
        out = torch.full((2 * new + 6, heads * 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(16, sv.paged_attention_workspace_bytes(c, b)), dtype=torch.uint8, device="cuda")
        sv.paged_attention(c, b, q, out[1:-1], ws)
        assert sv.get_status() == sv.ERR_INVALID_ARG and sv.get_status() == sv.OK
        assert (out[0] == 7).all() and (out[-1] == 7).all() and torch.isfinite(out.float()).all()


class Server:
    """A few steps of serving on the device and in the oracle: lengths, plan, append, attention."""

    def __init__(self, seed, heads, kv, d, bs, B, max_blocks, n_blocks, max_new, fmt, dtype):
        import torch
        self.P = P = Pool(seed, heads, kv, d, bs, n_blocks, fmt, dtype)
        self.B, self.max_new, self.dtype, self.cap = B, max_new, dtype, B * max_new
        self.codes, self.scale = [P.codes[0], P.codes[1]], [P.scale[0], P.scale[1]]
        self.table, self.ring, self.state = np.zeros((B, max_blocks), np.int32), np.arange(n_blocks, dtype=np.int32), (0, n_blocks)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.c = P.to_device()
        self.lens = [i32(B), i32(B)]
        self.target, self.cu, self.slots, self.tab = i32(B), i32(B + 1), i32(self.cap), i32(B, max_blocks)
        self.rng_dev, self.st = dev(self.ring), [dev(np.array([0, n_blocks, 0, 0], np.int32)), i32(4)]
        row = (heads + 2 * kv) * d
        self.x = torch.zeros(self.cap, row, dtype=dtype_of(dtype), device="cuda")
        self.out = torch.zeros(self.cap, heads * d, dtype=dtype_of(dtype), device="cuda")
        self.batches = [sv.paged_batch(self.tab, self.lens[k ^ 1], self.cu, self.slots, max_new=max_new, max_len=max_blocks * bs) for k in (0, 1)]
        self.ws = torch.empty(max(16, sv.paged_attention_workspace_bytes(self.c, self.batches[0])), dtype=torch.uint8, device="cuda")
        self.h = [0] * B
        self.k = 0

    def launch(self, k, stream=None):
        P = self.P
        q, kv = P.heads * P.d, P.kv * P.d
        sv.paged_plan(self.batches[k], P.bs, self.lens[k], self.target, self.rng_dev, self.st[k], self.st[k ^ 1], stream=stream)
        sv.paged_append(self.c, self.batches[k], self.x[:, q:q + kv], self.x[:, q + kv:], stream=stream)
        sv.paged_attention(self.c, self.batches[k], self.x[:, :q], self.out, self.ws, stream=stream)

    def step(self, target, run):
        import torch
        P, k = self.P, self.k
        x = torch.from_numpy((P.rng.normal(size=tuple(self.x.shape)) * 2).astype(np.float32)).to(dtype_of(self.dtype))
        self.x.copy_(x)
        self.target.copy_(torch.tensor(target, dtype=torch.int32))
        self.out.fill_(5.0)
        torch.cuda.synchronize()
        run(k)
        torch.cuda.synchronize()
        r = pk.plan(self.h, target, self.table, self.ring, *self.state, P.bs, self.cap, self.max_new, self.table.shape[1] * P.bs)
        self.table, self.ring, self.h, self.state = r["table"], r["ring"], r["lens"].tolist(), (int(r["state"][0]), int(r["state"][1]))
        n, x64 = int(r["cu"][-1]), x.double().numpy()
        q, kv = P.heads * P.d, P.kv * P.d
        for j in (0, 1):
            self.codes[j], self.scale[j] = pk.append(x64[:n, q + j * kv:q + (j + 1) * kv].reshape(n, P.kv, P.d), r["slots"], r["cu"],
                                                     self.codes[j], self.scale[j], P.fmt)
            assert np.array_equal(P.t[2 * j].cpu().numpy(), self.codes[j]) and np.array_equal(P.t[2 * j + 1].cpu().numpy(), self.scale[j])
        want, tol = pk.attend(x64[:n, :q].reshape(n, P.heads, P.d), r["cu"], self.h, self.table, self.codes[0], self.scale[0], self.codes[1],
                              self.scale[1], P.fmt, True, P.d ** -0.5, UNIT[self.dtype])
        got = self.out.double().cpu().numpy()
        assert np.all(got[n:] == 5.0)
        if n:
            assert np.all(np.abs(got[:n].reshape(want.shape) - want) <= tol)
        assert np.array_equal(self.st[k ^ 1].cpu().numpy(), r["state"])
        self.k ^= 1


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,heads,kv,d,bs,B,max_blocks,n_blocks,max_new", [
    ("int8", "bf16", 4, 2, 128, 16, 5, 8, 30, 40), ("e4m3", "fp16", 6, 3, 64, 32, 60, 4, 180, 1), ("e4m3", "bf16", 4, 4, 64, 64, 3, 20, 40, 500),
    ("int8", "fp16", 8, 1, 128, 128, 2, 20, 30, 2)])
@pytest.mark.parametrize("way", ["eager", "stream", "graph"])
def test_serving_steps(gpu, fmt, dtype, heads, kv, d, bs, B, max_blocks, n_blocks, max_new, way):
    """Plan, append and attention as a server runs them, call after call: eagerly, on another stream, and captured
    once and replayed with other lengths (two graphs that share the workspace, one for each of the swapped lengths)."""
    import torch
    S = Server(B + max_new, heads, kv, d, bs, B, max_blocks, n_blocks, max_new, fmt, dtype)
    run = S.launch
    if way == "stream":
        side = torch.cuda.Stream()
        run = lambda k: S.launch(k, stream=side)  # noqa: E731
    if way == "graph":
        graphs = []
        for k in (0, 1):                                   # captured with no work in it: the target is all zeros
            S.launch(k)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                S.launch(k)
            graphs.append(g)
        run = lambda k: graphs[k].replay()  # noqa: E731
    r = random.Random(B)
    for i in range(6):
        target = []
        for n in S.h:
            u = r.random()
            t = 0 if u < 0.15 else n if u < 0.25 else n + r.randint(1, max_new)
            target.append(min(t, max_blocks * bs))
        S.step(target, run)
    assert sv.get_status() == sv.OK


@pytest.mark.gpu
def test_two_calls_at_once(gpu):
    """Two streams, each with its own workspace, over one cache."""
    import torch
    for heads, kv, new, lens in ((2, 1, [1], [9000]), (8, 4, [1] * 48, [500] * 48), (4, 2, [120, 300], [500, 2000])):
        P = Pool(11, heads, kv, 128, 64, sum(-(-L // 64) for L in lens) + 1, "int8", "bf16")
        c, n = P.to_device(), sum(new)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b = sv.paged_batch(dev(make_table(P.rng, lens, 64, P.n, max(-(-L // 64) for L in lens))), dev(np.array(lens, np.int32)), dev(cu), n_tokens=n,
                           max_new=max(new), max_len=max(lens))
        q = [sixteen_bit(P.rng, (n, heads * 128), "bf16")[0] for _ in range(2)]
        size = sv.paged_attention_workspace_bytes(c, b)
        ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
        want = [torch.empty_like(x) for x in q]
        for x, o in zip(q, want):
            sv.paged_attention(c, b, x, o, ws[0])
        torch.cuda.synchronize()
        streams, out = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(x) for x in q]
        torch.cuda.synchronize()
        for _ in range(20):
            for i in (0, 1):
                sv.paged_attention(c, b, q[i], out[i], ws[i], stream=streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_calls_off_the_current_device_refused():
    """Buffers that are not on the current CUDA device never reach a launch."""
    import torch
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)  # noqa: E731
    codes, scale = z(4 * 2 * 16 * 64, t=torch.uint8), z(8, t=torch.float32)
    c = sv.paged_cache(4, 2, 64, 16, 4, "int8", "bf16", codes, scale, codes, scale)
    b = sv.paged_batch(z(2, 2), z(2), z(3), z(4), max_new=2, max_len=32)
    K, Q = z(4, 128, t=torch.bfloat16), z(4, 256, t=torch.bfloat16)
    with pytest.raises(sv.SVDQError):
        sv.paged_plan(b, 16, z(2), z(2), z(4), z(4), z(4))
    with pytest.raises(sv.SVDQError):
        sv.paged_append(c, b, K, K)
    with pytest.raises(sv.SVDQError):
        sv.paged_attention(c, b, Q, Q.clone(), z(1 << 20, t=torch.uint8))
    with pytest.raises(sv.SVDQError):
        sv.paged_batch(z(2, 2), z(2), z(3), max_new=2, max_len=32)   # neither slots nor n_tokens


def test_counts_near_2_31_refused():
    c, big = raw_cache(), 2 ** 31 - 65536
    for bad in (dict(n_tokens=big), dict(max_len=big, max_blocks=(2 ** 31 - 1) // 16, B=1)):
        b = raw_batch(**bad)
        assert call_append(c, b) == call_attend(c, b) == call_plan(raw_batch(lens=12288, **bad)) == sv.ERR_UNSUPPORTED
    b = raw_batch(max_new=2 ** 30)                         # two query heads a key head: 2^31 rows a request
    assert call_attend(c, b) == sv.ERR_UNSUPPORTED and sv.lib().svdq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b)) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("max_len,new", [(0, [1, 0, 1]), (40, [2, 3, 40])])
def test_attention_over_empty_caches(gpu, max_len, new):
    """Requests without a cached token, and more new tokens than cached ones: rows that see nothing are 0."""
    for B in (1, 60):
        P = Pool(2, 4, 4, 64, 16, 4, "int8", "bf16")
        lens = [0, min(max_len, 17), 0] * B
        table = np.zeros((3 * B, 4), np.int32)
        table[1::3, :2] = (1, 3)
        run_attend(P, new * B, lens, True, "bf16", table, max_len=max_len)
        run_attend(P, new * B, lens, False, "bf16", table, max_len=max_len)
    assert sv.get_status() == sv.OK
