"""Paged 8-bit KV cache at its limits: lengths that disagree with the free ring, value scales far apart, the smallest
and the largest magnitudes, skipped and misplaced tokens, bad pointers, and batches of many hundred requests."""
import random

import numpy as np
import pytest

import rank_gemm_svdq_b200 as sv
from oracle import pagedkv as pk
from tests.test_paged import dev


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
