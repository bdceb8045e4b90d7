"""A host model of gdn_attn_decode_shared's split: the shares cover every tile
of every job once, no two ranges share a slot, every slot lies inside the
workspace the call asks for, and the shares from a job's first range to its
last all hold one (the join walks them)."""
import random

import pytest

import gated_deltanet_linear_06_gb300 as gdn
from gated_deltanet_linear_06_gb300 import build as gbuild

TILE, COST_PREFIX, COST_TAIL, COST_JOB = 128, 4, 4, 2     # as in csrc/gdn_attn_shared.cu


def tiles_before(x, pos, per, n):
    d = x - pos - COST_JOB
    return 0 if d <= 0 else min(d // per, n)


def walk(job0, pos0, x0, x1, jobs):
    """A share's ranges, by the kernel's walk from its first job."""
    pos, out = pos0, []
    for j in range(job0, len(jobs)):
        if pos >= x1:
            break
        per, n, cost = jobs[j]
        a, b = tiles_before(x0, pos, per, n), tiles_before(x1, pos, per, n)
        pos += cost
        if a < b:
            out.append((j, a, b))
    return out


@pytest.mark.parametrize("seed", range(60))
def test_shares_cover_every_tile_once_and_in_a_row(seed):
    rng = random.Random(seed)
    batch, steps = rng.choice([1, 2, 7, 40, 200]), rng.choice([1, 1, 3, 8])
    hkv, G = rng.choice([1, 2, 5]), rng.choice([1, 2, 6, 8, 16])
    prefix = rng.choice([0, 1, 100, 128, 700, 5000, 33000])
    ncta = rng.choice([76, 80, 10])      # pairs of CTAs
    tails = [rng.choice([0, 1, rng.randrange(2000)]) for _ in range(batch)]
    ntok, R, tpb = batch * steps, steps * G, 128 // G
    nmb, pt = -(-ntok // (2 * tpb)), -(-prefix // TILE)
    np_ = hkv * nmb if pt else 0
    jobs = [(COST_PREFIX, pt, pt * COST_PREFIX + COST_JOB)] * np_
    scan = [0]
    for n in tails:
        t = -(-n // TILE)
        c = t * COST_TAIL + COST_JOB if n else 0
        jobs += [(COST_TAIL, t, c)] * hkv
        scan.append(scan[-1] + c * hkv)
    wp = np_ * (pt * COST_PREFIX + COST_JOB)
    total = wp + scan[-1]
    assert total == sum(c for _, _, c in jobs)
    shares = max(1, min(ncta, total // max(COST_PREFIX, COST_TAIL)))
    start = [total * c // shares for c in range(shares + 1)]

    done = [0] * len(jobs)
    slots, ranges = set(), {}
    prefix_rows = (np_ + ncta) * 256 if np_ else 0
    all_rows = prefix_rows + (batch * hkv + ncta) * R
    for c in range(shares):
        if start[c] >= total:
            continue
        if start[c] < wp:
            cost = pt * COST_PREFIX + COST_JOB
            job0, pos0 = start[c] // cost, start[c] // cost * cost
        else:
            b = max(i for i in range(batch) if scan[i] <= start[c] - wp)
            job0, pos0 = np_ + b * hkv, wp + scan[b]
        for j, a, b in walk(job0, pos0, start[c], start[c + 1], jobs):
            assert a == done[j]
            done[j] = b
            rows = 256 if j < np_ else R
            row0 = (j + c) * 256 if j < np_ else prefix_rows + (j - np_ + c) * R
            assert row0 not in slots and 0 <= row0 and row0 + rows <= all_rows
            slots.add(row0)
            ranges.setdefault(j, []).append((c, row0))
    assert done == [n for _, n, _ in jobs]

    # the join's view: consecutive shares, slots one job's rows apart
    for j, found in ranges.items():
        c0, row0 = found[0]
        apart = 256 if j < np_ else R
        assert [c for c, _ in found] == list(range(c0, c0 + len(found)))
        assert [r for _, r in found] == [row0 + apart * i for i in range(len(found))]

    # the workspace holds the costs, the statistics and the outputs of all slots
    gbuild.build()
    dims = gdn.make_attn_dims(h_q=hkv * G, h_kv=hkv, d=64, rot=0)
    if R <= 128:
        assert gdn.gdn_attn_decode_shared_workspace_bytes(dims, batch, steps) >= len(jobs) * 8 + all_rows * (16 + 256)
