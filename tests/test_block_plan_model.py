"""Host model of the block-sparse work lists: the numbering of blocks, pairs and groups along a pack, and the merging of
two lists into steps (``csrc/sparse_plan_sm100.cuh``), over random packs."""
import random

import pytest


def first_unit(cu, s, log2):
    return (cu[s] >> log2) + s


def unit_at(cu, total, longest, row, log2):
    lo, hi = 0, len(cu) - 1
    while hi - lo > 1:
        mid = (lo + hi) >> 1
        if first_unit(cu, mid, log2) <= row:
            lo = mid
        else:
            hi = mid
    beg, end = cu[lo], cu[lo + 1]
    ok = beg >= 0 and beg < end <= total and end - beg <= longest
    unit = row - first_unit(cu, lo, log2)
    n = (end - beg + (1 << log2) - 1) >> log2 if ok else 0
    return (lo, unit) if 0 <= unit < n else None


def _packs():
    rng = random.Random(11)
    for _ in range(300):
        n = rng.randint(1, 40)
        lens = [rng.choice([0, 0, 1, 127, 128, 129, 255, 256, 257, 1024, rng.randint(1, 3000)]) for _ in range(n)]
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        yield cu


@pytest.mark.parametrize("log2", [7, 8, 10])
def test_every_unit_has_one_row_and_every_row_at_most_one_unit(log2):
    for cu in _packs():
        total, batch = cu[-1], len(cu) - 1
        rows = (total >> log2) + batch
        found = [u for u in (unit_at(cu, total, total, r, log2) for r in range(rows)) if u]
        want = [(s, b) for s in range(batch) for b in range((cu[s + 1] - cu[s] + (1 << log2) - 1) >> log2)]
        assert sorted(found) == want
        # and the formula that names a block's row agrees with the search
        for s, b in want:
            assert unit_at(cu, total, total, first_unit(cu, s, log2) + b, log2) == (s, b)


def test_bad_packs_stay_inside_the_tables():
    """Whatever cu_seqlens holds, a unit that is found is one of a segment inside [0, total], and its row is in range."""
    rng = random.Random(12)
    for _ in range(2000):
        total, batch = rng.randint(1, 5000), rng.randint(1, 10)
        cu = [rng.randint(-3000, 8000) for _ in range(batch + 1)]
        for log2 in (7, 8, 10):
            rows = (total >> log2) + batch
            for r in range(rows):
                u = unit_at(cu, total, total, r, log2)
                if u is None:
                    continue
                s, b = u
                assert 0 <= cu[s] < cu[s + 1] <= total
                # the block rows that a pair or a group of this segment touches
                for blk in range(b << (log2 - 7), min((b + 1) << (log2 - 7), (cu[s + 1] - cu[s] + 127) // 128)):
                    assert 0 <= (cu[s] >> 7) + s + blk < (total >> 7) + batch


def test_bad_packs_have_a_map_for_every_unit():
    """Tensor maps are written for segment s by warp s of a plan, whichever segment that warp's own row is found to be."""
    def mapped(cu, total, warps):
        return {s for s in range(warps) if s < len(cu) - 1 and cu[s] >= 0 and cu[s] < cu[s + 1] <= total}

    rng = random.Random(13)
    packs = [[0, 5000, 300, 6000]]  # the first units of the last segment are found to be the first segment's
    packs += [[rng.randint(-3000, 8000) for _ in range(rng.randint(2, 11))] for _ in range(2000)]
    late = False
    for cu in packs:
        total = 6000
        for log2 in (7, 8):
            rows = (total >> log2) + len(cu) - 1
            found = [unit_at(cu, total, total, r, log2) for r in range(rows)]
            have = mapped(cu, total, rows)
            assert all(u[0] in have for u in found if u)
            late |= any(u and (u[0], 0) not in found for u in found)
    assert late


def merge(l0, l1):
    """(steps as pairs with None, shared steps): common blocks first, then the rest side by side."""
    both = [v for v in l0 if v in l1]
    r0, r1 = [v for v in l0 if v not in l1], [v for v in l1 if v not in l0]
    n = max(len(r0), len(r1))
    pad = lambda r: r + [None] * (n - len(r))  # noqa: E731
    return [(v, v) for v in both] + list(zip(pad(r0), pad(r1))), len(both)


def producer(steps, common, n0, n1):
    """Order of the tiles that the producer loads: (K or V, tile or both, step)."""
    out = []
    if n0:
        out.append(("K", 0, 0))
    if n1 and common == 0:
        out.append(("K", 1, 0))
    for j in range(len(steps)):
        if j < n0:
            out.append(("V", 0, j))
            if j + 1 < n0:
                out.append(("K", 0, j + 1))
        if j < n1:
            if j >= common:
                out.append(("V", 1, j))
            if j + 1 < n1 and j + 1 >= common:
                out.append(("K", 1, j + 1))
    return out


def consumer(steps, common, n0, n1, slots):
    """Order in which the MMA warp takes tiles, checking that each tile is taken before it is used and released once,
    and that never more than `slots` are held."""
    taken, held, uses = [], set(), []

    def take(t):
        taken.append(t)
        held.add(t)
        assert len(held) <= slots

    def use(t, release):
        assert t in held
        uses.append(t)
        if release:
            held.remove(t)

    cnt, k = (n0, n1), None
    for t in (0, 1):
        if cnt[t] == 0:
            continue
        if t == 0 or common == 0:
            k = ("K", t, 0)
            take(k)
        use(k, t == 1 or common == 0)
    for j in range(len(steps)):
        shared, shared_next = j < common, j + 1 < common
        for t in (0, 1):
            if j >= cnt[t]:
                continue
            if t == 0 or not shared:
                v = ("V", t, j)
                take(v)
            use(v, t == 1 or not shared)
            if j + 1 < cnt[t]:
                if t == 0 or not shared_next:
                    k = ("K", t, j + 1)
                    take(k)
                use(k, t == 1 or not shared_next)
    assert not held
    return taken, uses


def test_merged_steps_and_the_ring_order():
    rng = random.Random(13)
    for _ in range(3000):
        nb = rng.randint(1, 30)
        l0 = sorted(rng.sample(range(nb), rng.randint(0, nb)))
        l1 = sorted(rng.sample(range(nb), rng.randint(0, nb)))
        steps, common = merge(l0, l1)
        assert len(steps) == max(len(l0), len(l1))
        # tile t is active exactly in its first cnt_t steps, and meets exactly its own list
        for t, lst in ((0, l0), (1, l1)):
            assert sorted(s[t] for s in steps[:len(lst)]) == lst
            # the short last block, if the tile meets it, is the last of the shared or the last of the tile's steps
            if lst and lst[-1] == nb - 1:
                at = [s[t] for s in steps[:len(lst)]].index(nb - 1)
                assert at == (common - 1 if nb - 1 in l0 and nb - 1 in l1 else len(lst) - 1)
        taken, uses = consumer(steps, common, len(l0), len(l1), slots=3)
        assert taken == producer(steps, common, len(l0), len(l1))
        assert len(uses) == 2 * (len(l0) + len(l1))


# ---------------------------------------------------------------- splitting rules of the norms (csrc/block_norm.cu)

SMEM_PER_SM = 208 * 1024
SMEM_PER_BLOCK = 227 * 1024 - 8 * 1024  # the device's limit less the kernels' static shared memory


def split_fwd(hidden, row_bytes, rows):
    warps = 1 if hidden <= 2304 else 2 if hidden < 4096 else 4
    room = (SMEM_PER_SM - 12 * hidden) // row_bytes
    groups = max(1, min(24 // warps, room * 2 // 3, rows))
    stages = max(1, min(8, room // groups))
    return warps, groups, stages, 12 * hidden + groups * stages * row_bytes


def split_bwd(hidden, row_bytes):
    vecs = 1 if hidden <= 2048 else 2 if hidden <= 4096 else 4
    team_warps = (hidden + 256 * vecs - 1) // (256 * vecs)
    teams = 8 // team_warps
    per_sm = 16 // (teams * team_warps) if vecs == 1 else 1
    stages = min(24, max(1, (SMEM_PER_SM // per_sm - 8 * hidden) // row_bytes))
    warps, row_warps = teams * team_warps, 1
    while 2 * row_warps <= warps and 4 * row_warps * min(warps // row_warps, stages) < 3 * warps:
        row_warps *= 2
    tile = max(1, min(warps // row_warps, stages, 12))
    return dict(vecs=vecs, team_warps=team_warps, teams=teams, per_sm=per_sm, stages=stages, warps=warps,
                row_warps=row_warps, tile=tile, smem=8 * hidden + stages * row_bytes)


def test_norm_splits_fit_for_every_width():
    for hidden in range(8, 8193, 8):
        for wide in (2, 4):
            for row_bytes in (wide * hidden, (wide + 2) * hidden):
                for rows in (1, 5, 1000):
                    warps, groups, stages, smem = split_fwd(hidden, row_bytes, rows)
                    assert groups * warps <= 24 and groups * stages <= 8 * 24 and smem <= SMEM_PER_BLOCK
                    assert groups <= 24 // warps and (warps == 1 or groups <= 15)  # a named barrier each
                    assert groups * 8 <= groups * warps * 32  # threads that initialise the barriers
            for row_bytes in (wide * hidden, (wide + 2) * hidden, (2 * wide + 2) * hidden, (2 * wide + 4) * hidden):
                s = split_bwd(hidden, row_bytes)
                assert s["team_warps"] * 256 * s["vecs"] >= hidden and 1 <= s["warps"] <= 8
                assert s["row_warps"] <= s["warps"], "a group's barrier would count warps that the block does not have"
                assert s["tile"] * s["row_warps"] <= s["warps"] and s["tile"] <= s["stages"]
                assert s["smem"] <= SMEM_PER_BLOCK and s["stages"] <= s["warps"] * 32
                assert s["per_sm"] * (s["smem"] + 8 * 1024) <= 227 * 1024 + 4 * 1024 * s["per_sm"] or s["stages"] == 1
