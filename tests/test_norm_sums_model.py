"""Host model of how the norms' column sums are added up where a pack has many images (``block_norm_sum_kernel``): every
image is added once, by the block of its own or by the blocks behind them, and no thread walks a long image alone."""
import random

import pytest

SMS = 148


def split(total, hidden):
    vecs = 1 if hidden <= 2048 else 2 if hidden <= 4096 else 4
    team_warps = (hidden + 256 * vecs - 1) // (256 * vecs)
    teams = 8 // team_warps
    per_sm = 16 // (teams * team_warps) if vecs == 1 else 1
    rows = max(1, -(-total // (SMS * per_sm)))
    return teams, rows, -(-total // rows)


def adders(cu, hidden):
    """Per image: (column blocks that add it, most slots that one thread adds)."""
    total, batch = cu[-1], len(cu) - 1
    teams, rpc, chunks = split(total, hidden)
    long_runs = max(1, 32 // teams)
    by = -(-hidden // 1024)
    col_blocks = -(-hidden // (32 * by))
    out = {s: [] for s in range(batch)}

    def slots(s):
        beg, end = cu[s], cu[s + 1]
        return teams * (min((end - 1) // rpc + 1, chunks) - beg // rpc) if end > beg else 0

    for s in range(batch):
        if slots(s) <= long_runs * teams:
            out[s].append((range(0, hidden, 4), slots(s)))
    stride = long_runs * rpc
    for x in range(-(-chunks // long_runs) * col_blocks):
        j, rest = divmod(x, col_blocks)
        s = max(i for i in range(batch) if cu[i] <= j * stride)
        if slots(s) <= long_runs * teams or -(-cu[s] // stride) != j:
            continue
        for y in range(by):
            first = (rest * by + y) * 32
            out[s].append((range(first, min(first + 32, hidden), 4), -(-slots(s) // 32)))
    return out


def _packs():
    rng = random.Random(5)
    for _ in range(60):
        lens = [rng.choice([0, 1, 7, 64, 200, rng.randint(1, 900)]) for _ in range(rng.randint(41, 90))]
        for _ in range(rng.randint(0, 3)):
            lens[rng.randrange(len(lens))] = rng.randint(1, 70000)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        if cu[-1]:
            yield cu


@pytest.mark.parametrize("hidden", [8, 72, 264, 520, 1152, 1536, 2056, 4104, 8192])
def test_every_image_is_added_once(hidden):
    for cu in _packs():
        for s, parts in adders(cu, hidden).items():
            cols = sorted(c for p, _ in parts for c in p)
            assert cols == list(range(0, hidden, 4)), (s, cu)
            assert max(n for _, n in parts) <= 80  # (2368 slots in 32 parts)
