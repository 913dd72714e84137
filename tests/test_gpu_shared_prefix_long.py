"""Shared-prefix decode attention on every one of its kernels: table entries that no request sees, and CTAs of
the tensor-core kernel that walk many key tiles."""
import math

import pytest
import torch

import beam_ref as R
from test_gpu_shared_prefix import Case

pytestmark = pytest.mark.gpu

B16, F32 = torch.bfloat16, torch.float32
# (type, head size, query heads, key heads, requests): the kernels of up to 16, 32 and 64 rows of a key head, several
# row tiles, the tensor cores (one and two pairs of row tiles), and those without matrix instructions
KERNELS = [(B16, 128, 2, 2, 4), (B16, 64, 3, 3, 20), (B16, 128, 2, 2, 40), (B16, 64, 2, 2, 80), (B16, 256, 4, 2, 24), (B16, 128, 2, 2, 70), (B16, 128, 12, 3, 70),
           (B16, 32, 2, 2, 4), (B16, 32, 2, 2, 12), (F32, 64, 2, 2, 4), (F32, 64, 2, 2, 12), (F32, 128, 4, 2, 40)]


def release(c, group, how):
    """Puts what nobody may read into the entries of the group's prefix that none of its requests sees; returns how many."""
    P, rows = c.pre[group], range(c.cu[group], c.cu[group + 1])
    spans = [(max(0, c.lens[b] - c.window) if c.window else 0, min(P, c.lens[b])) for b in rows]
    n = 0
    for i in range(P // c.bs + (P % c.bs > 0 and min(c.lens[b] for b in rows) < P)):
        if not any(max(lo, i * c.bs) < min(hi, (i + 1) * c.bs) for lo, hi in spans):
            c.bt[c.cu[group], i] = {"none": -1, "outside": c.NB, "someone else's": int(c.spare)}[how]
            n += 1
    return n


def spare_block(c):
    """A block of the pool that no table names: it holds NaN."""
    used = set(c.bt.flatten().tolist())
    c.spare = next(i for i in range(c.NB) if i not in used)
    assert c.kc[c.spare].isnan().all() and c.vc[c.spare].isnan().all()


@pytest.mark.parametrize("how", ["none", "outside", "someone else's"])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_entries_behind_all_requests(hyb, devstatus, dt, D, Hq, Hk, rows, bs, how):
    """Every request is shorter than its prefix: the entries behind the longest one are not read."""
    c = Case(hyb, [(1500, [-1500 + 37 + (i * 131) % 700 for i in range(rows)]), (700, [-650 + i % 9 for i in range(rows)]), (60, [3, -60])], Hq, Hk, D, dt, bs=bs, seed=rows)
    spare_block(c)
    assert release(c, 0, how) > 700 // bs and release(c, 1, how) > 500 // bs
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("how", ["none", "outside", "someone else's"])
@pytest.mark.parametrize("window", [90, 333])
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_entries_between_windows(hyb, devstatus, dt, D, Hq, Hk, rows, window, how):
    """Some requests end early in the prefix, others behind it: the blocks between their windows are not read."""
    tails = [-1800 + 400 + (i * 29) % 150 if i % 3 == 1 else 1 + (i * 7) % 40 for i in range(rows)]
    c = Case(hyb, [(1800, tails), (1200, [20 + i % 5 for i in range(rows)]), (60, [3, -60])], Hq, Hk, D, dt, bs=32, window=window, seed=rows)
    spare_block(c)
    assert release(c, 0, how) > (1800 - 600 - 2 * window) // 32 and release(c, 1, how) > 10
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_no_request_of_a_group_sees_its_prefix(hyb, devstatus, dt, D, Hq, Hk, rows, window):
    c = Case(hyb, [(700, [-700] * rows), (650, [200 + i % 3 for i in range(rows)]), (60, [3, -60])], Hq, Hk, D, dt, window=window, seed=rows)
    spare_block(c)
    for how in ("none", "outside", "someone else's"):
        assert release(c, 0, how) == 44 and release(c, 1, how) == (40 if window else 0)
        c.check(how)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
@pytest.mark.parametrize("n,window", [(1005, 300), (1001, 990), (1015, 140), (1005, 5)])
def test_tokens_before_every_window(hyb, dt, D, Hq, Hk, rows, n, window):
    """What stands in a block before the first token that some request sees reaches none of them, NaN or not."""
    c = Case(hyb, [(1000, [n - 1000] * rows), (60, [3])], Hq, Hk, D, dt, window=window, seed=rows)
    lo = n - window
    assert lo % 16 and lo <= 1000
    for x in (c.kc, c.vc):
        x[c.bt[0, lo // 16].long(), :, :lo % 16] = math.nan
    c.check()
