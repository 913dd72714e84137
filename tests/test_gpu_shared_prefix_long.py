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
    for i in range(P // c.bs + (P % c.bs > 0 and c.lens[rows[0]] <= P)):       # (a last block with the first request's own tokens is its own)
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


# ------------------------------------------------ windows, bad input, peaks and order on every kernel
@pytest.mark.parametrize("window", [1, 100, 512, 1000])
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_windows_on_every_kernel(hyb, devstatus, dt, D, Hq, Hk, rows, window):
    tails = [1 + (i * 37) % 600 for i in range(rows)]
    c = Case(hyb, [(1100, tails), (37, [5, -20, 600]), (0, [700, 2])], Hq, Hk, D, dt, bs=32, window=window, seed=window, slack=40)
    spare_block(c)
    for g in range(3):
        release(c, g, "someone else's")
    for b, n in enumerate(c.lens):                   # a request's own blocks before its window
        P = c.pre[sum(b >= x for x in c.cu[1:])]
        first = b in c.cu
        c.bt[b, -(-P // c.bs) if first else P // c.bs:max(0, n - window) // c.bs] = -1
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_bad_blocks_on_every_kernel(hyb, devstatus, dt, D, Hq, Hk, rows):
    c = Case(hyb, [(900, [1 + (i * 7) % 50 for i in range(rows)]), (0, [40])], Hq, Hk, D, dt, seed=6)
    for i, bad in ((0, c.NB), (7, -1), (8, -7), (30, c.NB + 5), (55, -1)):
        c.bt[0, i] = bad
    c.bt[rows, :] = -7                     # all of a request
    hyb.check(c.call())
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_BLOCK)
    c.bt[c.bt >= c.NB] = -1
    R.check_attention(c.out, c.ref(), dt)
    assert (c.out[rows] == 0).all()


@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_non_finite_values_on_every_kernel(hyb, dt, D, Hq, Hk, rows):
    """A request's NaN in q or among its own tokens stays within it."""
    c = Case(hyb, [(650, [20 + i % 50 for i in range(rows)]), (150, [30])], Hq, Hk, D, dt, seed=7)
    clean = c.check().clone()
    c.q[1, Hq - 1, 5] = math.nan
    c.q[rows, 0, 1] = math.inf
    c.vc[c.bt[2, 650 // 16 + 1].long(), 0, 3, 7] = math.inf          # token 659 of request 2
    hyb.check(c.call())
    assert c.out[1, Hq - 1].isnan().all() and torch.equal(c.out[1, :Hq - 1], clean[1, :Hq - 1])
    assert not c.out[rows, 0].isfinite().any() and torch.equal(c.out[rows, 1:], clean[rows, 1:])
    rep = Hq // Hk
    assert not c.out[2, :rep, 7].isfinite().any() and torch.equal(c.out[2, rep:], clean[2, rep:])
    rest = [b for b in range(rows) if b not in (1, 2)]
    assert torch.equal(c.out[rest], clean[rest])


def peaks(c, P, profile, rows):
    """Scores that rise, fall or spike by dozens along the keys, for queries that look along the first."""
    c.q[:] = c.q.sign() * 0.5
    D = c.q.shape[-1]
    along = c.q[0, 0].sign().float() / D ** 0.5
    for b in range(rows):
        n = c.lens[b]
        at = torch.arange(0 if b == 0 else P, n, device="cuda")
        z = {"rising": at / n, "falling": 1 - at / n, "spike": (at % 777 == 5).float(), "waves": torch.sin(at / 90.0)}[profile] * 40
        c.kc[c.bt[b, at // c.bs].long(), :, at % c.bs] = (z[:, None] * along).to(c.dt)[:, None]


@pytest.mark.parametrize("profile", ["rising", "falling", "spike", "waves"])
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_peaked_scores_on_every_kernel(hyb, profile, dt, D, Hq, Hk, rows):
    c = Case(hyb, [(1600, [3 + (i * 17) % 90 for i in range(rows)])], Hq, Hk, D, dt, seed=3)
    peaks(c, 1600, profile, rows)
    c.check(profile)


@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_order_on_every_kernel(hyb, devstatus, dt, D, Hq, Hk, rows):
    """Calls one behind the other on one workspace, each fed by a kernel just before it; a captured call replayed with other
    lengths; two streams with workspaces of their own."""
    in_order(hyb, Case(hyb, [(900, [3 + (i * 7) % 40 for i in range(rows)]), (64, [3, 200])], Hq, Hk, D, dt, seed=10, slack=30))
    assert devstatus() == (0, 0)


def in_order(hyb, c):
    want, outs = [], []
    qs = [c.q.clone(), c.q.flip(0), c.q * 0.5, -c.q]
    for q in qs:
        c.q.copy_(q)
        want.append(c.check().clone())
    torch.cuda.synchronize()
    for i in range(40):                              # the queries change behind the last call's back, the outputs move away
        c.q.copy_(qs[i % 4])
        hyb.check(c.call())
        outs.append(c.out.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 4]) for i, o in enumerate(outs))
    others = [torch.empty_like(c.out) for _ in range(4)]
    c.q.copy_(qs[1])
    for o in others:                                 # nothing between them but the workspace
        hyb.check(c.call(o))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[1]) for o in others)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hyb.check(c.call())
        hyb.check(c.call(others[0]))
    c.dev[0][1] -= 2
    c.lens[1] -= 2
    c.out.fill_(7)
    for _ in range(5):
        graph.replay()
    R.check_attention(c.out, c.ref(), c.dt)
    assert torch.equal(c.out, others[0])
    two = [torch.empty_like(c.out) for _ in range(2)]
    spaces = [torch.empty_like(c.ws) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, two, spaces):
            hyb.check(c.call(o, w, s))
    torch.cuda.synchronize()
    assert torch.equal(two[0], c.out) and torch.equal(two[1], c.out)


# ------------------------------------------------ many key tiles in a CTA of the tensor-core kernel
def tall(hyb, P, Hq, window=0, seed=1):
    """A group of 70 requests on P tokens, 8 key heads, and 18 small ones: as many (group, key head) units as SMs, so that
    each has one CTA, which walks all key tiles."""
    c = Case(hyb, [(P, [1 + (i * 7) % 40 for i in range(70)])] + [(30 + 9 * g, [1 + g % 3] * (1 + g % 2)) for g in range(18)], Hq, 8, 128, seed=seed, window=window)
    spare_block(c)
    parts = c.n // (c.B * Hq * (128 * 4 + 8)) - 1    # one of the requests' own tokens
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert parts == 1
    return c


TALL = [(600, 8), (1152, 32), (1153, 24), (8190, 8), (8190, 32)]     # 5, 9, 10 and 64 key tiles; 1, 4 and 3 query heads a key head


@pytest.mark.parametrize("P,Hq", TALL)
def test_many_key_tiles(hyb, devstatus, P, Hq):
    tall(hyb, P, Hq).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("P,Hq", TALL)
@pytest.mark.parametrize("share", [0.3, 0.97])
def test_many_key_tiles_in_a_window(hyb, devstatus, P, Hq, share):
    c = tall(hyb, P, Hq, window=int(P * share))
    release(c, 0, "someone else's")
    c.check()
    # and some requests that end early: their windows lie before the others'
    c = tall(hyb, P, Hq, window=int(P * share))
    for b in range(0, 70, 5):
        c.lens[b] = P // 3 + b
    c.dev[0].copy_(torch.tensor(c.lens, dtype=torch.int32))
    release(c, 0, "someone else's")
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("P,Hq", TALL)
def test_many_key_tiles_with_bad_blocks(hyb, devstatus, P, Hq):
    c = tall(hyb, P, Hq)
    clean = c.check().clone()
    for i in range(3, P // 16, 11):
        c.bt[0, i] = -1 if i % 2 else c.NB
    hyb.check(c.call())
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_BLOCK)
    c.bt[c.bt >= c.NB] = -1
    R.check_attention(c.out, c.ref(), c.dt)
    assert torch.equal(c.out[70:], clean[70:])


@pytest.mark.parametrize("P,Hq", TALL)
@pytest.mark.parametrize("profile", ["rising", "falling", "spike", "waves"])
def test_many_key_tiles_of_peaked_scores(hyb, profile, P, Hq):
    """The maximum moves in every tile, in one, or now and then: the sums are rescaled behind the second tile too."""
    c = tall(hyb, P, Hq)
    peaks(c, P, profile, 70)
    c.check(profile)


@pytest.mark.parametrize("P,Hq", TALL[1:4])
def test_many_key_tiles_in_order(hyb, devstatus, P, Hq):
    c = tall(hyb, P, Hq)
    clean = c.check().clone()
    q = c.q.clone()
    c.q[1, Hq - 1, 5] = math.nan
    hyb.check(c.call())
    assert c.out[1, Hq - 1].isnan().all() and torch.equal(c.out[1, :Hq - 1], clean[1, :Hq - 1]) and torch.equal(c.out[2:], clean[2:])
    c.q.copy_(q)
    in_order(hyb, c)
    assert devstatus() == (0, 0)


# ------------------------------------------------ limits
@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_bounds_far_above_the_lengths(hyb, devstatus, dt, D, Hq, Hk, rows):
    """Bounds as a captured step holds them: the whole batch in a group, prefixes and answers as long as the table."""
    c = Case(hyb, [(300, [1 + i % 30 for i in range(rows)]), (5, [60]), (0, [0])], Hq, Hk, D, dt, seed=2, extra_rows=3)
    wide = torch.full((c.B, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.bt.shape[1]] = c.bt
    c.bt, c.d.max_blocks_per_seq = wide, 2048
    c.p = hyb.prefix_dims(Hq, c.G, c.B, 2048 * 16, 2048 * 16)
    c.n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(c.B, c.p, c.d)
    c.ws = torch.full((c.n // 4 + 4,), math.nan, device="cuda")
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("Hq", [64, 65, 100, 127, 128, 129])
def test_query_heads_about_a_row_tile(hyb, devstatus, Hq):
    Case(hyb, [(400, [1, 40, 3]), (513, [9] * 2), (20, [-4])], Hq, 1, 128, seed=Hq).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("D", [16, 64])
def test_the_most_heads(hyb, devstatus, D):
    H = 65535
    Case(hyb, [(20, [1, 3])], H, H, D, seed=1).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D", [(B16, 64), (F32, 64), (B16, 16)])
def test_the_largest_batch(hyb, devstatus, dt, D):
    """65535 requests: groups of none, one and many."""
    c = Case(hyb, [(30, [1 + i % 20 for i in range(300)])], 1, 1, D, dt, seed=3)
    B, n0 = 65535, 300
    pick = torch.arange(B, device="cuda") % n0               # each request many times, in groups of its own
    q, bt = torch.randn(B, 1, D, device="cuda").to(dt), c.bt[pick].contiguous()
    bt[:, 0] = c.bt[0, 0]
    lens = c.dev[0][pick].contiguous()
    cu, at = [0], 0
    while at < B:
        at = min(B, at + [0, 1, 7, 60][len(cu) % 4])
        cu.append(at)
    G = len(cu) - 1
    # the block in which the prefix ends is each request's own: it holds the same tokens there
    out = torch.full((B, 1, D), 7.0, device="cuda", dtype=dt)
    cu_d, pre = torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.full((G,), 30, dtype=torch.int32, device="cuda")
    p = hyb.prefix_dims(1, G, 60, 30, 20)
    n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(B, p, c.d)
    ws = torch.empty(n // 4 + 4, device="cuda")
    hyb.check(hyb.hyb_paged_attn_decode_shared_prefix(out, q, c.kc, c.vc, bt, lens, cu_d, pre, B, p, c.d, ws, n))
    rows = sorted({0, 1, 2, 59, 60, 31999, 32768, B - 2, B - 1, *range(5, B, 331)})
    # the plain form, each row a group of its own
    ref = R.attention(q[rows], c.kc, c.vc, bt[rows], lens[rows].tolist(), list(range(len(rows) + 1)), [30] * len(rows), c.d.scale)
    R.check_attention(out[rows], ref, dt)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D,rows", [(B16, 64, 2), (B16, 128, 66), (F32, 16, 2), (F32, 16, 9)])
def test_the_longest_prefix(hyb, devstatus, dt, D, rows):
    """2^24 tokens, one key head."""
    P, bs = 1 << 24, 256
    gen = torch.Generator(device="cuda").manual_seed(4)
    kc, vc = (torch.randn(P // bs + 1, 1, bs, D, generator=gen, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(rows, 1, D, generator=gen, device="cuda").to(dt)
    NB = P // bs + 1
    d = hyb.dims(1, D, NB, NB, dt, block_size=bs)
    bt = torch.arange(NB - 1, -1, -1, dtype=torch.int32, device="cuda").expand(rows, NB).contiguous()
    lens = [P + 1, P - 12345] + [P + 1 + i % 200 for i in range(rows - 2)]
    dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, [0, rows], [P])]
    p = hyb.prefix_dims(1, 1, rows, P, 256)
    n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(rows, p, d)
    ws, out = torch.full((n // 4 + 4,), math.nan, device="cuda"), torch.empty_like(q)
    hyb.check(hyb.hyb_paged_attn_decode_shared_prefix(out, q, kc, vc, bt, *dev, rows, p, d, ws, n))
    # all rows share one table: softmax sums over chunks of the sequence, scores are small enough for no maximum
    x, L = q[:, 0].double() * d.scale, torch.tensor(lens, device="cuda")
    num, mag = (torch.zeros(rows, D, dtype=torch.float64, device="cuda") for _ in range(2))
    den, amax = (torch.zeros(rows, 1, dtype=torch.float64, device="cuda") for _ in range(2))
    step = 4096
    for b0 in range(0, NB, step):
        ids = bt[0, b0:b0 + step].long()
        k, v = (c[ids, 0].double().flatten(0, 1) for c in (kc, vc))
        at = b0 * bs + torch.arange(len(k), device="cuda")
        w = torch.exp(x @ k.T) * (at < L[:, None])
        num += w @ v
        mag += w @ v.abs()
        den += w.sum(-1, keepdim=True)
        amax = torch.maximum(amax, (x.abs() @ k.abs().T).amax(-1, keepdim=True))
    ref = (num / den)[:, None], (mag / den)[:, None], amax[:, None], L.double()[:, None, None]
    lim = R.HALF[dt] * ref[0].abs() + ref[1] * (2 * D * R.U * ref[2] + 2.0 ** -22 + 4 * R.U * ref[3].sqrt() + (2.0 ** -8 + ref[3] / 16 * 2.0 ** -23 if dt == B16 else 0))
    assert ((out.double() - ref[0]).abs() <= lim * (1 + 2.0 ** -6) + 1e-30).all()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D,Hq,Hk,rows", KERNELS)
def test_tokens_behind_all_requests(hyb, devstatus, dt, D, Hq, Hk, rows):
    """Where every request is shorter than its prefix, what stands behind the longest in its last block reaches none."""
    c = Case(hyb, [(1000, [-1000 + 37 + (i * 131) % 700 for i in range(rows)]), (60, [3])], Hq, Hk, D, dt, bs=32, seed=rows)
    n = max(c.lens[:rows])
    assert n % 16 and n < 1000
    for x in (c.kc, c.vc):
        x[c.bt[0, n // 32].long(), :, n % 32:] = math.nan
    c.check()
    assert devstatus() == (0, 0)
