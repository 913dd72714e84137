"""Shared-prefix decode attention against its 64-bit form."""
import math

import pytest
import torch

import beam_ref as R

pytestmark = pytest.mark.gpu


class Case:
    """Groups of (prefix, [own tokens, ...]); own tokens may be negative: a request shorter than
    the prefix. Slots of the pools that no request may read hold NaN."""

    def __init__(self, hyb, groups, Hq, Hk, D, dt=torch.bfloat16, bs=16, window=0, seed=0, amp=1.5, extra_rows=0, spread=0, slack=0, empty_groups=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hyb, self.dt, self.bs, self.window = hyb, dt, bs, window
        self.lens, self.cu, self.pre, rows, ids = [], [0], [], [], 0
        B = sum(len(t) for _, t in groups) + extra_rows
        cols = max([(P + max([0] + list(t)) + bs - 1) // bs for P, t in groups]) + 1
        for P, tails in groups:
            common = list(range(ids, ids + P // bs))
            ids += len(common)
            for i, t in enumerate(tails):
                # the first row holds the whole prefix, others only their own part
                last = (max(P, P + t) + bs - 1) // bs if i == 0 else (max(0, P + t) + bs - 1) // bs
                mine = max(0, last - len(common))
                rows.append((common if i == 0 else [-1] * len(common)) + list(range(ids, ids + mine)))
                rows[-1] += [-1] * (cols - len(rows[-1]))
                ids += mine
                self.lens.append(max(0, P + t))
            self.pre.append(P)
            self.cu.append(len(self.lens))
            if empty_groups:
                self.pre.append(7)
                self.cu.append(len(self.lens))
        rows += [[-1] * cols] * extra_rows
        self.lens += [5] * extra_rows
        self.NB = ids + 2 + spread
        where = torch.randperm(self.NB, generator=gen, device="cuda")
        if spread:
            where[:ids] = self.NB - 1 - torch.arange(ids, device="cuda")     # the end of a large pool
        t = torch.tensor(rows, device="cuda").view(B, cols)
        self.bt = torch.where(t >= 0, where[t.clamp(min=0)], -1).to(torch.int32)
        self.kc, self.vc = (torch.full((self.NB, Hk, bs, D), math.nan, device="cuda", dtype=dt) for _ in range(2))
        b = 0
        for P, tails in groups:
            b0 = b
            for i, t in enumerate(tails):
                at = torch.arange(0 if i == 0 else P, max(P, P + t), device="cuda")
                blk = self.bt[b, at // bs].long()
                for c in (self.kc, self.vc):
                    c[blk, :, at % bs] = torch.randn(len(at), Hk, D, generator=gen, device="cuda").to(dt)
                b += 1
            if P % bs:                                                       # the prefix's end in every row's own block
                for j in range(b0 + 1, b):
                    blk = int(self.bt[j, P // bs])
                    if blk >= 0:
                        for c in (self.kc, self.vc):
                            c[blk, :, :P % bs] = c[self.bt[b0, P // bs].long(), :, :P % bs]
        self.q = (amp * torch.randn(B, Hq, D, generator=gen, device="cuda")).to(dt)
        self.B, self.G = B, len(self.pre)
        size = max([1] + [self.cu[i + 1] - self.cu[i] for i in range(self.G)])
        self.bounds = (size, max(self.pre), max([0] + [self.lens[j] - self.pre[g] for g in range(self.G) for j in range(self.cu[g], self.cu[g + 1])]) + slack)
        self.d = hyb.dims(Hk, D, self.NB, cols, dt, block_size=bs, window=window)
        self.p = hyb.prefix_dims(Hq, self.G, *self.bounds)
        self.dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.lens, self.cu, self.pre)]
        self.out = torch.full((B, Hq, D), 7.0, device="cuda", dtype=dt)
        n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(B, self.p, self.d)
        self.ws = torch.full((n // 4 + 4,), math.nan, device="cuda")          # nothing of it may be relied on
        self.n = n

    def call(self, out=None, ws=None, stream=None):
        out = self.out if out is None else out
        ws = self.ws if ws is None else ws
        return self.hyb.hyb_paged_attn_decode_shared_prefix(out, self.q, self.kc, self.vc, self.bt, *self.dev, self.B, self.p, self.d, ws, self.n, stream)

    def ref(self):
        return R.attention(self.q, self.kc, self.vc, self.bt, self.lens, self.cu, self.pre, self.d.scale, self.window)

    def check(self, what=""):
        self.hyb.check(self.call())
        ref = self.ref()
        R.check_attention(self.out, ref, self.dt, what)
        assert (self.out[ref[0].isnan()] == 7).all()
        return self.out


SMALL = [(37, [1, 20, 5]), (0, [3, 1]), (64, [1, 1, 1, 17, 40]), (16, [33]), (5, [0, 2, -3, -5, 1])]


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, d) for d in (16, 32, 64, 128, 256)] + [(torch.float32, d) for d in (16, 32, 64, 128)])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (6, 2), (8, 1)])
def test_types_and_heads(hyb, devstatus, dt, D, Hq, Hk):
    Case(hyb, SMALL, Hq, Hk, D, dt, seed=D + Hq, extra_rows=2, empty_groups=True).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("bs", [16, 32, 128, 256])
@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("P", [1, 15, 16, 17, 127, 128, 129, 255, 257, 1000])
def test_prefix_ends(hyb, devstatus, P, dt, D, bs):
    Case(hyb, [(P, [1, 16, 17, 0, 130, -1, -P, 3])], 4, 2, D, dt, bs=bs, seed=P).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 63, 65, 127, 128, 129, 257, 300])
@pytest.mark.parametrize("Hq,Hk,D,dt", [(2, 2, 128, torch.bfloat16), (8, 2, 128, torch.bfloat16), (3, 1, 64, torch.bfloat16), (5, 5, 64, torch.bfloat16), (3, 1, 128, torch.bfloat16),
                                        (2, 1, 256, torch.bfloat16), (4, 2, 32, torch.bfloat16), (4, 2, 128, torch.float32), (3, 3, 16, torch.float32)])
def test_group_sizes(hyb, devstatus, rows, Hq, Hk, D, dt):
    """From one row to more than a CTA takes, on both sides of every tile and of the choice of the kernel."""
    tails = [1 + (i * 7) % 50 for i in range(rows)]
    Case(hyb, [(700, tails), (130, tails[:rows // 2 + 1])], Hq, Hk, D, dt, seed=rows).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("Hq,Hk,D", [(17, 1, 64), (24, 1, 128), (40, 2, 128), (96, 1, 128), (130, 1, 128), (20, 1, 256)])
def test_many_query_heads(hyb, devstatus, Hq, Hk, D):
    """More query heads to a key head than a row tile has rows, and than the tensor-core kernel takes."""
    Case(hyb, [(300, [1, 40, 3, 0]), (513, [9] * 5), (20, [-4, 300])], Hq, Hk, D, seed=Hq).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0, 1e-30])
@pytest.mark.parametrize("dt,D,rows", [(torch.bfloat16, 128, 3), (torch.bfloat16, 128, 70), (torch.bfloat16, 32, 9), (torch.float32, 64, 3), (torch.float32, 64, 12)])
def test_scales(hyb, devstatus, scale, dt, D, rows):
    c = Case(hyb, [(200, [1 + i % 9 for i in range(rows)]), (40, [5, 30])], 2, 2, D, dt, seed=rows, amp=0.3)
    c.d.scale = scale
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_no_keys_at_all(hyb, devstatus, dt, D):
    """Bounds of zero, requests without tokens, and a bound on a group of none."""
    c = Case(hyb, [(0, [0, 0]), (0, [0])], 2, 2, D, dt)
    out = c.check()
    assert (out == 0).all()
    c.p = hyb.prefix_dims(2, 2, 0, 5, 0)           # groups of rows, none allowed
    c.n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(c.B, c.p, c.d)
    c.ws = torch.empty(c.n // 4 + 4, device="cuda")
    c.out.fill_(7)
    hyb.check(c.call())
    assert (c.out == 7).all() and devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)


@pytest.mark.parametrize("dt,D,Hq,Hk", [(torch.bfloat16, 128, 8, 2), (torch.bfloat16, 128, 32, 32), (torch.bfloat16, 256, 2, 1), (torch.float32, 64, 3, 3)])
@pytest.mark.parametrize("P", [5000, 20011])
def test_long_prefixes(hyb, devstatus, P, dt, D, Hq, Hk):
    Case(hyb, [(P, [1, 700, 3, 2100]), (P // 3, [50] * 9), (12, [2500])], Hq, Hk, D, dt, seed=P).check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("window", [1, 16, 100, 512, 1000, 3000])
@pytest.mark.parametrize("dt,D,Hq,Hk", [(torch.bfloat16, 128, 4, 2), (torch.bfloat16, 64, 3, 3), (torch.float32, 64, 2, 2)])
def test_windows_and_released_blocks(hyb, devstatus, window, dt, D, Hq, Hk):
    groups = [(1100, [1, 60, 400, 1300]), (37, [5, -20, 600]), (0, [700, 2])]
    c = Case(hyb, groups, Hq, Hk, D, dt, bs=32, window=window, seed=window, slack=40)
    # blocks that no request's window reaches are gone
    for g, P in enumerate(c.pre):
        rows = range(c.cu[g], c.cu[g + 1])
        low = [max(0, c.lens[b] - window) for b in rows]
        c.bt[c.cu[g], :min(min(low), P) // c.bs] = -1
        for b, lo in zip(rows, low):
            if lo > P:
                c.bt[b, P // c.bs + (P % c.bs > 0 and b == c.cu[g]):lo // c.bs] = -1
    c.check()
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("profile", ["rising", "falling", "spike"])
@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_peaked_scores(hyb, profile, dt, D):
    """Scores that rise, fall or spike by dozens over the keys: the running maximum moves through
    tiles, parts and the step from the prefix to the row's own tokens."""
    c = Case(hyb, [(2000, [300, 1, 90, 700])], 2, 1, D, dt, seed=3)
    c.q[:] = c.q.sign() * 0.5
    along = c.q[0, 0].sign().float() / D ** 0.5
    for b in range(4):
        n = c.lens[b]
        at = torch.arange(n, device="cuda")
        rows = torch.where(at < 2000, 0, b)
        z = {"rising": at / n, "falling": 1 - at / n, "spike": (at % 777 == 5).float()}[profile] * 40
        blk = c.bt[rows, at // 16].long()
        fresh = at >= (0 if b == 0 else 2000)
        c.kc[blk[fresh], :, at[fresh] % 16] = (z[fresh, None] * along).to(dt)[:, None]
    c.check(profile)


def test_equal_to_the_plain_decode(hyb):
    """One key head to each query head: the plain decode over whole tables gives the same to rounding, and with
    groups of one and no prefix as well."""
    c = Case(hyb, [(300, [5, 60, 200])], 4, 4, 128, seed=9)
    full = c.bt.clone()
    full[1:, :300 // 16] = full[0, :300 // 16]
    n = hyb.hyb_paged_attn_decode_workspace_size(3, 512, c.d)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    plain, alone = torch.empty_like(c.out), torch.empty_like(c.out)
    hyb.check(hyb.hyb_paged_attn_decode(plain, c.q, c.kc, c.vc, full, c.dev[0], 3, 512, c.d, ws, n))
    c.check()
    ref = c.ref()
    R.check_attention(plain, ref, c.dt)
    p = hyb.prefix_dims(4, 3, 1, 0, 512)
    n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(3, p, c.d)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    hyb.check(hyb.hyb_paged_attn_decode_shared_prefix(alone, c.q, c.kc, c.vc, full, c.dev[0], cu, torch.zeros(3, dtype=torch.int32, device="cuda"), 3, p, c.d, ws, n))
    R.check_attention(alone, ref, c.dt)


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_many_groups(hyb, devstatus, dt, D):
    """More groups than a warp has lanes, some empty, and rows of none between them."""
    groups = [(10 + 13 * g, [1 + g % 5] * (g % 4)) for g in range(150)]
    Case(hyb, groups, 2, 2, D, dt, seed=1).check()
    Case(hyb, groups, 2, 2, D, dt, seed=1, empty_groups=True, extra_rows=3).check()
    assert devstatus() == (0, 0)


def test_groups_of_one_in_thousands(hyb, devstatus):
    """A search among more than 32 x 32 groups, rows before, between and behind them."""
    g = torch.Generator().manual_seed(3)
    groups = [(int(p), [int(t)] if keep else []) for p, t, keep in zip(torch.randint(0, 40, (2500,), generator=g), torch.randint(1, 20, (2500,), generator=g), torch.rand(2500, generator=g) < 0.7)]
    c = Case(hyb, groups, 1, 1, 64, seed=4, extra_rows=5)
    c.check()
    # the first rows are nobody's either
    for i in range(3):
        c.cu[i] = c.cu[3]
    c.dev[1].copy_(torch.tensor(c.cu, dtype=torch.int32))
    c.out.fill_(7)
    c.check()
    assert devstatus() == (0, 0) and c.cu[0] > 0


def test_a_table_of_more_tokens_than_an_integer_counts(hyb, devstatus):
    c = Case(hyb, [(300, [70])], 2, 1, 128, bs=256, seed=2)
    wide = torch.full((1, 1 << 23), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.bt.shape[1]] = c.bt
    c.bt = wide
    c.d.max_blocks_per_seq = 1 << 23
    c.check()
    assert devstatus() == (0, 0)


def test_bad_groups_and_lengths_are_flagged_and_left(hyb, devstatus):
    groups = [(40, [3, 4]), (50, [1, 2, 9]), (30, [5]), (64, [2, 8])]
    for what, edit in {
        "more rows than the bound": lambda c: setattr(c, "p", hyb.prefix_dims(4, 4, 2, 64, 9)),
        "a prefix above the bound": lambda c: setattr(c, "p", hyb.prefix_dims(4, 4, 3, 49, 9)),
        "a negative prefix": lambda c: c.dev[2].__setitem__(1, -1),
        "rows behind the batch": lambda c: c.dev[1].__setitem__(4, 9),
        "rows before the batch": lambda c: c.dev[1].__setitem__(0, -1),
    }.items():
        c = Case(hyb, groups, 4, 2, 128, seed=5)
        edit(c)
        c.n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(c.B, c.p, c.d)
        c.ws = torch.full((c.n // 4 + 4,), math.nan, device="cuda")
        hyb.check(c.call())
        assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH), what
        ref = list(c.ref())
        gone = {"more rows than the bound": [2, 3, 4], "a prefix above the bound": [2, 3, 4, 6, 7], "a negative prefix": [2, 3, 4], "rows behind the batch": [6, 7], "rows before the batch": [0, 1]}[what]
        ref[0][gone] = math.nan
        R.check_attention(c.out, ref, c.dt, what)
        assert (c.out[gone] == 7).all(), what
    # requests longer than the bound, and longer than the table
    c = Case(hyb, groups, 4, 2, 128, seed=5)
    c.p = hyb.prefix_dims(4, 4, 3, 64, 8)
    c.n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(c.B, c.p, c.d)
    hyb.check(c.call())
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)
    ref = list(c.ref())
    ref[0][4] = math.nan
    R.check_attention(c.out, ref, c.dt)
    assert (c.out[4] == 7).all()
    # a negative length is no key
    for n in (-3, -2 ** 31):
        c = Case(hyb, groups, 4, 2, 128, seed=5)
        c.dev[0][1] = n
        hyb.check(c.call())
        assert (c.out[1] == 0).all() and devstatus() == (0, 0)
    for n in (2 ** 31 - 1, 1 << 20):
        c.dev[0][1] = n
        c.out.fill_(7)
        hyb.check(c.call())
        assert (c.out[1] == 7).all() and devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_bad_blocks_are_flagged_and_left_out(hyb, devstatus, dt, D):
    c = Case(hyb, [(200, [30, 5, 70]), (0, [40])], 4, 2, D, dt, seed=6)
    c.bt[0, 3] = c.NB                      # in the prefix
    c.bt[2, 14] = -1                       # in a row's own part
    c.bt[3, :] = -7                        # all of a row
    hyb.check(c.call())
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_BLOCK)
    c.bt[0, 3] = -1
    R.check_attention(c.out, c.ref(), dt)
    assert (c.out[3] == 0).all()


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_non_finite_values_stay_in_their_request(hyb, dt, D):
    c = Case(hyb, [(150, [30, 5, 70, 3])], 4, 2, D, dt, seed=7)
    clean = c.check().clone()
    c.q[1, 2, 5] = math.nan
    c.vc[c.bt[2, 10].long(), 0, 3, 7] = math.inf
    hyb.check(c.call())
    assert c.out[1, 2].isnan().all() and torch.equal(c.out[1, [0, 1, 3]], clean[1, [0, 1, 3]])
    assert not c.out[2, :2, 7].isfinite().any()
    assert torch.equal(c.out[[0, 3]], clean[[0, 3]]) and torch.equal(c.out[2, 2:], clean[2, 2:])


def test_far_end_of_a_large_pool(hyb, devstatus):
    """Element offsets beyond 2^32."""
    c = Case(hyb, [(300, [20, 3, 90])], 4, 2, 128, bs=128, seed=8, spread=(1 << 32) // (2 * 128 * 128) + 50)
    assert c.NB * 2 * 128 * 128 > 1 << 32 and int(c.bt.max()) == c.NB - 1
    c.check()
    assert devstatus() == (0, 0)


def test_replayed_in_a_graph_and_on_two_streams(hyb, devstatus):
    c = Case(hyb, [(900, [30, 5, 70, 1]), (64, [3, 200])], 8, 2, 128, seed=10, slack=30)
    first = c.check().clone()
    hyb.check(c.call())
    assert torch.equal(c.out, first)                       # equal calls, equal bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hyb.check(c.call())
    c.q.copy_(c.q.flip(0))                                 # other inputs, and one token more in places
    c.dev[0][1] -= 2
    c.lens[1] -= 2
    c.out.fill_(7)
    graph.replay()
    R.check_attention(c.out, c.ref(), c.dt)
    want = c.out.clone()
    outs = [torch.empty_like(c.out) for _ in range(2)]
    spaces = [torch.empty_like(c.ws) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w in zip(streams, outs, spaces):
            hyb.check(c.call(o, w, s))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and devstatus() == (0, 0)
