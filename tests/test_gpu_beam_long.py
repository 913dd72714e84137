"""Beam selection where a list runs over and is thinned out, again and again: many kept of many
beams, and rows that a CTA walks in several batches."""
import math

import pytest
import torch

import beam_ref as R

pytestmark = pytest.mark.gpu

INF = math.inf


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def want_of(x, scores, N):
    """R.select of logits [R][W][V] without finished beams, row by row on the GPU (ties: the lowest token first)."""
    Rn, W, V = x.shape
    N0 = min(N, V)
    got = ([], [], [], [])
    for r in range(Rn):
        found = []
        for w in range(W):
            y = x[r, w].double()
            y = y - y.max()
            y = y - y.exp().sum().log()
            v, at = torch.sort(y, descending=True, stable=True)
            found += [(-(float(scores[r, w]) + a), w, b) for a, b in zip(v[:N0].tolist(), at[:N0].tolist()) if a > -INF]
        found = sorted(found)[:N]
        found += [(INF, -1, -1)] * (N - len(found))
        for g, c in zip(got, ([-f[0] for f in found], [f[1] for f in found], [f[2] for f in found], [0] * N)):
            g.append(c)
    return got


class Select:
    def __init__(self, hyb, x, scores, N):
        self.hyb, self.x, self.s, self.R = hyb, x, scores, x.shape[0]
        self.d = hyb.beam_dims(x.shape[1], N, x.shape[2], x.dtype)
        self.n = hyb.hyb_beam_select_workspace_size(self.R, self.d)
        self.ws = torch.full((self.n // 4 + 4,), math.nan, device="cuda")
        # slices of a row, from the workspace's definition
        self.slices = self.n // (8 * (1 + N) * x.shape[0] * x.shape[1])
        self.N = N

    def call(self):
        outs = torch.empty(self.R, self.N, device="cuda"), *(torch.empty(self.R, self.N, device="cuda", dtype=torch.int32) for _ in range(2)), \
            torch.full((self.R, self.N), 7, device="cuda", dtype=torch.uint8)
        self.hyb.check(self.hyb.hyb_beam_select(*outs, self.x, self.s, None, self.R, self.d, self.ws, self.n))
        return outs

    def check(self, what="", again=0):
        got = self.call()
        R.check_select(got, want_of(self.x, self.s.cpu(), self.N), what)
        runs = [self.call() for _ in range(again)]
        for other in runs:
            assert all(torch.equal(a, b) for a, b in zip(got, other)), what
        return got


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Rn,W,N,V", [(1, 16, 32, 200000), (3, 128, 128, 20000), (1, 128, 4, 300), (7, 16, 64, 3001)])
def test_candidates_in_many_rounds(hyb, devstatus, Rn, W, N, V, dt):
    """The candidates of a request run over the list of the second kernel dozens of times; calls repeat bit for bit."""
    x = (3 * rnd(V, Rn, W, V)).to(dt)
    s = -rnd(W, Rn, W).abs()
    c = Select(hyb, x, s, N)
    assert W * c.slices * N >= 512
    c.check(again=50)
    c.s.fill_(-1.5)
    x[:] = x[:, :1].clone()                      # equal beams: every total is there W times
    c.check(again=50)
    assert devstatus() == (0, 0)


# -------------------------------------------------------------- several batches of a slice
def ranked(x, scores, N):
    """Per request the candidates in the exact order, N and those whose totals lie next to the N-th: (total, beam, token).
    Each row's sum is a reduction of its own: within one over all rows the order of the terms, and so the last bit, goes
    by where a row lies, and equal rows would not tie. The maximum is taken off first: beside logits of 1e30 the log of
    a sum is lost in 64 bits too."""
    res = []
    for r in range(x.shape[0]):
        y = x[r].double()
        y = y - y.amax(-1, keepdim=True)
        y = y - torch.stack([row.clone().exp().sum().log() for row in y])[:, None]
        v, at = torch.sort(y, dim=-1, descending=True, stable=True)
        v, at, found = v[:, :N + 8].tolist(), at[:, :N + 8].tolist(), []
        for w, s in enumerate(scores[r].tolist()):
            found += [(-(s + a), w, b) for a, b in zip(v[w], at[w]) if a > -INF]
        res.append([(-t, w, b) for t, w, b in sorted(found)[:N + 8 * len(v)]])
    return res


def check_order(got, ref, N, what=""):
    """The sums over the vocabulary are of 32-bit terms, each total off by 2^-18 at most (beam_ref), the same in all of a
    beam's. So two beams' candidates may change places where their exact totals are nearer than twice that, but not where
    they are equal (equal rows have equal sums), and a beam's own never."""
    lim = 2.0 ** -18
    for scores, parents, tokens, exact in zip(*(t.tolist() for t in got[:3]), ref):
        assert len(exact) >= N
        total = {(w, v): t for t, w, v in exact}
        mine = list(zip(parents, tokens))
        assert len(set(mine)) == N, what
        for i, (pair, s) in enumerate(zip(mine, scores)):
            assert pair in total, (what, i, pair)
            t = total[pair]
            assert abs(s - t) <= lim + R.U * abs(t), (what, i, s, t)
            if pair != exact[i][1:]:
                assert 0 < abs(t - exact[i][0]) <= 2 * lim, (what, i, pair, exact[i])
        for w in set(parents):
            seq = [v for p, v in mine if p == w]
            assert seq == [v for _, p, v in exact if p == w][:len(seq)], (what, w)
    assert (got[3] == 0).all(), what


KINDS = ["random", "constant", "few values", "rising", "falling", "one block", "zeros of both signs", "equal beams", "large", "far apart", "late best"]


def logits_of(kind, Rn, W, V, dt):
    x = rnd(5, Rn, W, V)
    s = -rnd(6, Rn, W).abs()
    at = torch.arange(V, device="cuda")
    if kind == "constant":
        x = torch.full_like(x, -2.5)
    elif kind == "few values":
        x = (x * 1.5).round()
    elif kind == "rising":
        x = (at / V * 9).expand(Rn, W, V)
    elif kind == "falling":
        x = (-at / V * 9).expand(Rn, W, V)
    elif kind == "one block":
        x = torch.where((at >= V // 2) & (at < V // 2 + 200), 8 + x, x)
    elif kind == "zeros of both signs":
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "equal beams":
        x, s = x[:, :1].expand(Rn, W, V), s[:, :1].expand(Rn, W).contiguous()
    elif kind == "large":
        x = x * 1e30
    elif kind == "far apart":
        x = x * 100
    elif kind == "late best":                        # rising steps, each tied over most of a batch
        x = (at // 3000).float().expand(Rn, W, V)
    return x.to(dt).contiguous(), s


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Rn,W,batches", [(19, 4, 2), (38, 3, 3), (76, 4, 8)])
@pytest.mark.parametrize("kind", KINDS)
def test_slices_of_several_batches(hyb, devstatus, kind, Rn, W, batches, dt):
    """Slices of 2, 3 and 8 batches (fp32: twice as many): what one batch leaves bounds the next, lists are carried
    over and thinned out, ties cross batches."""
    V = 130001
    x, s = logits_of(kind, Rn, W, V, dt)
    ref = ranked(x, s, 128)
    for N in (8, 25, 128):
        c = Select(hyb, x, s, N)
        if torch.cuda.get_device_properties(0).multi_processor_count == 152:
            assert c.slices == -(-16 // batches)
        got = c.call()
        check_order(got, ref, N, f"{kind}, {N} kept")
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(got, c.call())), (kind, N)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt,V", [(torch.float32, 1100001), (torch.bfloat16, 2200003)])
@pytest.mark.parametrize("kind", ["random", "constant", "rising", "equal beams"])
def test_more_than_256_slices(hyb, devstatus, kind, dt, V):
    x, s = logits_of(kind, 1, 2, V, dt)
    ref = ranked(x, s, 128)
    for N in (4, 128):
        c = Select(hyb, x, s, N)
        assert c.slices > 256
        check_order(c.call(), ref, N, f"{kind}, {N} kept")
    assert devstatus() == (0, 0)


def test_the_largest_vocabulary(hyb, devstatus):
    """Two beams of 2^30 - 1 tokens, the second row off the 16-byte boundary: all equal but a few."""
    V, N = (1 << 30) - 1, 6
    x = torch.zeros(2, V, device="cuda", dtype=torch.bfloat16)
    x[0, 12345], x[0, V - 1], x[1, V - 1], x[1, V - 2] = 5.0, 4.0, 4.5, 4.5
    c = Select(hyb, x.view(1, 2, V), torch.tensor([[-1.0, -1.25]], device="cuda"), N)
    got = c.call()
    base = [-1 - math.log(V - 2 + math.exp(5) + math.exp(4)), -1.25 - math.log(V - 2 + 2 * math.exp(4.5))]
    want = [(0, 12345, 5.0), (1, V - 2, 4.5), (1, V - 1, 4.5), (0, V - 1, 4.0), (0, 0, 0.0), (0, 1, 0.0)]
    assert got[1][0].tolist() == [p for p, _, _ in want] and got[2][0].tolist() == [v for _, v, _ in want]
    for g, (p, _, y) in zip(got[0][0].tolist(), want):
        assert abs(g - (base[p] + y)) <= 2.0 ** -18 + R.U * abs(base[p] + y)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["none before the end", "few here and there", "masked by the lowest value", "all masked by the lowest value"])
def test_masks_over_several_batches(hyb, devstatus, kind, dt):
    """Slices whose first batches hold nothing, or less than is kept."""
    Rn, W, V = 76, 4, 130001
    x, s = logits_of("random", Rn, W, V, dt)
    if kind == "none before the end":
        x[:, :, :V - 300] = -INF
        x[3] = -INF
        x[3, 2, V - 1] = 1.0
    elif kind == "few here and there":
        keep = torch.rand(V, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") < 2e-3
        x[:, :, ~keep] = -INF
    else:
        x[:, :, 100:] = torch.finfo(dt).min
        if kind == "all masked by the lowest value":
            x[:] = torch.finfo(dt).min
    for N in (8, 128):
        c = Select(hyb, x, s, N)
        got = c.call()
        if kind == "none before the end":            # request 3 has one candidate
            assert got[1][3].tolist() == [2] + [-1] * (N - 1) and got[2][3].tolist() == [V - 1] + [-1] * (N - 1) and (got[0][3, 1:] == -INF).all()
            got, x2, s2 = tuple(t[4:] for t in got), x[4:], s[4:]
        else:
            x2, s2 = x, s
        check_order(got, ranked(x2, s2, N), N, f"{kind}, {N} kept")
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.nan, INF])
def test_bad_values_in_a_late_batch(hyb, devstatus, bad, dt):
    Rn, W, V, N = 76, 4, 130001, 8
    x, s = logits_of("random", Rn, W, V, dt)
    c = Select(hyb, x, s, N)
    clean = [t.clone() for t in c.call()]
    x[5, 2, 60000] = x[70, 0, V - 1] = bad
    got = c.call()
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_VALUE)
    assert not (got[1][5] == 2).any() and not (got[1][70] == 0).any() and (got[1][[5, 70]] >= 0).all()
    rest = [r for r in range(Rn) if r not in (5, 70)]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, clean))
    for r, w in ((5, 2), (70, 0)):
        y = x[r:r + 1, [i for i in range(W) if i != w]]
        ref = ranked(y, s[r:r + 1, [i for i in range(W) if i != w]], N)
        ref = [[(t, p + (p >= w), v) for t, p, v in ref[0]]]
        check_order(tuple(t[r:r + 1] for t in got), ref, N)


def test_a_million_rows(hyb, devstatus):
    Rn, V, N = 1 << 20, 3, 2
    x, s = rnd(1, Rn, 1, V), -rnd(2, Rn, 1).abs()
    c = Select(hyb, x, s, N)
    got = c.call()
    v, at = torch.sort(torch.log_softmax(x[:, 0].double(), -1), dim=-1, descending=True, stable=True)
    want = v[:, :N] + s.double()
    assert (got[1] == 0).all() and torch.equal(got[2].long(), at[:, :N])
    assert ((got[0].double() - want).abs() <= 2.0 ** -18 + R.U * want.abs()).all()
    assert devstatus() == (0, 0)


# ----------------------------------------------------------------------------- reordering
def test_reorders_back_to_back(hyb, devstatus):
    """Each call begins on what the last one left, without the host in between; no prefixes given."""
    from test_gpu_beam import FULL, LINEAR, SLIDING, Stack, on_gpu, parents_of
    for types, pre in (([FULL, LINEAR, SLIDING], True), ([LINEAR, FULL], False)):
        make = lambda: Stack(hyb, types, 5, 6, 37 if pre else 0, 50, seed=8)
        s, t = make(), make()
        kw = {} if pre else {"pre": None}
        par = [parents_of(5, 6, i, ["random", "none", "same"][i % 3]) for i in range(8)]
        dev = [on_gpu(p) for p in par]
        for p in dev:
            hyb.check(s.call(p, **kw))
        for p in par:                                # one at a time, each checked
            want = t.expect(p)
            hyb.check(t.call(on_gpu(p), **kw))
            t.check(p, want)
        assert torch.equal(s.bt, t.bt) and torch.equal(s.lens_d, t.lens_d) and torch.equal(s.slots, t.slots)
        for a, b in zip(s.pools, t.pools):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert devstatus() == (0, 0)


def test_reorder_of_65528_beams(hyb, devstatus):
    from test_gpu_beam import LINEAR, on_gpu, parents_of
    Rn, W = 8191, 8
    B = Rn * W
    p = parents_of(Rn, W, 5, "none")
    pool = torch.arange(4 * B, device="cuda", dtype=torch.float32).view(B, 4)
    slots = torch.randperm(B, device="cuda").to(torch.int32)
    lens = torch.arange(B, device="cuda", dtype=torch.int32)
    old, want = slots.clone(), pool.clone()
    rows, src, dst, wl = [], [], [], []
    for r in range(Rn):
        seat, copy = R.seats(p[r])
        for i in range(W):
            rows.append(r * W + seat[i])
            wl.append(r * W + (p[r][i] if p[r][i] >= 0 else seat[i]))
            if copy[i] is not None:
                src.append(r * W + copy[i])
                dst.append(r * W + seat[i])
    want[old[dst].long()] = pool[old[src].long()]
    hyb.check(hyb.hyb_beam_reorder(on_gpu(p), None, lens, None, slots, [LINEAR], 1, [hyb.layer_io(state_pool=pool, num_state_slots=B)], Rn, W, 0, 4, hyb.dims(1, 16, 1, 1), None, 0))
    assert torch.equal(slots, old[rows]) and torch.equal(pool, want) and lens.tolist() == wl
    assert devstatus() == (0, 0)
