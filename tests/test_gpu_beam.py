"""Beam selection and reordering against their plain forms, and a whole beam search of a hybrid
model's layers."""
import math

import pytest
import torch

import beam_ref as R

pytestmark = pytest.mark.gpu

INF = math.inf


def run_select(hyb, logits, scores, N, finished=None, eos=-1, stride=0, ws=None):
    """logits [R][W][V] on the GPU."""
    Rn, W, V = logits.shape
    d = hyb.beam_dims(W, N, V, logits.dtype, eos_token=eos, row_stride=stride)
    n = hyb.hyb_beam_select_workspace_size(Rn, d)
    ws = torch.full((n // 4 + 4,), math.nan, device="cuda") if ws is None else ws
    outs = torch.full((Rn, N), 7.0, device="cuda"), torch.full((Rn, N), 7, device="cuda", dtype=torch.int32), torch.full((Rn, N), 7, device="cuda", dtype=torch.int32), \
        torch.full((Rn, N), 7, device="cuda", dtype=torch.uint8)
    if stride:
        rows = torch.full((Rn * W, stride), INF, device="cuda", dtype=logits.dtype)       # the padding is nobody's
        rows[:, :V] = logits.view(Rn * W, V)
        x = rows[:, :V]
    else:
        x = logits.contiguous()
    hyb.check(hyb.hyb_beam_select(*outs, x, scores, finished, Rn, d, ws, n))
    return outs


def both(hyb, logits, scores, N, finished=None, eos=-1, stride=0, what=""):
    got = run_select(hyb, logits, scores, N, finished, eos, stride)
    ref = R.select(logits, scores.cpu(), None if finished is None else finished.cpu(), eos, N)
    R.check_select(got, ref, what)
    return got


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Rn,W,N,V", [(1, 1, 1, 1), (1, 1, 1, 2), (2, 3, 6, 2), (1, 4, 8, 1000), (3, 5, 10, 50021), (2, 128, 128, 257), (5, 2, 4, 4097), (1, 1, 128, 128),
                                      (1, 8, 16, 262145), (70, 4, 4, 8191), (2, 16, 32, 31999), (300, 1, 2, 300)])
def test_shapes(hyb, devstatus, Rn, W, N, V, dt):
    x = (3 * rnd(V + N, Rn, W, V)).to(dt)
    s = -4 * rnd(N, Rn, W).abs()
    both(hyb, x, s, N)
    both(hyb, x, s, N, stride=V + 1 + V % 5)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["constant", "few values", "rising", "falling", "one block", "zeros of both signs", "equal beams", "large", "far apart"])
@pytest.mark.parametrize("N", [4, 100])
def test_orders_and_ties(hyb, kind, N, dt):
    Rn, W, V = 2, 4, 70001
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
    elif kind == "one block":                        # the best all side by side
        x = torch.where((at >= 40000) & (at < 40200), 8 + x, x)
    elif kind == "zeros of both signs":
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "equal beams":
        x, s = x[:, :1].expand(Rn, W, V), s[:, :1].expand(Rn, W).contiguous()
    elif kind == "large":
        x = x * 1e30
    else:
        x = x * 100
    both(hyb, x.to(dt), s, N, what=kind)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", [0.5, 0.999, 1.0])
def test_banned_tokens(hyb, devstatus, masked, dt):
    """Beams with few candidates or none."""
    Rn, W, V, N = 3, 4, 5000, 16
    x = rnd(7, Rn, W, V).to(dt)
    x[torch.rand(Rn, W, V, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < masked] = -INF
    x[0, 1] = -INF
    x[0, 1, 4999] = 3
    both(hyb, x, -rnd(8, Rn, W).abs(), N)
    x[1] = -INF
    got = both(hyb, x, -rnd(8, Rn, W).abs(), N)
    assert (got[1][1] == -1).all() and devstatus() == (0, 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_finished_and_unborn_beams(hyb, devstatus, dt):
    Rn, W, V, N = 4, 5, 3001, 10
    x = rnd(9, Rn, W, V).to(dt)
    s = -rnd(10, Rn, W).abs()
    fin = torch.zeros(Rn, W, dtype=torch.uint8, device="cuda")
    fin[0, 2] = fin[1, :] = fin[3, 0] = 1
    s[2, 1:] = -INF                                 # a request's first step
    s[3, :] = -INF
    x[0, 2] = math.nan                              # logits that are not read
    x[2, 3] = INF
    x[0, 4, 17] = 20                                # a beam that ends
    got = both(hyb, x, s, N, finished=fin, eos=17)
    assert got[3][0].sum() >= 2 and (got[1][2] == 0).all() and (got[1][3] == -1).all()
    # one finished and unborn: none
    assert devstatus() == (0, 0)
    both(hyb, x, s, 5, finished=fin, eos=0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.nan, INF])
def test_bad_values_are_flagged(hyb, devstatus, bad, dt):
    x = rnd(11, 2, 3, 9000).to(dt)
    s = -rnd(12, 2, 3).abs()
    x[0, 1, 8999] = bad
    both(hyb, x, s, 6)
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_VALUE)
    x[0, 1, 8999] = 0
    s[1, 2] = bad
    both(hyb, x, s, 6)
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_VALUE)


def test_select_in_place_in_a_graph_and_on_two_streams(hyb, devstatus):
    Rn, W, V = 6, 4, 20000
    x = rnd(13, Rn, W, V)
    s0 = -rnd(14, Rn, W).abs()
    f0 = torch.zeros(Rn, W, dtype=torch.uint8, device="cuda")
    f0[3, 1] = 1
    want = run_select(hyb, x, s0, W, f0, 5)
    d = hyb.beam_dims(W, W, V, eos_token=5)
    n = hyb.hyb_beam_select_workspace_size(Rn, d)
    s, f = s0.clone(), f0.clone()
    par, tok = (torch.empty(Rn, W, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hyb.check(hyb.hyb_beam_select(s, par, tok, f, x, s, f, Rn, d, ws, n))
    graph.replay()
    for g, w in zip((s, par, tok, f), want):
        assert torch.equal(g, w)
    x.copy_(x.flip(1))
    s.copy_(s0)
    f.copy_(f0)
    graph.replay()
    R.check_select((s, par, tok, f), R.select(x, s0.cpu(), f0.cpu(), 5, W))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                res.append(run_select(hyb, x, s0, W, f0, 5))
    torch.cuda.synchronize()
    for r in res:
        assert torch.equal(r[0], res[0][0]) and torch.equal(r[1], par) and torch.equal(r[2], tok)
    assert devstatus() == (0, 0)


# ----------------------------------------------------------------------------- reordering
FULL, LINEAR, SLIDING = 0, 1, 2


class Stack:
    def __init__(self, hyb, types, Rn, W, P, most, H=2, D=64, dt=torch.bfloat16, bs=16, state=1024, window=40, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hyb, self.types, self.Rn, self.W, self.bs, self.state, self.window, self.most = hyb, types, Rn, W, bs, state, window, most
        B = Rn * W
        self.P = P if isinstance(P, list) else [P] * Rn
        cols = (max(self.P) + most + bs - 1) // bs + 2
        rows, ids = [], 0
        for r in range(Rn):
            common = list(range(ids, ids + self.P[r] // bs))
            ids += len(common)
            for _ in range(W):
                rows.append(common + list(range(ids, ids + cols - len(common))))
                ids += cols - len(common)
        self.NB = ids + 1
        where = torch.randperm(self.NB, generator=gen, device="cuda").to(torch.int32)
        self.bt = where[torch.tensor(rows, device="cuda")].contiguous()
        self.lens = [self.P[b // W] + int(x) for b, x in enumerate(torch.randint(0, most + 1, (B,), generator=gen, device="cuda").tolist())]
        self.lens[0] = self.P[0] + most
        self.NS = B + 3
        self.slots = torch.randperm(self.NS, generator=gen, device="cuda")[:B].to(torch.int32)
        self.io, self.pools = [], []
        for t in types:
            if t == LINEAR:
                x = torch.randn(self.NS, state, generator=gen, device="cuda")
                self.pools.append((x,))
                self.io.append(hyb.layer_io(state_pool=x, num_state_slots=self.NS))
            else:
                kv = tuple(torch.randn(self.NB, H, bs, D, generator=gen, device="cuda").to(dt) for _ in range(2))
                self.pools.append(kv)
                self.io.append(hyb.layer_io(k_cache=kv[0], v_cache=kv[1], window=window if t == SLIDING else 0))
        self.d = hyb.dims(H, D, self.NB, cols, dt, block_size=bs)
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.pre_d = torch.tensor(self.P, dtype=torch.int32, device="cuda")
        self.ws = torch.full((hyb.hyb_beam_reorder_workspace_size(Rn, W),), 255, dtype=torch.uint8, device="cuda")

    def call(self, parents, **kw):
        a = dict(bt=self.bt, lens=self.lens_d, pre=self.pre_d, slots=self.slots, most=self.most)
        a.update(kw)
        return self.hyb.hyb_beam_reorder(parents, a["bt"], a["lens"], a["pre"], a["slots"], self.types, len(self.types), self.io, self.Rn, self.W, a["most"], self.state,
                                         self.d, self.ws, self.ws.numel())

    def expect(self, parents):
        """What the tables, lengths, slots and pools are to be, from the present ones."""
        W, bs = self.W, self.bs
        bt, slots, lens = self.bt.cpu(), self.slots.cpu(), self.lens_d.cpu()
        nbt, nslots, nlens = bt.clone(), slots.clone(), lens.clone()
        pools = [tuple(x.clone() for x in p) for p in self.pools]
        for r in range(self.Rn):
            rows, copy = R.seats([p if -1 <= p < W else -1 for p in parents[r]])
            for i in range(W):
                b, old, par = r * W + i, r * W + rows[i], parents[r][i]
                nbt[b], nslots[b] = bt[old], slots[old]
                nlens[b] = lens[r * W + par] if 0 <= par < W else lens[old]
                if copy[i] is None:
                    continue
                src = r * W + copy[i]
                n = int(lens[src])
                for t, p in zip(self.types, pools):
                    if t == LINEAR:
                        p[0][int(slots[old])] = p[0][int(slots[src])]
                        continue
                    lo = max(self.P[r], n + 1 - self.window) if t == SLIDING else self.P[r]
                    for x in p:
                        at = torch.arange(lo, max(lo, n))
                        s, q = bt[src, at // bs].long().cuda(), bt[old, at // bs].long().cuda()
                        x[q, :, (at % bs).cuda()] = x[s, :, (at % bs).cuda()]
        return nbt, nlens, nslots, pools

    def check(self, parents, want=None):
        nbt, nlens, nslots, pools = want or self.expect(parents)
        assert torch.equal(self.lens_d.cpu(), nlens) and torch.equal(self.slots.cpu(), nslots) and torch.equal(self.bt.cpu(), nbt)
        for p, x in zip(self.pools, pools):
            for a, b in zip(p, x):
                assert torch.equal(a, b)


def parents_of(Rn, W, seed, kind="random"):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, W, (Rn, W), generator=g)
    if kind == "same":
        p[:] = W - 1
    elif kind == "keep":
        p[:] = torch.arange(W)
    elif kind == "turn":
        p[:] = torch.arange(W).roll(1)
    elif kind == "none":
        p[torch.rand(Rn, W, generator=g) < 0.4] = -1
    return p.tolist()


def on_gpu(p):
    return torch.tensor(p, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["random", "same", "keep", "turn", "none"])
@pytest.mark.parametrize("Rn,W", [(1, 1), (1, 4), (5, 3), (3, 16), (2, 128)])
def test_reorder_parents(hyb, devstatus, Rn, W, kind):
    p = parents_of(Rn, W, W, kind)
    s = Stack(hyb, [FULL, LINEAR, SLIDING], Rn, W, 37, 50, seed=W)
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p)))
    s.check(p, want)
    want = s.expect(p)                               # and again from there
    hyb.check(s.call(on_gpu(p)))
    s.check(p, want)
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,P,most,H,D", [(16, 0, 1, 1, 16), (16, 16, 33, 3, 128), (32, 31, 100, 2, 64), (256, 300, 700, 1, 256), (64, [0, 5, 64, 63], 129, 8, 32)])
def test_reorder_sizes(hyb, devstatus, bs, P, most, H, D, dt):
    s = Stack(hyb, [FULL, SLIDING, FULL], 4, 5, P, most, H, D, dt, bs, window=17, seed=most)
    p = parents_of(4, 5, most)
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p), slots=None))
    s.check(p, (want[0], want[1], s.slots.cpu(), want[3]))
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("state", [4, 256, 4100, 32 * 128 * 128])
def test_reorder_states_alone(hyb, devstatus, state):
    s = Stack(hyb, [LINEAR] * 3, 3, 4, 0, 4, state=state, seed=state)
    p = parents_of(3, 4, 1)
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p), bt=None, lens=None, pre=None))
    s.check(p, (s.bt.cpu(), s.lens_d.cpu(), want[2], want[3]))
    assert devstatus() == (0, 0)


def test_reorder_many_layers_and_none(hyb, devstatus):
    """More layers than one launch takes; and no layer: tables, lengths and slots move all the same."""
    s = Stack(hyb, [LINEAR, FULL] * 130, 2, 4, 5, 20, 1, 16, state=64, seed=2)
    p = parents_of(2, 4, 3, "same")
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p)))
    s.check(p, want)
    s.types, s.io, s.pools = [], [], []
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p)))
    s.check(p, want)
    assert devstatus() == (0, 0)


def test_reorder_bad_values_are_flagged_and_left_out(hyb, devstatus):
    err = hyb.HYB_ERR_DEVICE_CHECK
    s = Stack(hyb, [FULL, LINEAR], 2, 3, 20, 30, seed=4)
    p = [[0, 3, 0], [-2, 1, 1]]                      # 3 and -2 are no beams
    want = s.expect(p)
    hyb.check(s.call(on_gpu(p)))
    assert devstatus() == (err, hyb.HYB_DEVERR_BAD_VALUE)
    s.check(p, want)
    # a slot outside the pool, a block outside the pool, a parent longer than the bound
    s = Stack(hyb, [FULL, LINEAR], 2, 3, 20, 30, seed=4)
    p = [[0, 0, 2], [1, 1, 1]]
    want = s.expect(p)
    s.slots[1] = s.NS
    before = s.pools[1][0].clone()
    hyb.check(s.call(on_gpu(p)))
    assert devstatus() == (err, hyb.HYB_DEVERR_BAD_STATE)
    changed = (s.pools[1][0] != before).any(-1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted(s.slots[[4, 5]].tolist())
    s = Stack(hyb, [FULL], 2, 3, 20, 30, seed=4)
    last = (s.lens[0] - 1) // 16
    s.bt[1, last] = s.NB
    before = [x.clone() for x in s.pools[0]]
    hyb.check(s.call(on_gpu(p), slots=None))
    assert devstatus() == (err, hyb.HYB_DEVERR_BAD_BLOCK)
    s = Stack(hyb, [FULL], 2, 3, 20, 30, seed=4)
    before = [x.clone() for x in s.pools[0]]
    lens = s.lens_d.clone()
    hyb.check(s.call(on_gpu([[0, 0, 0], [0, 1, 2]]), slots=None, most=29))
    assert devstatus() == (err, hyb.HYB_DEVERR_BAD_LENGTH)
    assert all(torch.equal(a, b) for a, b in zip(before, s.pools[0])) and (s.lens_d[:3] == lens[0]).all()


@pytest.mark.parametrize("types", [[LINEAR, FULL], [LINEAR, LINEAR, SLIDING], [FULL, LINEAR], ([LINEAR] + [FULL] * 95) * 2])
def test_reorder_flags_a_long_parent_in_any_layer(hyb, devstatus, types):
    """A parent longer than the bound, or than its table, is flagged wherever a launch's Full layers stand."""
    for most, n in ((29, 50), (30, 16 * 40)):
        s = Stack(hyb, types, 2, 3, 20, 30, 1, 16, state=64, seed=4)
        s.lens_d[0] = n
        p = [[0, 0, 0], [0, 1, 2]]
        lens = s.lens_d.clone()
        before = [[x.clone() for x in pool] for pool, t in zip(s.pools, types) if t != LINEAR]
        hyb.check(s.call(on_gpu(p), most=most))
        assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)
        after = [pool for pool, t in zip(s.pools, types) if t != LINEAR]
        assert all(torch.equal(a, b) for x, y in zip(before, after) for a, b in zip(x, y))
        assert (s.lens_d[:3] == n).all() and torch.equal(s.lens_d[3:], lens[3:])


def test_reorder_of_odd_lengths_copies_nothing(hyb, devstatus):
    """A parent without tokens behind the prefix, shorter than it, or of a length below zero."""
    for n in (20, 7, 0, -1, -2 ** 31):
        s = Stack(hyb, [FULL, SLIDING], 1, 3, 20, 30, seed=4)
        s.lens_d[0] = n
        before = [x.clone() for p in s.pools for x in p]
        hyb.check(s.call(on_gpu([[0, 0, 0]]), slots=None))
        assert s.lens_d.tolist() == [n] * 3 and all(torch.equal(a, b) for a, b in zip(before, [x for p in s.pools for x in p]))
    assert devstatus() == (0, 0)


def test_reorder_in_a_graph(hyb, devstatus):
    s = Stack(hyb, [FULL, LINEAR], 3, 4, 18, 60, seed=6)
    p = on_gpu(parents_of(3, 4, 0, "keep"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hyb.check(s.call(p))
    for seed in range(4):
        q = parents_of(3, 4, seed)
        p.copy_(on_gpu(q))
        want = s.expect(q)
        graph.replay()
        s.check(q, want)
    assert devstatus() == (0, 0)


# ------------------------------------------------------------------------- a beam search
def test_beam_search_of_a_hybrid_model(hyb, devstatus):
    """A Full and a gated Linear layer on R prompts of W beams: prompt, then steps of append,
    shared-prefix attention, delta step, selection and reordering, the later ones replayed from one
    captured graph. Each step's outputs are checked against 64-bit attention and recurrence over each beam's own history."""
    import layer_ops_ref as L
    Rn, W, H, D, V, bs, steps = 2, 4, 4, 128, 997, 16, 9
    prompts, B = [70, 33], 8
    gen = torch.Generator(device="cuda").manual_seed(20)

    def rn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    # token -> rows of q, k, v, gate and strength; outputs -> logits
    emb = (rn(V, 3 * H * D)).bfloat16()
    gates, betas = -0.2 * torch.rand(V, H, generator=gen, device="cuda"), torch.rand(V, H, generator=gen, device="cuda")
    head = (0.3 * rn(2 * H * D, V)).float()
    d = hyb.dims(H, D, 200, 16, block_size=bs)
    stride = 3 * H * D
    dd = hyb.delta_dims(H, H, D, qk_norm_eps=1e-6, q_stride=stride, k_stride=stride, v_stride=stride)
    kc, vc = (torch.full((200, H, bs, D), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    states = torch.zeros(B + 1, H, D, D, device="cuda")
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    where = torch.randperm(200, generator=gen, device="cuda").to(torch.int32)
    bt, at = torch.full((B, 16), -1, dtype=torch.int32, device="cuda"), 0
    tokens_in = [torch.randint(0, V, (n,), generator=gen, device="cuda") for n in prompts]
    for r, n in enumerate(prompts):                 # the prompt, once for the request and its last block for every beam
        whole = n // bs
        for w in range(W):
            bt[r * W + w, :whole] = where[at:at + whole]
        at += whole
        for w in range(W):
            bt[r * W + w, whole:8] = where[at:at + 8 - whole]
            at += 8 - whole
            rows = emb[tokens_in[r]].view(n, 3, H, D)
            pos = torch.arange(n, device="cuda")
            for c, x in ((kc, rows[:, 1]), (vc, rows[:, 2])):
                c[bt[r * W + w, pos // bs].long(), :, pos % bs] = x
    for r, n in enumerate(prompts):                 # its state, the same for every beam
        rows = emb[tokens_in[r]]
        q, k, v = (x.unflatten(1, (H, D)) for x in rows.split(H * D, dim=1))
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ws = torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(1, n, dd), dtype=torch.uint8, device="cuda")
        hyb.check(hyb.hyb_gated_delta_chunked_prefill(torch.empty(n, H, D, device="cuda", dtype=torch.bfloat16), q, k, v, gates[tokens_in[r]], betas[tokens_in[r]], cu, states, B + 1,
                                                      slots[r * W:], torch.ones(1, dtype=torch.uint8, device="cuda"), 1, n, n, dd, ws, ws.numel()))
        states[slots[r * W + 1:(r + 1) * W].long()] = states[slots[r * W].long()].clone()
    lens = torch.tensor([n for n in prompts for _ in range(W)], dtype=torch.int32, device="cuda")
    pre = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, W, 2 * W], dtype=torch.int32, device="cuda")
    step_cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    last = torch.randint(0, V, (B,), generator=gen, device="cuda")          # the first step's tokens: another one for each beam
    scores = torch.tensor([[0.0] + [-INF] * (W - 1)] * Rn, device="cuda")
    fin = torch.zeros(Rn, W, dtype=torch.uint8, device="cuda")
    eos = 11
    par, tok = (torch.empty(Rn, W, dtype=torch.int32, device="cuda") for _ in range(2))
    p = hyb.prefix_dims(H, Rn, W, max(prompts), steps)
    sd = hyb.beam_dims(W, W, V, eos_token=eos)
    sizes = [hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(B, p, d), hyb.hyb_beam_select_workspace_size(Rn, sd), hyb.hyb_beam_reorder_workspace_size(Rn, W)]
    w1, w2, w3 = (torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for n in sizes)
    io = [hyb.layer_io(k_cache=kc, v_cache=vc), hyb.layer_io(state_pool=states, num_state_slots=B + 1)]
    att, lin = (torch.empty(B, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sm = torch.empty(B, dtype=torch.int64, device="cuda")
    logits = torch.empty(B, V, device="cuda")

    def step():
        rows = emb[last]
        q, k, v = (x.unflatten(1, (H, D)) for x in rows.split(H * D, dim=1))
        hyb.check(hyb.hyb_slot_mapping(sm, bt, step_cu, lens, B, B, d))
        hyb.check(hyb.hyb_paged_kv_append(k.contiguous(), v.contiguous(), sm, B, kc, vc, d))
        lens.add_(1)
        hyb.check(hyb.hyb_paged_attn_decode_shared_prefix(att, q.contiguous(), kc, vc, bt, lens, cu, pre, B, p, d, w1, w1.numel()))
        hyb.check(hyb.hyb_gated_delta_step(lin, q, k, v, gates[last], betas[last], states, B + 1, slots, B, dd))
        torch.mm(torch.cat([att, lin], 1).flatten(1).float(), head, out=logits)
        s_in.copy_(scores)
        f_in.copy_(fin)
        hyb.check(hyb.hyb_beam_select(scores, par, tok, fin, logits, scores, fin, Rn, sd, w2, w2.numel()))
        hyb.check(hyb.hyb_beam_reorder(par, bt, lens, pre, slots, [FULL, LINEAR], 2, io, Rn, W, steps, H * D * D, d, w3, w3.numel()))
        last.copy_(tok.flatten().clamp(min=0))

    s_in, f_in = torch.empty_like(scores), torch.empty_like(fin)
    history = [[tokens_in[b // W].tolist(), []] for b in range(B)]           # prompt, answer
    graph = None
    for n in range(steps):
        fed = last.tolist()
        if n < 2:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            history[b] = [history[b][0], history[b][1] + [fed[b]]]
            seq = torch.tensor(history[b][0] + history[b][1], device="cuda")
            q, k, v = (x.unflatten(1, (H, D)) for x in emb[seq].double().split(H * D, dim=1))
            s = torch.einsum("hd,phd->hp", q[-1], k) * D ** -0.5
            w = torch.softmax(s, -1)
            out, mag = torch.einsum("hp,phd->hd", w, v), torch.einsum("hp,phd->hd", w, v.abs())
            a = (torch.einsum("hd,phd->hp", q[-1].abs(), k.abs()) * D ** -0.5).amax(-1, keepdim=True)
            R.check_attention(att[b:b + 1], (out[None], mag[None], a[None], torch.full((1, 1, 1), float(len(seq)), device="cuda")), torch.bfloat16, f"attention of beam {b}, step {n}")
            h = [x.double().cpu().numpy() for x in (q, k, v, gates[seq], betas[seq])]
            o, S, m, norm = L.delta_rule(*h, torch.zeros(H, D, D).numpy(), D ** -0.5, 1e-6)
            L.check_out(lin[b:b + 1].double().cpu().numpy(), o[-1:], m[-1:], 2.0 ** -8, len(seq), f"delta rule of beam {b}, step {n}", split=True)
        R.check_select((scores, par, tok, fin), R.select(logits.view(Rn, W, V), s_in.cpu(), f_in.cpu(), eos, W), f"step {n}")
        kept = par.cpu().tolist()
        assert all(x >= 0 for row in kept for x in row)
        history = [history[(b // W) * W + kept[b // W][b % W]] for b in range(B)]
        assert lens.tolist() == [prompts[b // W] + n + 1 for b in range(B)]
        assert sorted(slots.tolist()) == list(range(1, B + 1))
    assert len({tuple(h[1]) for h in history}) > 1 and devstatus() == (0, 0)
