"""The gated delta rule's step and prefill against the 64-bit recurrence, through the C ABI."""
import math

import numpy as np
import pytest
import torch

import layer_ops_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def host(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


class Case:
    """Seeded inputs: rows of `T` tokens in all, a pool of `NS` states, packed or in fused rows."""

    def __init__(self, seed, T, Hk, Hv, D, dt, NS, fused=False, eps=EPS, gate="mixed", kscale=1.0, same_keys=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s):
            return torch.randn(*s, generator=gen, device="cuda")

        self.Hk, self.Hv, self.D, self.dt, self.NS, self.eps, self.T = Hk, Hv, D, dt, NS, eps, T
        width = (2 * Hk + Hv) * D + (16 if fused else 0)       # wider than the three together
        rows = rnd(T, width)
        rows[:, Hk * D:2 * Hk * D] *= kscale
        if same_keys:
            rows[:, Hk * D:2 * Hk * D] = rows[:1, Hk * D:2 * Hk * D]
        rows = rows.to(dt)
        parts = [rows[:, :Hk * D], rows[:, Hk * D:2 * Hk * D], rows[:, 2 * Hk * D:(2 * Hk + Hv) * D]]
        self.q, self.k, self.v = (p.unflatten(1, (-1, D)) for p in parts)
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.stride = width if fused else 0
        u = torch.rand(T, Hv, generator=gen, device="cuda")
        if gate == "mixed":        # head 0 keeps everything, the others fade by up to e^-8 a token
            self.g = -8 * u ** 4 * (torch.arange(Hv, device="cuda") % 3)
        elif gate == "none":
            self.g = torch.zeros(T, Hv, device="cuda")
        elif gate == "steep":      # long runs of nearly nothing kept, then slow ones
            self.g = torch.where((torch.arange(T, device="cuda")[:, None] // 7) % 2 == 0, -40 * u, -1e-3 * u)
        elif gate == "clear":      # now and then the state is cleared
            self.g = torch.where(u < 0.1, torch.full_like(u, -math.inf), -0.1 * u)
        self.beta = torch.rand(T, Hv, generator=gen, device="cuda")
        self.pool = rnd(NS, Hv, D, D) * 0.3
        self.gen = gen

    def dims(self, hyb, scale=None):
        return hyb.delta_dims(self.Hk, self.Hv, self.D, self.dt, scale=scale, qk_norm_eps=self.eps, q_stride=self.stride, k_stride=self.stride, v_stride=self.stride)

    def ref(self, rows, S, scale=None):
        a = [host(x[rows]) for x in (self.q, self.k, self.v, self.g, self.beta)]
        return R.delta_rule(*a, S, self.D ** -0.5 if scale is None else scale, self.eps)


def step(hyb, c, out, slots, B, d=None, stream=None):
    hyb.check(hyb.hyb_gated_delta_step(out, c.q, c.k, c.v, c.g, c.beta, c.pool, c.NS, slots, B, d or c.dims(hyb), stream))


def prefill(hyb, c, out, cu, slots, reset, ws=None, max_len=None, d=None, stream=None, first=0, T=None):
    d = d or c.dims(hyb)
    B = cu.numel() - 1
    T = c.T if T is None else T
    if ws is None:
        ws = torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(B, T, d), dtype=torch.uint8, device="cuda")
    lens = cu[1:] - cu[:-1]
    hyb.check(hyb.hyb_gated_delta_chunked_prefill(out, c.q, c.k, c.v, c.g, c.beta, cu, c.pool, c.NS, slots, reset, B, T,
                                                  int(lens.max()) if max_len is None else max_len, d, ws, ws.numel(), stream))
    return ws


def check_prefill(hyb, c, lens, reset, what, gap=0):
    """Runs requests of `lens` rows (gap rows behind the last) and checks everything."""
    B = len(lens)
    cu_h = np.concatenate([[0], np.cumsum(lens)])
    assert cu_h[-1] + gap == c.T
    cu = torch.tensor(cu_h, dtype=torch.int32, device="cuda")
    slots_h = np.random.RandomState(B).permutation(c.NS)[:B]
    slots = torch.tensor(slots_h, dtype=torch.int32, device="cuda")
    rs = None if reset is None else torch.tensor(reset, dtype=torch.uint8, device="cuda")
    before = host(c.pool)
    out = torch.full((c.T, c.Hv, c.D), 7.0, device="cuda", dtype=c.dt)
    prefill(hyb, c, out, cu, slots, rs)
    torch.cuda.synchronize()
    assert hyb.hyb_device_status(clear=True) == (0, 0)
    got, after = host(out), host(c.pool)
    tc = c.dt == torch.bfloat16 and c.D == 128
    for b in range(B):
        S0 = before[slots_h[b]] * (0 if reset is not None and reset[b] else 1)
        rows = slice(int(cu_h[b]), int(cu_h[b + 1]))
        o, S, mag, norm = c.ref(rows, S0)
        if lens[b] == 0:
            assert np.array_equal(after[slots_h[b]], S0), f"{what}: request {b} without rows"
            continue
        R.check_out(got[rows], o, mag, HALF[c.dt], lens[b], f"{what}: out of request {b}", split=tc)
        R.check_state(after[slots_h[b]], S, norm, lens[b], f"{what}: state of request {b}")
    rest = np.setdiff1d(np.arange(c.NS), slots_h)
    assert np.array_equal(after[rest], before[rest]), f"{what}: other slots"
    assert (got[cu_h[-1]:] == 7.0).all(), f"{what}: rows of no request"


# ------------------------------------------------------------------------------ one token
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hk,Hv,fused,eps", [(3, 3, False, EPS), (2, 6, True, EPS), (1, 2, True, 0.0)])
def test_step(hyb, devstatus, D, dt, Hk, Hv, fused, eps):
    B, NS = 5, 9
    c = Case(D + Hv, B, Hk, Hv, D, dt, NS, fused=fused, eps=eps, kscale=1.0 if eps else D ** -0.5)
    slots_h = [8, 0, 3, 5, 1]
    before = host(c.pool)
    out = torch.empty(B, Hv, D, device="cuda", dtype=dt)
    step(hyb, c, out, torch.tensor(slots_h, dtype=torch.int32, device="cuda"), B)
    after, got = host(c.pool), host(out)
    for b, s in enumerate(slots_h):
        o, S, mag, norm = c.ref(slice(b, b + 1), before[s])
        R.check_out(got[b:b + 1], o, mag, HALF[dt], 1, f"out {b}")
        R.check_state(after[s], S, norm, 1, f"state {b}")
    rest = [i for i in range(NS) if i not in slots_h]
    assert np.array_equal(after[rest], before[rest])
    assert devstatus() == (0, 0)


def test_step_clears_with_infinite_decay(hyb):
    c = Case(3, 2, 2, 2, 128, torch.float32, 2, gate="none")
    c.g[0, 0] = -math.inf
    c.g[1, 1] = -20000.0
    before = host(c.pool)
    out = torch.empty(2, 2, 128, device="cuda")
    step(hyb, c, out, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 2)
    for b in range(2):
        o, S, mag, norm = c.ref(slice(b, b + 1), before[b])
        R.check_out(host(out)[b:b + 1], o, mag, HALF[torch.float32], 1, "out")
        R.check_state(host(c.pool)[b], S, norm, 1, "state")


def test_step_bad_slot_is_flagged_and_skipped(hyb, devstatus):
    c = Case(4, 3, 2, 2, 64, torch.bfloat16, 4)
    before = host(c.pool)
    out = torch.full((3, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    step(hyb, c, out, torch.tensor([4, 2, -1], dtype=torch.int32, device="cuda"), 3)
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_STATE)
    assert (host(out)[[0, 2]] == 7.0).all()
    o, S, mag, norm = c.ref(slice(1, 2), before[2])
    R.check_out(host(out)[1:2], o, mag, HALF[torch.bfloat16], 1, "out")
    assert np.array_equal(host(c.pool)[[0, 1, 3]], before[[0, 1, 3]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gate", [-12.0, -0.75, -0.6, -1e-3])
def test_decay_alone_keeps_its_precision(hyb, D, gate):
    """With beta 0 the state only fades: every element to a few roundings of its own value, after one
    token and after many of the same gate (T tokens: T of them, at most u T in all)."""
    for T in (1, 3, 200):
        c = Case(5, T, 1, 1, D, torch.float32, 1, gate="none")
        c.g.fill_(gate)
        c.beta.zero_()
        g32 = float(c.g[0, 0])
        S0 = host(c.pool)[0, 0]
        out = torch.empty(T, 1, D, device="cuda")
        slots = torch.zeros(1, dtype=torch.int32, device="cuda")
        if T == 1:
            step(hyb, c, out, slots, 1)
        else:
            prefill(hyb, c, out, torch.tensor([0, T], dtype=torch.int32, device="cuda"), slots, None)
        ref = S0 * math.exp(g32 * T)
        live = np.abs(ref) > 1e-30          # below, fp32 itself loses bits
        err = np.abs(host(c.pool)[0, 0] - ref)[live]
        # a token rounds once (half an ulp is at most u of the value) and, in the slow form, e^g - 1 is off
        # by 2 u |e^g - 1| / e^g, in the fast one e^g by 2 u: 4 u T covers both
        assert (err <= 4 * R.U * T * np.abs(ref)[live]).all(), (gate, T, (err / np.abs(ref)[live]).max() / R.U)


# -------------------------------------------------------------------------------- prefill
@pytest.mark.parametrize("D,dt", [(16, torch.float32), (32, torch.bfloat16), (64, torch.float32), (64, torch.bfloat16), (128, torch.float32), (256, torch.bfloat16), (128, torch.bfloat16)])
@pytest.mark.parametrize("lens,reset", [([1], None), ([64, 0, 63, 65, 0], [0, 0, 1, 0, 1]), ([17, 130, 1], None)])
def test_prefill_shapes(hyb, D, dt, lens, reset):
    c = Case(D + len(lens), sum(lens) + 3, 2, 4, D, dt, len(lens) + 2, fused=D != 16)
    check_prefill(hyb, c, lens, reset, f"D {D} {dt}", gap=3)


@pytest.mark.parametrize("lens,reset", [([8, 3, 0, 1], [0, 1, 1, 0]), ([9, 8, 0, 1], [0, 1, 1, 0]), ([8] * 60, None),
                                        ([40], None), ([41, 2], None), ([12] * 32, None), ([12] * 33, None)])
def test_prefill_calls_of_a_few_rows(hyb, lens, reset):
    """At both sides of the bound between the recurrence and the tensor-core kernel."""
    c = Case(23, sum(lens) + 2, 2, 4, 128, torch.bfloat16, len(lens) + 1, fused=True)
    check_prefill(hyb, c, lens, reset, f"{lens[:4]}", gap=2)


@pytest.mark.parametrize("gate", ["none", "mixed", "steep", "clear"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_prefill_gates(hyb, gate, dt):
    lens = [200, 77]
    c = Case(11, sum(lens), 3, 3, 128, dt, 3, gate=gate)
    check_prefill(hyb, c, lens, [1, 0], gate)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kscale,eps", [(128 ** -0.5, 0.0), (1e-3, EPS), (1e3, EPS)])
def test_prefill_key_scales(hyb, dt, kscale, eps):
    c = Case(12, 150, 2, 2, 128, dt, 2, kscale=kscale, eps=eps)
    if eps == 0.0:
        c.beta *= 0.7          # |k|^2 is near 1 but not 1: beta |k|^2 stays below 2
    check_prefill(hyb, c, [150], None, f"keys of {kscale}")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_prefill_same_key_every_token(hyb, dt):
    """The corrections' system is as far from the identity as it gets (all ones below the
    diagonal for beta 1): the value of the key is replaced by each token."""
    c = Case(13, 140, 1, 2, 128, dt, 1, gate="none", same_keys=True)
    c.beta.fill_(1.0)
    check_prefill(hyb, c, [140], None, "one key")


def test_prefill_long_prompt_of_small_changes_does_not_drift(hyb):
    """A state that is kept (no decay) and changed little: rounded to nearest once in 64 rows it is
    off by u sqrt(T / 64) of its norm. Each 64 rows' change is a sum of 12 products cut to 24 bits
    (2 u each) of corrections that 24 such products make: 2 x 36 u of that change's norm at most.
    Were the state itself cut 12 times in 64 rows, towards zero, it would be off by 1.5e-5 here."""
    T, u = 4096, 2.0 ** -24
    c = Case(22, T, 1, 2, 128, torch.bfloat16, 1, gate="none")
    c.beta *= 0.01
    S = host(c.pool)[0]
    out = torch.empty(T, 2, 128, device="cuda", dtype=torch.bfloat16)
    prefill(hyb, c, out, torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), None)
    change, most = np.zeros(2), np.zeros(2)
    for t in range(0, T, 64):
        o, S1, mag, norm = c.ref(slice(t, t + 64), S)
        change += np.sqrt(((S1 - S) ** 2).sum((1, 2)))
        most, S = np.maximum(most, norm), S1
    err = np.sqrt(((host(c.pool)[0] - S) ** 2).sum((1, 2)))
    lim = u * (math.sqrt(T / 64) * most + 72 * change)
    assert (lim < 5e-6 * most).all() and (err <= lim).all(), (err / most, lim / most)


@pytest.mark.parametrize("D,dt", [(16, torch.bfloat16), (32, torch.bfloat16), (64, torch.float32), (64, torch.bfloat16)])
def test_prefill_many_chains_of_small_heads(hyb, D, dt):
    """More chains than the GPU holds at once: the recurrence then keeps 32 rows of a column a lane."""
    lens = [20, 3, 0, 17, 1] * 20
    c = Case(24, sum(lens), 4, 4, D, dt, 100, fused=True)
    check_prefill(hyb, c, lens, None, f"400 chains of {D}")


def test_prefill_many_ragged_chains(hyb):
    """More chains than the GPU has SMs, with empty and short ones: chains are shared out."""
    rs = np.random.RandomState(5)
    lens = [int(n) for n in rs.randint(0, 150, 40)]
    lens[7] = 400
    lens[8] = 0
    c = Case(14, sum(lens), 4, 8, 128, torch.bfloat16, 41)
    check_prefill(hyb, c, lens, [int(x) for x in rs.randint(0, 2, 40)], "320 chains")


@pytest.mark.parametrize("D,dt", [(128, torch.bfloat16), (64, torch.float32)])
def test_prefill_in_parts_then_steps(hyb, D, dt):
    """A prompt cut at odd rows, then decoded token by token, follows the one recurrence."""
    T, cuts = 210, [0, 1, 70, 201]
    c = Case(15, T, 2, 4, D, dt, 2, fused=True)
    S0 = host(c.pool)[1]
    out = torch.empty(T, c.Hv, D, device="cuda", dtype=dt)
    slots = torch.tensor([1], dtype=torch.int32, device="cuda")
    ws = None
    for a, b in zip(cuts, cuts[1:]):
        ws = prefill(hyb, c, out, torch.tensor([a, b], dtype=torch.int32, device="cuda"), slots, None, ws=ws)
    full = (c.q, c.k, c.v, c.g, c.beta)
    for t in range(cuts[-1], T):
        c.q, c.k, c.v, c.g, c.beta = (x[t:t + 1] for x in full)
        step(hyb, c, out[t:t + 1], slots, 1)
    c.q, c.k, c.v, c.g, c.beta = full
    o, S, mag, norm = c.ref(slice(0, T), S0)
    R.check_out(host(out), o, mag, HALF[dt], T, "out", split=dt == torch.bfloat16)
    R.check_state(host(c.pool)[1], S, norm, T, "state")


@pytest.mark.parametrize("D,dt", [(128, torch.bfloat16), (64, torch.float32)])
def test_prefill_bad_requests_are_flagged_and_skipped(hyb, devstatus, D, dt):
    c = Case(16, 100, 2, 2, D, dt, 4)
    before = host(c.pool)
    out = torch.full((100, 2, D), 7.0, device="cuda", dtype=dt)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    d = c.dims(hyb)

    def call(cu, slots, max_len, T):
        cu, slots = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, slots))
        hyb.check(hyb.hyb_gated_delta_chunked_prefill(out, c.q, c.k, c.v, c.g, c.beta, cu, c.pool, 4, slots, None, len(slots), T, max_len, d, ws, 4096))

    call([0, 10, 30], [4, 2], 60, 100)                      # a slot beyond the pool
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_STATE)
    call([-5, 10, 30], [0, 2], 60, 100)                     # rows before the first
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)
    call([30, 90, 80], [0, 1], 60, 80)                      # rows behind the last; a negative count
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)
    call([30, 95], [0], 60, 100)                            # more rows than the bound given
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_LENGTH)
    got, after = host(out), host(c.pool)
    assert np.array_equal(after[[0, 1, 3]], before[[0, 1, 3]])
    assert (got[:10] == 7.0).all() and (got[30:] == 7.0).all()
    S = before[2]
    for _ in range(2):                                      # the good request ran twice
        o, S, mag, norm = c.ref(slice(10, 30), S)
    R.check_out(got[10:30], o, mag, HALF[dt], 40, "out", split=dt == torch.bfloat16)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_prefill_without_rows_resets_and_keeps(hyb, devstatus, dt):
    c = Case(20, 1, 2, 2, 128, dt, 3)
    before = host(c.pool)
    d = c.dims(hyb)
    ws = torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(2, 0, d), dtype=torch.uint8, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    reset = torch.tensor([1, 0], dtype=torch.uint8, device="cuda")
    hyb.check(hyb.hyb_gated_delta_chunked_prefill(None, None, None, None, None, None, cu, c.pool, 3, slots, reset, 2, 0, 0, d, ws, ws.numel()))
    assert devstatus() == (0, 0)
    assert (host(c.pool)[2] == 0).all() and np.array_equal(host(c.pool)[:2], before[:2])


def test_prefill_one_chain_per_sm_and_more(hyb):
    """Chains at and around the number of SMs: the boundary between one chain a CTA and the cut
    work split."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for chains in (sms - 1, sms, sms + 1, 2 * sms + 1):
        lens = [int(n) for n in np.random.RandomState(chains).randint(1, 140, chains)]
        c = Case(chains, sum(lens), 1, 1, 128, torch.bfloat16, chains)
        check_prefill(hyb, c, lens, None, f"{chains} chains")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_prefill_nan_gate_and_growth(hyb, dt):
    """A NaN gate makes its head's state NaN from its row on; a gate above 0 lets it grow."""
    c = Case(21, 100, 1, 2, 128, dt, 1)
    c.g[:, 0] = 0.02
    c.g[70, 1] = math.nan
    S0 = host(c.pool)[0]
    out = torch.empty(100, 2, 128, device="cuda", dtype=dt)
    prefill(hyb, c, out, torch.tensor([0, 100], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), None)
    with np.errstate(invalid="ignore"):
        o, S, mag, norm = c.ref(slice(0, 100), S0)
    R.check_out(host(out)[:, :1], o[:, :1], mag[:, :1], HALF[dt], 100, "head 0", split=dt == torch.bfloat16)
    R.check_state(host(c.pool)[0, :1], S[:1], norm[:1], 100, "head 0")
    assert np.isnan(host(out)[70:, 1]).all() and np.isnan(host(c.pool)[0, 1]).all()
    assert np.isfinite(host(out)[:64, 1]).all()


def test_prefill_nan_stays_in_its_request(hyb):
    c = Case(17, 3 * 70, 2, 2, 128, torch.bfloat16, 3)
    c.v[75, 0, 3] = math.nan
    c.q[80] = math.inf
    c.k[139, 1] = math.nan       # a row of the last, partial chunk
    cu = torch.tensor([0, 70, 140, 210], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    before = host(c.pool)
    out = torch.empty(210, 2, 128, device="cuda", dtype=torch.bfloat16)
    prefill(hyb, c, out, cu, slots, None)
    for b, s in ((0, 2), (2, 1)):
        rows = slice(70 * b, 70 * b + 70)
        o, S, mag, norm = c.ref(rows, before[s])
        R.check_out(host(out)[rows], o, mag, HALF[torch.bfloat16], 70, f"request {b}", split=True)
        R.check_state(host(c.pool)[s], S, norm, 70, f"state {b}")
    assert np.isnan(host(c.pool)[0]).any()


def test_prefill_same_inputs_same_bits(hyb):
    lens = [200, 3, 129, 64] * 12
    c = Case(18, sum(lens), 4, 4, 128, torch.bfloat16, 48)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    slots = torch.arange(48, dtype=torch.int32, device="cuda")
    start = c.pool.clone()
    res = []
    for _ in range(3):
        c.pool.copy_(start)
        out = torch.empty(c.T, 4, 128, device="cuda", dtype=torch.bfloat16)
        prefill(hyb, c, out, cu, slots, None)
        res.append((out.clone(), c.pool.clone()))
    assert all(torch.equal(a, b) for r in res[1:] for a, b in zip(res[0], r))
    # and a request's result does not depend on its batch
    c.pool.copy_(start)
    out = torch.zeros(c.T, 4, 128, device="cuda", dtype=torch.bfloat16)
    prefill(hyb, c, out, cu[2:4], slots[2:3], None)
    assert torch.equal(out[203:332], res[0][0][203:332]) and torch.equal(c.pool[2], res[0][1][2])


def test_prefill_graph_replay_and_two_streams(hyb):
    lens = [150, 64, 9] * 30
    cs = [Case(19 + i, sum(lens), 2, 4, 128, torch.bfloat16, 90) for i in range(2)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    slots = torch.arange(90, dtype=torch.int32, device="cuda")
    start = [c.pool.clone() for c in cs]
    want = []
    for c, s in zip(cs, start):
        out = torch.empty(c.T, 4, 128, device="cuda", dtype=torch.bfloat16)
        prefill(hyb, c, out, cu, slots, None)
        want.append((out, c.pool.clone()))
    # two calls at once on two streams, each with its own workspace
    outs = [torch.empty_like(w[0]) for w in want]
    d = cs[0].dims(hyb)
    wss = [torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(90, cs[0].T, d), dtype=torch.uint8, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for c, s in zip(cs, start):
        c.pool.copy_(s)
    torch.cuda.synchronize()
    for c, o, w, st in zip(cs, outs, wss, streams):
        with torch.cuda.stream(st):
            prefill(hyb, c, o, cu, slots, None, ws=w, max_len=150)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w[0]) and torch.equal(c.pool, w[1]) for c, o, w in zip(cs, outs, want))
    # captured, then replayed on other inputs in the same buffers
    c = cs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prefill(hyb, c, outs[0], cu, slots, None, ws=wss[0], max_len=150)
        step(hyb, c, outs[1][:90], slots, 90)
    for x, y in zip((c.q, c.k, c.v, c.g, c.beta), (cs[1].q, cs[1].k, cs[1].v, cs[1].g, cs[1].beta)):
        x.copy_(y)
    for _ in range(2):
        c.pool.copy_(start[1])
        outs[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[1][0])
    after = torch.empty_like(outs[1][:90])
    cs[1].pool.copy_(want[1][1])
    step(hyb, cs[1], after, slots, 90)
    assert torch.equal(after, outs[1][:90]) and torch.equal(c.pool, cs[1].pool)
    assert hyb.hyb_device_status(clear=True) == (0, 0)


def test_prefill_nan_stays_in_its_request_where_chains_share_ctas(hyb):
    """More chains than two per SM, short and long ones mixed, so that a CTA runs several and cuts some: NaN
    or infinity in every third request's rows, gates or state, and in the rows of no request behind the
    last, changes no bit of the other requests."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, gap = (2 * sms + 1 + 3) // 4 + 2, 70
    rs = np.random.RandomState(9)
    lens = [int(n) for n in np.where(rs.rand(B) < 0.7, rs.randint(1, 90, B), rs.randint(90, 330, B))]
    lens[1], lens[5] = 0, 64
    first = np.concatenate([[0], np.cumsum(lens)])
    c = Case(25, sum(lens) + gap, 2, 4, 128, torch.bfloat16, B)
    cu = torch.tensor(first, dtype=torch.int32, device="cuda")
    slots = torch.tensor(rs.permutation(B), dtype=torch.int32, device="cuda")
    start = c.pool.clone()

    def call():
        c.pool.copy_(start)
        out = torch.full((c.T, 4, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        prefill(hyb, c, out, cu, slots, None)
        return out, c.pool.clone()

    clean, clean_pool = call()
    assert clean.isfinite().all() and clean_pool.isfinite().all()
    bad = [b for b in range(2, B, 3) if lens[b] > 0]
    what = [c.q, c.k, c.v, c.g, c.beta]
    for i, b in enumerate(bad):
        x = start if i % 6 == 5 else what[i % 6]
        row = int(slots[b]) if i % 6 == 5 else int(first[b]) + int(rs.randint(lens[b]))
        x[row] = math.inf if i % 12 < 6 and x is not c.g else math.nan
    for x in what:
        x[int(first[-1]):] = math.nan
    out, pool = call()
    same = torch.ones(c.T, dtype=torch.bool, device="cuda")
    for b in bad:
        same[int(first[b]):int(first[b + 1])] = False
        rows = out[int(first[b]):int(first[b + 1])]
        assert not (pool[slots[b].long()].isfinite().all() and rows.isfinite().all()), b
    assert torch.equal(out[same], clean[same])
    others = slots[[b for b in range(B) if b not in bad]].long()
    assert torch.equal(pool[others], clean_pool[others])
    assert hyb.hyb_device_status(clear=True) == (0, 0)


def test_prefill_request_alone_and_in_a_batch(hyb):
    """Which kernel and which order of its sums a request gets depends on max_len and the number of
    chains: alone, in a batch, or with a larger bound on the rows, it equals the recurrence to the same
    tolerance, not bit by bit."""
    T, B = 20, 64
    c = Case(27, T * B, 2, 4, 128, torch.bfloat16, B)
    start = c.pool.clone()
    S0 = host(start[3])
    o, S, mag, norm = c.ref(slice(3 * T, 4 * T), S0)
    cu = torch.arange(0, T * B + 1, T, dtype=torch.int32, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    for a, b, bound in ((0, B, None), (3, 4, None), (3, 4, 41)):
        c.pool.copy_(start)
        out = torch.zeros(c.T, 4, 128, device="cuda", dtype=torch.bfloat16)
        prefill(hyb, c, out, cu[a:b + 1], slots[a:b], None, max_len=bound)
        R.check_out(host(out)[3 * T:4 * T], o, mag, HALF[torch.bfloat16], T, f"{a} to {b}", split=True)
        R.check_state(host(c.pool)[3], S, norm, T, f"{a} to {b}")


@pytest.mark.parametrize("long_rows", [9, 16, 64, 100])
@pytest.mark.parametrize("n", [3, 255])
def test_prefill_decode_rows_beside_a_prompt(hyb, n, long_rows):
    """A batch of one-row requests and one of more rows, at both sides of the choice of the kernel."""
    lens = [1] * n
    lens.insert(n // 2, long_rows)
    c = Case(26, sum(lens) + 1, 2, 4, 128, torch.bfloat16, n + 2, fused=True)
    check_prefill(hyb, c, lens, [int(i % 5 == 0) for i in range(n + 1)], f"{n} rows and {long_rows}", gap=1)


@pytest.mark.parametrize("lens,heads,launches", [([16], 32, 1), ([64], 32, 1), ([1] * 255 + [64], 4, 1), ([1] * 255 + [100], 4, 2), ([1] * 31 + [32], 32, 1), ([1] * 31 + [200], 32, 2),
                                                 ([5] * 100 + [9] * 100, 4, 1), ([11] * 200, 4, 2)])
def test_prefill_rows_of_the_whole_call_choose_the_kernel(hyb, lens, heads, launches):
    """Decode rows beside a prompt are the recurrence's (one launch) where their states are most of the
    work; the tensor-core kernel on more chains than SMs takes two launches."""
    c = Case(28, sum(lens), heads // 2, heads, 128, torch.bfloat16, len(lens))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    out = torch.empty(c.T, heads, 128, device="cuda", dtype=torch.bfloat16)
    hyb.hyb_launch_count(reset=True)
    prefill(hyb, c, out, cu, slots, None)
    assert hyb.hyb_launch_count(reset=True) == launches


@pytest.mark.parametrize("lens,heads", [([32], 4), ([33], 4), ([32, 16], 32), ([32, 17], 32), ([10] * 40, 4), ([10] * 40 + [11], 4), ([1] * 59 + [31], 4), ([1] * 59 + [32], 4), ([1] * 37 + [25], 4)])
def test_prefill_at_both_sides_of_the_kernel_choice(hyb, lens, heads):
    c = Case(29, sum(lens), 2, heads, 128, torch.bfloat16, len(lens))
    check_prefill(hyb, c, lens, None, f"{len(lens)} requests, the longest of {max(lens)}")
