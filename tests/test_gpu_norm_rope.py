"""Query/key preparation (norm, rotary position, append) against its 64-bit form, and the
layers' operators one after another as a model runs them."""
import numpy as np
import pytest
import torch

import layer_ops_ref as R
import oracle
import workloads as W
from gpu_helpers import assert_out_close

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def host(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def freqs(rot, base=1e6):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device="cuda")


def run(hyb, T, Hq, Hk, D, rot, dt, interleaved=False, bs=16, fused=False, norm=True, w_off=0.0, m=1.0, far=5000, cache=True, k_out=False, in_place=False, seed=0, holes=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    width = (Hq + 2 * Hk) * D + (8 if fused else 0)
    rows = (3 * rnd(T, width)).to(dt)
    q, k, v = (p.unflatten(1, (-1, D)) for p in rows[:, :(Hq + 2 * Hk) * D].split([Hq * D, Hk * D, Hk * D], dim=1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    stride = width if fused else 0
    pos = torch.randint(0, far + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)
    pos[0] = far
    if T > 2:
        pos[1] = 0
    NB = (T + bs - 1) // bs + 2
    slots = torch.randperm(NB * bs, generator=gen, device="cuda")[:T]
    if holes and T > 4:
        slots[2] = -1
        pos[3] = -1          # a padded row: nothing of it is written
    qw, kw = (1 - w_off + 0.2 * rnd(D) for _ in range(2)) if norm else (None, None)
    kc0, vc0 = (rnd(NB, Hk, bs, D).to(dt) for _ in range(2))
    kc, vc = kc0.clone(), vc0.clone()
    q_in, k_in = host(q), host(k)
    q_out = q if in_place else torch.full((T, Hq, D), 7.0, device="cuda", dtype=dt) if Hq else None
    ko = k if in_place else torch.full((T, Hk, D), 7.0, device="cuda", dtype=dt) if k_out else None
    r = hyb.rope_dims(Hq, rot, eps=1e-5, interleaved=interleaved, weight_offset=w_off, attn_factor=m, q_stride=stride, k_stride=stride, v_stride=stride)
    d = hyb.dims(Hk, D, NB, 4, dt, block_size=bs)
    f = freqs(rot) if rot else None
    hyb.check(hyb.hyb_qk_norm_rope_append(q_out, ko, q if Hq else None, k, v if cache else None, pos, slots if cache else None, f, qw, kw, T,
                                          kc if cache else None, vc if cache else None, r, d))
    torch.cuda.synchronize()
    assert hyb.hyb_device_status(clear=True) == (0, 0)
    p_h, s_h = pos.cpu().numpy(), slots.cpu().numpy()
    live = p_h >= 0
    args = (w_off, 1e-5, np.maximum(p_h, 0), f.cpu().numpy() if rot else None, m, rot, interleaved)

    def check(got, x, w, what, where=live):
        w = None if w is None else w.cpu().numpy()
        ref = R.norm_rope(x, w, *args)
        lim = R.rope_limit(x, ref, w, w_off, 1e-5, m, rot, interleaved, HALF[dt])
        err = np.abs(got - ref)[where]
        assert (err <= lim[where]).all(), f"{what}: {(err / lim[where]).max():.2f} of the limit"

    if Hq:
        check(host(q_out), q_in, qw, "q")
        assert in_place or (host(q_out)[~live] == 7.0).all()
    if ko is not None:
        check(host(ko), k_in, kw, "k_out")
        assert in_place or (host(ko)[~live] == 7.0).all()
    if cache:
        put = live & (s_h >= 0)
        at = s_h[put]
        gk = host(kc)[at // bs, :, at % bs]
        full = np.zeros_like(k_in)
        full[put] = gk
        check(full, k_in, kw, "k cache", put)
        want_v, want_k = vc0.clone(), kc0.clone()
        sel = torch.tensor(at, device="cuda")
        want_v[sel // bs, :, sel % bs] = v[torch.tensor(put, device="cuda")]
        want_k[sel // bs, :, sel % bs] = kc[sel // bs, :, sel % bs]
        assert torch.equal(vc, want_v) and torch.equal(kc, want_k), "the caches beside the written rows"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (16, 8), (32, 8), (64, 64), (64, 16), (128, 128), (128, 64), (128, 96), (128, 0), (256, 256), (256, 64)])
def test_head_sizes_and_parts(hyb, D, rot, interleaved, dt):
    run(hyb, 23, 3, 3, D, rot, dt, interleaved=interleaved, fused=rot % 16 == 0, seed=D + rot)


@pytest.mark.parametrize("T", [1, 2, 7, 64, 1000, 5001])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 2), (5, 3)])
def test_rows_and_heads(hyb, T, Hq, Hk):
    run(hyb, T, Hq, Hk, 128, 128, torch.bfloat16, fused=True, seed=T + Hq)


@pytest.mark.parametrize("far", [1, 4095, 131072, 1000003, 1 << 24])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_far_positions(hyb, far, dt):
    run(hyb, 40, 2, 2, 64, 64, dt, far=far, m=1.2, seed=far % 1000)


@pytest.mark.parametrize("kw", [dict(norm=False), dict(w_off=1.0), dict(cache=False, k_out=True), dict(k_out=True), dict(in_place=True), dict(in_place=True, cache=False),
                                dict(bs=64), dict(norm=False, rot=0, holes=False), dict(Hq=0)])
def test_forms(hyb, kw):
    a = dict(T=33, Hq=4, Hk=2, D=128, rot=128, dt=torch.bfloat16)
    a.update(kw)
    run(hyb, **a)


def test_rows_pass_unchanged_without_norm_and_rotation(hyb):
    """Norm and rotation left out: q comes through and the caches equal the plain append's."""
    T, H, D = 37, 4, 128
    q, k, v = (torch.randn(T, H, D, device="cuda").bfloat16() for _ in range(3))
    slots = torch.randperm(64, device="cuda")[:T]
    caches = [torch.zeros(4, H, 16, D, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    d, r = hyb.dims(H, D, 4, 4), hyb.rope_dims(H, 0)
    q_out = torch.empty_like(q)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    hyb.check(hyb.hyb_qk_norm_rope_append(q_out, None, q, k, v, pos, slots, None, None, None, T, caches[0], caches[1], r, d))
    hyb.check(hyb.hyb_paged_kv_append(k, v, slots, T, caches[2], caches[3], d))
    assert torch.equal(q_out, q) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_bad_slots_and_positions_are_flagged_and_skipped(hyb, devstatus):
    T, H, D = 4, 2, 64
    q, k, v = (torch.randn(T, H, D, device="cuda") for _ in range(3))
    pos = torch.tensor([3, (1 << 24) + 1, 5, 6], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 32, 1 << 40], device="cuda")
    kc, vc = (torch.full((2, H, 16, D), 7.0, device="cuda") for _ in range(2))
    out = torch.full((T, H, D), 7.0, device="cuda")
    d, r = hyb.dims(H, D, 2, 4, torch.float32), hyb.rope_dims(H, D)
    hyb.check(hyb.hyb_qk_norm_rope_append(out, None, q, k, v, pos, slots, freqs(D), None, None, T, kc, vc, r, d))
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_BAD_SLOT | hyb.HYB_DEVERR_BAD_LENGTH)
    assert (out[1] == 7).all() and (out[[0, 2, 3]] != 7).any(-1).all()
    assert (kc[0, :, 0] != 7).any() and torch.equal(vc[0, :, 0], v[0])
    kc[0, :, 0], vc[0, :, 0] = 7, 7
    assert (kc == 7).all() and (vc == 7).all()


def test_zero_and_non_finite_rows(hyb):
    """A row of zeros stays zero; a NaN stays in its head row."""
    T, H, D = 3, 2, 128
    q, k, v = (torch.randn(T, H, D, device="cuda").bfloat16() for _ in range(3))
    q[0] = 0
    k[1, 1, 5] = float("nan")
    v[1, 0, 5] = float("inf")
    ones = torch.ones(D, device="cuda")
    kc, vc = (torch.zeros(1, H, 16, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out = torch.empty_like(q)
    pos = torch.tensor([9, 8, 7], dtype=torch.int32, device="cuda")
    hyb.check(hyb.hyb_qk_norm_rope_append(out, None, q, k, v, pos, torch.arange(3, device="cuda"), freqs(D), ones, ones, T, kc, vc, hyb.rope_dims(H, D), hyb.dims(H, D, 1, 1)))
    assert (out[0] == 0).all() and out.isfinite().all()
    assert kc[0, 1, 1].isnan().all()
    kc[0, 1, 1] = 0
    assert kc.isfinite().all() and torch.equal(vc[0, :, :3].transpose(0, 1), v)


def test_hybrid_layers_prefill_then_decode(hyb, devstatus):
    """A Full and a gated Linear layer on the same requests: queries and keys prepared into the
    cache, causal attention over it, the delta rule over the prompt; then three decode steps,
    one of them captured in a graph. Checked against the oracle's attention on the prepared rows
    and the 64-bit recurrence."""
    H, D, bs, B = 4, 128, 16, 3
    prompts, steps = np.array([37, 64, 5]), 3
    gen = torch.Generator(device="cuda").manual_seed(4)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    g = W.rng(3)
    pool = W.block_pool(g, (prompts + steps).astype(np.int32))
    bt = torch.from_numpy(np.ascontiguousarray(pool.block_tables)).cuda()
    kc, vc = (torch.zeros(pool.num_blocks, H, bs, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    d = hyb.dims(H, D, pool.num_blocks, pool.max_blocks)
    f, qw, kw = freqs(D), 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    stride = 3 * H * D
    r = hyb.rope_dims(H, D, q_stride=stride, k_stride=stride, v_stride=stride)
    dd = hyb.delta_dims(H, H, D, qk_norm_eps=1e-6, q_stride=stride, k_stride=stride, v_stride=stride)
    state = 0.3 * rnd(B, H, D, D)
    state0 = host(state)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    seen = [[] for _ in range(B)]         # (q rows, k rows, v rows, gate, beta, attention out, delta out)
    lin_ws = torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(B, 200, dd), dtype=torch.uint8, device="cuda")
    done = np.zeros(B, int)
    for n in range(steps + 1):
        counts = prompts if n == 0 else np.ones(B, int)
        T = int(counts.sum())
        cu_h = np.concatenate([[0], np.cumsum(counts)])
        cu = torch.tensor(cu_h, dtype=torch.int32, device="cuda")
        ctx = torch.tensor(done, dtype=torch.int32, device="cuda")
        qkv = rnd(T, 3 * H * D).bfloat16()
        q, k, v = (x.unflatten(1, (H, D)) for x in qkv.split(H * D, dim=1))
        gate, beta = -torch.rand(T, H, generator=gen, device="cuda"), torch.rand(T, H, generator=gen, device="cuda")
        pos = torch.tensor(np.concatenate([np.arange(c) + o for c, o in zip(counts, done)]), dtype=torch.int32, device="cuda")
        sm = torch.empty(T, dtype=torch.int64, device="cuda")
        q_rot, att, lin = (torch.empty(T, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
        lens = torch.tensor(done + counts, dtype=torch.int32, device="cuda")
        longest = int((done + counts).max())
        ws_n = hyb.hyb_paged_attn_decode_workspace_size(B, 128, d)
        ws = torch.empty(max(ws_n, 16), dtype=torch.uint8, device="cuda")

        def layer():
            hyb.check(hyb.hyb_slot_mapping(sm, bt, cu, ctx, B, T, d))
            hyb.check(hyb.hyb_qk_norm_rope_append(q_rot, None, q, k, v, pos, sm, f, qw, kw, T, kc, vc, r, d))
            if n == 0:
                hyb.check(hyb.hyb_paged_attn_prefill_causal(att, q_rot, kc, vc, bt, cu, ctx, B, T, 64, d))
                hyb.check(hyb.hyb_gated_delta_chunked_prefill(lin, q, k, v, gate, beta, cu, state, B, slots, None, B, T, 64, dd, lin_ws, lin_ws.numel()))
            else:
                hyb.check(hyb.hyb_paged_attn_decode(att, q_rot, kc, vc, bt, lens, B, longest, d, ws, ws_n))
                hyb.check(hyb.hyb_gated_delta_step(lin, q, k, v, gate, beta, state, B, slots, B, dd))

        if n == 2:
            saved = state.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layer()
            state.copy_(saved)
            graph.replay()
        else:
            layer()
        torch.cuda.synchronize()
        ref_q = R.bf16(R.norm_rope(host(q), qw.cpu().numpy(), 0.0, 1e-6, pos.cpu().numpy(), f.cpu().numpy(), 1.0, D, False))
        assert np.abs(host(q_rot) - ref_q).max() <= 2.0 ** -7 * np.abs(ref_q).max()
        kc_h, vc_h = (x.view(torch.int16).cpu().numpy().view(np.uint16) for x in (kc, vc))
        q_h = q_rot.view(torch.int16).cpu().numpy().view(np.uint16)
        assert_out_close(att, oracle.full_prefill(q_h, kc_h, vc_h, pool.block_tables, cu_h.astype(np.int32), done.astype(np.int32), D ** -0.5), f"attention {n}")
        for b in range(B):
            seen[b].append([host(x[cu_h[b]:cu_h[b + 1]]) for x in (q, k, v, gate, beta, lin)])
        done = done + counts
    for b in range(B):
        q, k, v, gate, beta, lin = (np.concatenate(x) for x in zip(*seen[b]))
        o, S, mag, norm = R.delta_rule(q, k, v, gate, beta, state0[b], D ** -0.5, 1e-6)
        R.check_out(lin, o, mag, 2.0 ** -8, len(q), f"delta rule, request {b}", split=True)
        R.check_state(host(state)[b], S, norm, len(q), f"state {b}")
    assert devstatus() == (0, 0)


@pytest.mark.parametrize("share", [2, 3, 5, 6])
@pytest.mark.parametrize("Hq,Hk", [(32, 8), (32, 32), (5, 3)])
def test_tokens_in_shares_and_more_than_one_pass(hyb, Hq, Hk, share):
    """Tokens enough for several items a warp, but few enough that each is shared by several warps: the
    steps from item to item carry from share to token."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    run(hyb, 32 * sms // share, Hq, Hk, 128, 128, torch.bfloat16, fused=True, seed=share + Hq)
    run(hyb, 32 * sms // share - 7, Hq, Hk, 64, 32, torch.float32, interleaved=True, seed=share)
