"""Measured cases of the hybrid-model layer operators: the gated delta rule (one-token step and
chunked prefill over a pool of fp32 states) and the query/key preparation of a Full layer (norm
of each head, rotary position, append to the paged cache, in one pass).

`run` computes each operator in plain torch (32 bits; angles and long sums in 64) when `own` is
false, and calls the library's entry points when it is true. `exact` is the definition in
64 bits.

Sizes are the ones this repository serves: 32 value heads of 128, 64 requests a decode step,
8 prompts of 8192 rows, 16-token cache blocks, the 80 % short / 20 % long request mix.
"""
import math
import random

import torch

own = False

CHUNK = 64          # rows the plain chunked form treats at once
L2_EPS = 1e-6       # under the root of a query's or key's length
RMS_EPS = 1e-6
BLOCK = 16


# ---------------------------------------------------------------------------------- cases
def _step(name, B, Hk, Hv, D, dtype="bf16", spare=3):
    return {"name": name, "op": "step", "B": B, "Hk": Hk, "Hv": Hv, "D": D, "dtype": dtype, "spare": spare}


def _prefill(name, B, max_len, ragged, Hk, Hv, D, dtype="bf16"):
    return {"name": name, "op": "prefill", "B": B, "max_len": max_len, "ragged": ragged, "Hk": Hk, "Hv": Hv, "D": D, "dtype": dtype}


def _rope(name, T, Hq, Hk, D, rot, interleaved, far, fused, dtype="bf16"):
    return {"name": name, "op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot, "interleaved": interleaved, "far": far, "fused": fused, "dtype": dtype}


def listed():
    return [
        # one user's decode step: latency is everything
        _step("step_one_request", 1, 32, 32, 128),
        # the 64-request decode batch
        _step("step_64_requests", 64, 32, 32, 128),
        # a full decode batch, two value heads to each query/key head
        _step("step_256_shared_keys", 256, 16, 32, 128),
        # fp32 rows, small heads, a batch of odd size
        _step("step_fp32_small_heads", 13, 6, 6, 64, "f32"),
        # a chat turn of one request: a few rows on a state that is there already
        _prefill("prefill_short_turn", 1, 77, False, 16, 32, 128),
        # one prompt: few chains, so the chain's own latency counts
        _prefill("prefill_one_prompt", 1, 4096, False, 16, 32, 128),
        # a batch of short and long prompts, with an empty one among them
        _prefill("prefill_ragged", 24, 5000, True, 32, 32, 128),
        # the 8 x 8192 prefill
        _prefill("prefill_8x8192", 8, 8192, False, 32, 32, 128),
        # fp32 rows, ragged
        _prefill("prefill_fp32", 3, 700, True, 8, 8, 64, "f32"),
        # one decode step's queries and keys
        _rope("rope_decode_64", 64, 32, 32, 128, 128, False, 131072, False),
        # prompts straight from a fused projection, 8 key heads, far positions
        _rope("rope_prefill_65536", 65536, 32, 8, 128, 128, False, 131072, True),
        # fp32, pairs side by side, half of the head rotated, odd number of rows
        _rope("rope_fp32_partial", 1021, 4, 4, 64, 32, True, 8192, False, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "rope"])
    if op == "step":
        Hv = rng.choice([1, 4, 6, 16, 32, 48])
        Hk = rng.choice([h for h in range(1, Hv + 1) if Hv % h == 0 and Hv // h <= 4])
        c = _step("", _log(rng, 1, 256 if Hv <= 32 else 160), Hk, Hv, rng.choice([64, 128, 128, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.randrange(0, 5))
    elif op == "prefill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        D = 128 if dtype == "bf16" and rng.random() < 0.8 else 64
        Hv = rng.choice([2, 4, 8, 16, 32])
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h <= Hv and Hv // h <= 4])
        max_len = _log(rng, 1, 8192 if dtype == "bf16" and D == 128 else 1024)
        most = max(1, min(64, (1 << 20) // (max_len * Hv)))
        c = _prefill("", _log(rng, 1, most), max_len, rng.random() < 0.7, Hk, Hv, D, dtype)
    else:
        dtype, D = rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        c = _rope("", _log(rng, 1, 32768 if dtype == "bf16" else 8192), Hq, Hk, D, rng.choice([D, D, D // 2, D // 4]), rng.random() < 0.4,
                  rng.choice([4096, 32768, 131072, 1000000]), rng.random() < 0.5, dtype)
    del c["name"]
    return c


def _lens(case):
    """Rows of each request: all alike, or 80 % short (log-uniform) and 20 % long, one of them empty."""
    B, M = case["B"], case["max_len"]
    if not case["ragged"]:
        return [M] * B
    r = random.Random(B * 100003 + M)
    short = [max(1, int(round(math.exp(r.uniform(0, math.log(max(2, M / 4))))))) for _ in range(B)]
    lens = [min(M, n if r.random() < 0.8 else r.randint(max(1, M // 2), M)) for n in short]
    lens[B // 2] = M
    if B >= 4:
        lens[1] = 0
    return lens


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "rope":
        T, rows = case["T"], case["Hq"] + 2 * case["Hk"]
        # rows read and written once; position, slot, weights, frequencies
        return {"bytes": 2 * T * rows * D * es + 12 * T + 2 * D * 4 + 2 * case["rot"], "flops": T * (case["Hq"] + case["Hk"]) * D * 7}
    Hk, Hv = case["Hk"], case["Hv"]
    T = case["B"] if case["op"] == "step" else sum(_lens(case))
    chains = case["B"] * Hv
    rows = T * (2 * Hk + 2 * Hv) * D * es + 8 * T * Hv   # q, k, v, out, gate and beta
    states = 2 * chains * D * D * 4
    if case["op"] == "step":
        return {"bytes": rows + states, "flops": T * Hv * D * D * 7}
    # k k^T and q k^T (lower half), the inverse's product, k S, q S, the row and the state product, for chunks of 64
    per_row = CHUNK * D * 2 + CHUNK * D + CHUNK * D + 6 * D * D
    return {"bytes": rows + states, "flops": T * Hv * per_row}


# --------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    D = case["D"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    st = {"case": case, "dt": dt}
    if case["op"] == "rope":
        T, Hq, Hk, rot, far = case["T"], case["Hq"], case["Hk"], case["rot"], case["far"]
        width = (Hq + 2 * Hk) * D
        if case["fused"]:      # q, k and v are parts of one projection's rows
            qkv = normal(T, width).to(dt)
            st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
        else:
            st["q"], st["k"], st["v"] = (normal(T, h, D).to(dt) for h in (Hq, Hk, Hk))
        # rows of several requests, each going on from its own position
        start = torch.randint(0, max(1, far - T), (8,), generator=gen, device=dev)
        at = torch.arange(T, device=dev)
        part = at * 8 // T
        first = (part * T + 7) // 8
        st["positions"] = (start[part] + at - first).to(torch.int32)
        blocks = (T + BLOCK - 1) // BLOCK + 4
        where = torch.randperm(blocks, generator=gen, device=dev)[: (T + BLOCK - 1) // BLOCK]
        st["slots"] = where[at // BLOCK] * BLOCK + at % BLOCK
        if T > 8:
            st["slots"][T // 3] = -1          # a row that has no place in the cache
        # frequencies 1e6^(-2i/rot), interpolated for a context four times as long where a turn is longer than 8192 positions
        f = 1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        st["inv_freq"] = torch.where(2 * math.pi / f > 8192, f / 4, f).float()
        st["attn_factor"] = 0.1 * math.log(4.0) + 1.0
        st["qw"], st["kw"] = (1 + 0.1 * normal(D) for _ in range(2))
        st["kc"], st["vc"] = (torch.zeros(blocks, Hk, BLOCK, D, device=dev, dtype=dt) for _ in range(2))
        st["out"] = torch.empty(T, Hq, D, device=dev, dtype=dt)
    else:
        Hk, Hv, B = case["Hk"], case["Hv"], case["B"]
        lens = [1] * B if case["op"] == "step" else _lens(case)
        T = sum(lens)
        # one projection's rows hold q, k and v side by side
        qkv = normal(T, (2 * Hk + Hv) * D).to(dt)
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hk * D, Hk * D, Hv * D], dim=1))
        # log decay -a * softplus(x + bias): heads with a near 0 keep their state, heads near 16 soon drop it
        a, bias = 16 * uniform(Hv), torch.log(torch.expm1(10 ** (-3 + 2 * uniform(Hv))))
        st["g"] = -a * torch.nn.functional.softplus(normal(T, Hv) + bias)
        st["beta"] = torch.sigmoid(normal(T, Hv))
        NS = B + case.get("spare", 2)
        st["pool"] = 0.3 * normal(NS, Hv, D, D)
        st["slots"] = torch.randperm(NS, generator=gen, device=dev)[:B].to(torch.int32)
        st["NS"], st["lens"], st["T"] = NS, lens, T
        st["out"] = torch.empty(T, Hv, D, device=dev, dtype=dt)
        if case["op"] == "prefill":
            st["cu"] = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
            # every third request starts anew, the others go on from their state
            st["reset"] = (torch.arange(B, device=dev) % 3 == 2).to(torch.uint8)
    if own:   # the sizes and the workspace that a serving program keeps
        import paged_kv_linear_gb300 as hyb
        if case["op"] == "rope":
            stride = width if case["fused"] else 0
            st["d"] = hyb.dims(Hk, D, st["kc"].shape[0], 1, dt)
            st["r"] = hyb.rope_dims(Hq, rot, eps=RMS_EPS, interleaved=case["interleaved"], attn_factor=st["attn_factor"], q_stride=stride, k_stride=stride, v_stride=stride)
        else:
            stride = (2 * Hk + Hv) * D
            st["d"] = hyb.delta_dims(Hk, Hv, D, dt, qk_norm_eps=L2_EPS, q_stride=stride, k_stride=stride, v_stride=stride)
            if case["op"] == "prefill":
                n = hyb.hyb_gated_delta_chunked_prefill_workspace_size(B, T, st["d"])
                st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------------------------ run
def run(st):
    return {"step": _run_step, "prefill": _run_prefill, "rope": _run_rope}[st["case"]["op"]](st)


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + L2_EPS)


def _run_step(st):
    c = st["case"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_gated_delta_step(st["out"], st["q"], st["k"], st["v"], st["g"], st["beta"], st["pool"], st["NS"], st["slots"], c["B"], st["d"]))
        return {"out": st["out"], "state": st["pool"]}
    rep = c["Hv"] // c["Hk"]
    q, k = (_unit(st[n].float()).repeat_interleave(rep, dim=1) for n in ("q", "k"))
    slots = st["slots"].long()
    S = st["pool"][slots] * torch.exp(st["g"])[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    st["pool"][slots] = S
    out = (q[..., None] * S).sum(-2) * c["D"] ** -0.5
    return {"out": out.to(st["dt"]), "state": st["pool"]}


def _run_prefill(st):
    """Within a chunk, with G the running sum of g, S the state at its start and A_ij =
    beta_i exp(G_i - G_j) k_i.k_j below the diagonal: the chunk's corrections are
    X = (1 + A)^-1 beta (v - exp(G) k S), its outputs q (exp(G) S) + tril(exp(G_i - G_j) q_i.k_j) X,
    and the next state is exp(G_end) S + sum_i exp(G_end - G_i) k_i X_i."""
    c = st["case"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_gated_delta_chunked_prefill(st["out"], st["q"], st["k"], st["v"], st["g"], st["beta"], st["cu"], st["pool"], st["NS"], st["slots"], st["reset"], c["B"],
                                                      st["T"], max(st["lens"]), st["d"], st["ws"], st["ws"].numel()))
        return {"out": st["out"], "state": st["pool"]}
    B, Hv, D, dev = c["B"], c["Hv"], c["D"], st["q"].device
    rep = Hv // c["Hk"]
    N = (max(st["lens"]) + CHUNK - 1) // CHUNK
    lens = (st["cu"][1:] - st["cu"][:-1]).long()
    at = torch.arange(N * CHUNK, device=dev)
    valid = at[None, :] < lens[:, None]                                   # [B, L]
    rows = torch.where(valid, st["cu"][:-1, None].long() + at[None, :], 0)

    def chunks(x):                                                        # [T, H, ...] -> [B, H, N, C, ...], 0 past the end
        x = torch.where(valid.view(B, N * CHUNK, *[1] * (x.dim() - 1)), x[rows], 0)
        return x.transpose(1, 2).unflatten(2, (N, CHUNK))

    q, k = (chunks(_unit(st[n].float()).repeat_interleave(rep, dim=1)) for n in ("q", "k"))
    v, beta = chunks(st["v"].float()), chunks(st["beta"])
    G = chunks(st["g"].double()).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    fade = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    A = (beta[..., None] * fade * (k @ k.transpose(-1, -2))).tril(-1)
    W = torch.eye(CHUNK, device=dev).expand_as(A).clone()                 # (1 + A)^-1, row after row
    for i in range(1, CHUNK):
        W[..., i, :i] = -(A[..., i, None, :i] @ W[..., :i, :i]).squeeze(-2)
    del A
    eG = torch.exp(G).float()[..., None]
    X0 = W @ (beta[..., None] * v)
    X1 = W @ (beta[..., None] * eG * k)
    P = fade * (q @ k.transpose(-1, -2))
    last = torch.exp(G[..., -1:] - G).float()[..., None]
    end = torch.exp(G[..., -1]).float()[..., None, None]
    slots = st["slots"].long()
    S = torch.where(st["reset"].view(B, 1, 1, 1) != 0, 0, st["pool"][slots])
    O = torch.empty(B, Hv, N, CHUNK, D, device=dev)
    for n in range(N):
        X = X0[:, :, n] - X1[:, :, n] @ S
        O[:, :, n] = (eG[:, :, n] * q[:, :, n]) @ S + P[:, :, n] @ X
        S = end[:, :, n] * S + (last[:, :, n] * k[:, :, n]).transpose(-1, -2) @ X
    st["pool"][slots] = S
    out = (O.flatten(2, 3).transpose(1, 2) * D ** -0.5).to(st["dt"])[valid]
    return {"out": out, "state": st["pool"]}


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(st):
    c = st["case"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_qk_norm_rope_append(st["out"], None, st["q"], st["k"], st["v"], st["positions"], st["slots"], st["inv_freq"], st["qw"], st["kw"], c["T"],
                                              st["kc"], st["vc"], st["r"], st["d"]))
        return {"q": st["out"], "k_cache": st["kc"], "v_cache": st["vc"]}
    angle = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    cos, sin = (torch.cos(angle) * st["attn_factor"]).float(), (torch.sin(angle) * st["attn_factor"]).float()
    done = []
    for n, w in (("q", st["qw"]), ("k", st["kw"])):
        x = st[n].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS) * w
        done.append(_rotate(x, cos, sin, c["rot"], c["interleaved"]).to(st["dt"]))
    keep = st["slots"] >= 0
    at = st["slots"][keep]
    st["kc"][at // BLOCK, :, at % BLOCK] = done[1][keep]
    st["vc"][at // BLOCK, :, at % BLOCK] = st["v"][keep]
    return {"q": done[0], "k_cache": st["kc"], "v_cache": st["vc"]}


# ---------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    st = prepare(case, seed)
    D = case["D"]
    if case["op"] == "rope":
        T, rot = case["T"], case["rot"]
        angle = torch.outer(st["positions"].double(), st["inv_freq"].double())
        turn = torch.polar(torch.full_like(angle, st["attn_factor"]), angle)[:, None]          # [T, 1, rot / 2]

        def prepared(x, w):
            x = x.double()
            x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / D + RMS_EPS).sqrt()
            head = x[..., :rot]
            pairs = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            return x

        q, k = prepared(st["q"], st["qw"]), prepared(st["k"], st["kw"])
        caches = []
        for x in (k, st["v"].double()):
            flat = torch.zeros(st["kc"].shape[0] * BLOCK, *x.shape[1:], dtype=torch.float64, device=x.device)
            kept = (st["slots"] >= 0).nonzero().flatten()
            flat[st["slots"][kept]] = x[kept]
            caches.append(flat.unflatten(0, (-1, BLOCK)).transpose(1, 2))
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}

    lens = st["lens"]
    if max(lens) * (2 + case["B"] * case["Hv"] * D * D / 2e6) > 60000:
        return None
    Hv, rep = case["Hv"], case["Hv"] // case["Hk"]
    head = torch.arange(Hv, device="cuda") // rep
    pool = st["pool"].double()
    out = torch.zeros(st["T"], Hv, D, dtype=torch.float64, device="cuda")
    first = [sum(lens[:b]) for b in range(len(lens))]
    order = sorted(range(len(lens)), key=lambda b: -lens[b])              # longest first: those with a token t are a prefix
    slots = st["slots"].long()[order]
    S = pool[slots]
    if case["op"] == "prefill":
        S[st["reset"][order] != 0] = 0
    begin = torch.tensor([first[b] for b in order], device="cuda")
    active = len(order)
    for t in range(max(lens)):
        while active and lens[order[active - 1]] <= t:
            active -= 1
        r, now = begin[:active] + t, S[:active]
        k, q = st["k"][r].double()[:, head], st["q"][r].double()[:, head]
        k = k / (k.pow(2).sum(-1, keepdim=True) + L2_EPS).sqrt()
        q = q / (q.pow(2).sum(-1, keepdim=True) + L2_EPS).sqrt()
        now *= st["g"][r].double().exp()[..., None, None]
        miss = st["v"][r].double() - torch.einsum("bhi,bhij->bhj", k, now)
        now += torch.einsum("bhi,bhj->bhij", k, st["beta"][r].double()[..., None] * miss)
        out[r] = torch.einsum("bhi,bhij->bhj", q, now) / math.sqrt(D)
    pool[slots] = S
    return {"out": out, "state": pool}
