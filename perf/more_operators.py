"""Measured cases of a decode step that continues one prompt in several ways (beam search, several
answers to a prompt, requests behind one system prompt): paged decode attention that reads a
group's shared prefix once, the selection of the next beams over beams and vocabulary, and the
reordering of the beams' caches and states by that selection.

`run` computes each operator in plain torch (32 bits; sums over the vocabulary and the scores that
are compared in 64) when `own` is false, and calls the library's entry points when it is true.
`exact` is the definition in 64 bits.

Sizes are the ones this repository serves: 32 query heads of 128 (8 key heads where they are
shared), 16-token cache blocks, 64 requests a decode step, the 80 % short / 20 % long request mix,
fp32 states of 32 x 128 x 128, three Full layers to a Linear one. Vocabularies are generic.
"""
import math
import random

import torch

own = False

FULL, LINEAR = "F", "L"        # layers of a stack, as in "FFFL"


# ---------------------------------------------------------------------------------- cases
def _prefix(name, groups, most, ragged, prefix, suffix, Hq, Hk, D, dtype="bf16", block=16, window=0):
    return {"name": name, "op": "prefix", "groups": groups, "most": most, "ragged": ragged, "prefix": prefix, "suffix": suffix, "Hq": Hq, "Hk": Hk, "D": D, "dtype": dtype,
            "block": block, "window": window}


def _select(name, R, W, N, V, dtype="bf16", pad=0, masked=0.0, mixed=False):
    return {"name": name, "op": "select", "R": R, "W": W, "N": N, "V": V, "dtype": dtype, "pad": pad, "masked": masked, "mixed": mixed}


def _reorder(name, R, W, layers, prefix, suffix, Hk, Hv, D, dtype="bf16", block=16):
    return {"name": name, "op": "reorder", "R": R, "W": W, "layers": layers, "prefix": prefix, "suffix": suffix, "Hk": Hk, "Hv": Hv, "D": D, "dtype": dtype, "block": block}


def listed():
    return [
        # one user's beam search over a long prompt: latency counts
        _prefix("prefix_one_prompt_4_beams", 1, 4, False, 4096, 40, 32, 32, 128),
        # a 64-request decode batch behind one system prompt, short and long conversations
        _prefix("prefix_64_requests", 1, 64, False, 2048, 2048, 32, 32, 128),
        # several prompts of different lengths, each with up to 8 beams, shared key heads
        _prefix("prefix_16_prompts_of_8", 16, 8, True, 8192, 300, 32, 8, 128, block=32),
        # a large batch that asks about one long document
        _prefix("prefix_256_on_a_document", 1, 256, False, 32768, 256, 32, 8, 128),
        # smaller heads, a sliding window that ends inside the prefix for some requests
        _prefix("prefix_window_small_heads", 3, 24, True, 5000, 700, 12, 4, 64, block=64, window=2048),
        # fp32, odd sizes
        _prefix("prefix_fp32", 2, 5, True, 777, 90, 6, 6, 64, "f32"),
        # one user's beams over a small vocabulary
        _select("select_one_request", 1, 4, 8, 32768, "f32"),
        # a full batch: 64 requests of 8 beams
        _select("select_64_requests", 64, 8, 8, 131072),
        # odd sizes, rows of a padded projection, banned tokens, finished and unborn beams
        _select("select_odd", 9, 5, 10, 50021, "f32", pad=27, masked=0.3, mixed=True),
        # one user's beams: four layers
        _reorder("reorder_one_request", 1, 4, "FFFL", 1000, 40, 8, 32, 128),
        # 16 requests of 4 beams, long answers
        _reorder("reorder_16_requests", 16, 4, "FFFLFFFL", 500, 1024, 8, 32, 128),
        # Linear layers alone: 32 requests of 8 beams
        _reorder("reorder_states", 32, 8, "LL", 0, 64, 8, 32, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "select", "reorder"])
    if op == "prefix":
        dtype = rng.choice(["bf16"] * 5 + ["f32"])
        D = rng.choice([64, 128, 128, 128] if dtype == "bf16" else [64, 128])
        Hk = rng.choice([1, 2, 4, 8, 16, 32] if dtype == "bf16" else [1, 2, 4, 8])
        Hq = Hk * rng.choice([r for r in (1, 1, 2, 3, 4, 8) if Hk * r <= 48])
        prefix = _log(rng, 1, 32768 if dtype == "bf16" else 4096)
        groups = _log(rng, 1, max(1, min(24, (1 << 21) // (prefix * Hk))))
        most = _log(rng, 1, max(1, min(256, (1 << 28 if dtype == "bf16" else 1 << 24) // (prefix * Hq * groups))))
        suffix = _log(rng, 1, max(1, min(2048, (1 << 22) // (most * groups * Hk))))
        c = _prefix("", groups, most, rng.random() < 0.6, prefix, suffix, Hq, Hk, D, dtype, rng.choice([16, 16, 32, 64, 128]), rng.choice([0, 0, 0, _log(rng, 16, 8192)]))
    elif op == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        V = _log(rng, 1000, 200000)
        dtype = rng.choice(["bf16", "f32"])
        most = max(1, min(64, (1 << (25 if dtype == "f32" else 26)) // (W * V)))
        c = _select("", _log(rng, 1, most), W, rng.choice([W, W, 2 * W]), V, dtype, rng.choice([0, 0, 3, 64]), rng.choice([0.0, 0.0, 0.5]), rng.random() < 0.5)
    else:
        W = rng.choice([2, 3, 4, 5, 8, 16])
        layers = rng.choice(["FFFL", "FF", "LL", "FLFLFL", "FFFLFFFL"])
        Hk, Hv, D = rng.choice([1, 2, 4, 8]), rng.choice([4, 8, 16, 32]), rng.choice([64, 128, 128])
        suffix = _log(rng, 1, 1024)
        most = max(1, min(64 // W, (1 << 20) // (W * suffix * Hk * len(layers))))
        c = _reorder("", _log(rng, 1, most), W, layers, rng.choice([0, 17, 250, 1000]), suffix, Hk, Hv, D, rng.choice(["bf16", "bf16", "f32"]) if suffix <= 256 else "bf16",
                     rng.choice([16, 16, 32, 64]))
    del c["name"]
    return c


def _shape(case):
    """What the case alone decides: the lengths, and which beams go on."""
    if case["op"] == "prefix":
        G, M = case["groups"], case["most"]
        r = random.Random(G * 7919 + M * 104729 + case["prefix"])
        size = [M if g == G // 2 or not case["ragged"] else r.randint(1, M) for g in range(G)]
        pre = [case["prefix"] if g == G // 2 or not case["ragged"] else max(1, int(case["prefix"] * r.random())) for g in range(G)]
        tails = []
        for g in range(G):      # 80 % short answers, 20 % long ones; every request has its own newest token at least
            S = case["suffix"]
            tails.append([max(1, min(S, int(round(math.exp(r.uniform(0, math.log(max(2, S / 4)))))) if r.random() < 0.8 else r.randint(max(1, S // 2), S))) for _ in range(size[g])])
        tails[G // 2][0] = case["suffix"]
        return size, pre, tails
    R, W = case["R"], case["W"]
    r = random.Random(R * 7919 + W * 104729)
    if case["op"] == "select":
        kind = []               # of each beam: 0 goes on, 1 finished, 2 unborn
        for q in range(R):
            first = case["mixed"] and q % 4 == 1       # a request at its first token: one beam lives
            kind.append([0 if not case["mixed"] or w == 0 else 2 if first else (1 if r.random() < 0.25 else 0) for w in range(W)])
        return kind
    lens = [case["suffix"] if q == R // 2 else max(1, int(case["suffix"] * (0.25 + 0.75 * r.random()))) for q in range(R)]
    # parents as a beam search leaves them: good beams have several children
    parents = [sorted(min(W - 1, int(W * r.random() ** 1.5)) for _ in range(W)) for _ in range(R)]
    return lens, parents


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D = case["D"] if "D" in case else 0
    if case["op"] == "prefix":
        size, pre, tails = _shape(case)
        Hq, Hk, win = case["Hq"], case["Hk"], case["window"]
        keys = dots = 0
        for g in range(len(size)):
            lows = [max(0, pre[g] + t - win) if win else 0 for t in tails[g]]
            keys += max(0, pre[g] - min(lows)) + sum(t - max(0, lo - pre[g]) for t, lo in zip(tails[g], lows))
            dots += sum(pre[g] + t - lo for t, lo in zip(tails[g], lows))
        rows = sum(size)
        return {"bytes": keys * Hk * D * 2 * es + 2 * rows * Hq * D * es + 8 * rows, "flops": 4 * D * Hq * dots}
    if case["op"] == "select":
        live = sum(k == 0 for ks in _shape(case) for k in ks)
        return {"bytes": live * case["V"] * es + case["R"] * (case["W"] * 5 + case["N"] * 13), "flops": live * case["V"] * 4}
    lens, parents = _shape(case)
    dup = [len(p) - len(set(p)) for p in parents]
    full = case["layers"].count(FULL)
    moved = sum(dup) * case["layers"].count(LINEAR) * case["Hv"] * D * D * 4 + sum(n * c for n, c in zip(lens, dup)) * full * case["Hk"] * D * 2 * es
    return {"bytes": 2 * moved + 16 * case["R"] * case["W"], "flops": 0}


# --------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, t=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=t)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=dev)

    st = {"case": case, "dt": dt}
    if case["op"] == "prefix":
        size, pre, tails = _shape(case)
        bs, Hk, D, B = case["block"], case["Hk"], case["D"], sum(size)
        at_most = (max(pre[g] + max(tails[g]) for g in range(len(size))) + bs - 1) // bs
        # whole blocks of a prefix are one group's, the rest a request's own
        ids, n, rows = 0, 0, []
        for g in range(len(size)):
            common = list(range(ids, ids + pre[g] // bs))
            ids += len(common)
            for t in tails[g]:
                mine = (pre[g] + t + bs - 1) // bs - len(common)
                rows.append(common + list(range(ids, ids + mine)) + [0] * (at_most - len(common) - mine))
                ids += mine
        NB = ids + 3
        where = shuffled(NB).to(torch.int32)
        bt = where[torch.tensor(rows, device=dev)]
        used = torch.tensor([-(-(pre[g] + t) // bs) for g in range(len(size)) for t in tails[g]], device=dev)
        st["bt"] = torch.where(torch.arange(at_most, device=dev) < used[:, None], bt, -1).contiguous()
        st["kc"], st["vc"] = (normal(NB, Hk, bs, D, t=dt) for _ in range(2))
        first = [sum(size[:g]) for g in range(len(size) + 1)]
        for g in range(len(size)):          # the prefix's tail in a block that is a request's own is the same in all of them
            if pre[g] % bs:
                own_blocks = st["bt"][first[g]:first[g + 1], pre[g] // bs].long()
                for c in (st["kc"], st["vc"]):
                    c[own_blocks, :, :pre[g] % bs] = c[own_blocks[0], :, :pre[g] % bs].clone()
        st["q"] = (1.5 * normal(B, case["Hq"], D)).to(dt)
        st["lens"] = torch.tensor([pre[g] + t for g in range(len(size)) for t in tails[g]], dtype=torch.int32, device=dev)
        st["cu"] = torch.tensor(first, dtype=torch.int32, device=dev)
        st["pre"] = torch.tensor(pre, dtype=torch.int32, device=dev)
        st["size"], st["prefixes"], st["tails"], st["B"], st["NB"] = size, pre, tails, B, NB
        st["out"] = torch.empty(B, case["Hq"], D, device=dev, dtype=dt)
    elif case["op"] == "select":
        R, W, V = case["R"], case["W"], case["V"]
        kind = torch.tensor(_shape(case), device=dev)
        rows = (3 * normal(R * W, V + case["pad"])).to(dt)
        if case["masked"]:       # banned tokens
            for part in rows.split(max(1, (1 << 24) // V)):
                part[torch.rand(part.shape, generator=gen, device=dev) < case["masked"]] = -math.inf
        st["logits"] = rows[:, :V]
        st["scores"] = torch.where(kind == 2, -math.inf, -5 - 3 * torch.rand(R, W, generator=gen, device=dev))
        st["finished"] = (kind == 1).to(torch.uint8)
        st["eos"] = V // 3
        st["s_out"] = torch.empty(R, case["N"], device=dev)
        st["parents"], st["tokens"] = (torch.empty(R, case["N"], device=dev, dtype=torch.int32) for _ in range(2))
        st["f_out"] = torch.empty(R, case["N"], device=dev, dtype=torch.uint8)
    else:
        R, W, bs, Hk, D, P = case["R"], case["W"], case["block"], case["Hk"], case["D"], case["prefix"]
        lens, parents = _shape(case)
        B = R * W
        swap = torch.stack([shuffled(W) for _ in range(R)])                 # which beam is the good one
        kids = torch.stack([torch.tensor(p, device=dev)[shuffled(W)] for p in parents])
        st["parents"] = swap.gather(1, kids).to(torch.int32)
        st["lens"] = (P + torch.tensor(lens, dtype=torch.int32, device=dev)).repeat_interleave(W)
        st["pre"] = torch.full((R,), P, dtype=torch.int32, device=dev)
        st["caches"], st["pools"], st["bt"] = [], [], None
        if FULL in case["layers"]:
            cols = (P + case["suffix"] + bs - 1) // bs + 1
            common = P // bs
            NB = R * common + B * (cols - common) + 2
            where = shuffled(NB).to(torch.int32)
            shared = where[: R * common].view(R, 1, common).expand(R, W, common).reshape(B, common)
            st["bt"] = torch.cat([shared, where[R * common: R * common + B * (cols - common)].view(B, cols - common)], 1).contiguous()
            st["NB"] = NB
        NS = B + 2
        st["NS"], st["slots"] = NS, shuffled(NS)[:B].to(torch.int32)
        for kind in case["layers"]:
            if kind == FULL:
                st["caches"].append(tuple(normal(NB, Hk, bs, D, t=dt) for _ in range(2)))
            else:
                st["pools"].append(normal(NS, case["Hv"], D, D))
    if own:   # the sizes and the workspace that a serving program keeps
        import paged_kv_linear_gb300 as hyb
        if case["op"] == "prefix":
            st["d"] = hyb.dims(Hk, D, NB, at_most, dt, block_size=bs, window=case["window"])
            st["p"] = hyb.prefix_dims(case["Hq"], len(size), max(size), max(pre), max(max(t) for t in tails))
            n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(B, st["p"], st["d"])
        elif case["op"] == "select":
            st["d"] = hyb.beam_dims(W, case["N"], V, dt, eos_token=st["eos"], row_stride=V + case["pad"])
            n = hyb.hyb_beam_select_workspace_size(R, st["d"])
        else:
            st["d"] = hyb.dims(Hk, D, st.get("NB", 1), st["bt"].shape[1] if st["bt"] is not None else 1, dt, block_size=bs)
            full, lin = iter(st["caches"]), iter(st["pools"])
            st["io"], st["types"] = [], [hyb.HYB_FULL if kind == FULL else hyb.HYB_LINEAR for kind in case["layers"]]
            for kind in case["layers"]:
                if kind == FULL:
                    k, v = next(full)
                    st["io"].append(hyb.layer_io(k_cache=k, v_cache=v))
                else:
                    st["io"].append(hyb.layer_io(state_pool=next(lin), num_state_slots=NS))
            n = hyb.hyb_beam_reorder_workspace_size(R, W)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------------------------ run
def run(st):
    return {"prefix": _run_prefix, "select": _run_select, "reorder": _run_reorder}[st["case"]["op"]](st)


def _gather(cache, blocks, at, bs):
    """Rows [.., H, D] of a paged cache at positions `at` through block numbers `blocks`."""
    return cache[blocks, :, at % bs].float()


def _run_prefix(st):
    """Per group: scores against the prefix's keys, once gathered, and against each request's own;
    one softmax over both."""
    c = st["case"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_paged_attn_decode_shared_prefix(st["out"], st["q"], st["kc"], st["vc"], st["bt"], st["lens"], st["cu"], st["pre"], st["B"], st["p"], st["d"],
                                                          st["ws"], st["ws"].numel()))
        return st["out"]
    bs, Hk, D, win = c["block"], c["Hk"], c["D"], c["window"]
    rep, dev = c["Hq"] // Hk, st["q"].device
    bt = st["bt"].long()
    outs, b0 = [], 0
    for n, P, tails in zip(st["size"], st["prefixes"], st["tails"]):
        q = st["q"][b0:b0 + n].float().view(n, Hk, rep, D) * D ** -0.5
        lens = st["lens"][b0:b0 + n].long()
        low = (lens - win).clamp(min=0) if win else torch.zeros_like(lens)
        at = torch.arange(P, device=dev)
        kp, vp = (_gather(x, bt[b0, at // bs], at, bs) for x in (st["kc"], st["vc"]))          # [P, Hk, D]
        s0 = torch.einsum("nhrd,phd->nhrp", q, kp)
        s0 = s0.masked_fill((at < low[:, None])[:, None, None], -math.inf)
        mine = P + torch.arange(max(tails), device=dev)
        there = (mine < lens[:, None]) & (mine >= low[:, None])                                # [n, S]
        blocks = torch.where(there, bt[b0:b0 + n, (mine // bs).clamp(max=bt.shape[1] - 1)], 0)
        ks, vs = (_gather(x, blocks, mine.expand(n, -1), bs) for x in (st["kc"], st["vc"]))   # [n, S, Hk, D]
        s1 = torch.einsum("nhrd,nshd->nhrs", q, ks).masked_fill(~there[:, None, None], -math.inf)
        m = torch.maximum(s0.amax(-1), s1.amax(-1))[..., None]
        p0, p1 = torch.exp(s0 - m), torch.exp(s1 - m)
        o = torch.einsum("nhrp,phd->nhrd", p0, vp) + torch.einsum("nhrs,nshd->nhrd", p1, vs)
        outs.append((o / (p0.sum(-1) + p1.sum(-1))[..., None]).reshape(n, Hk * rep, D))
        b0 += n
    return torch.cat(outs).to(st["dt"])


def _run_select(st):
    c = st["case"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_beam_select(st["s_out"], st["parents"], st["tokens"], st["f_out"], st["logits"], st["scores"], st["finished"], c["R"], st["d"],
                                      st["ws"], st["ws"].numel()))
        return {"scores": st["s_out"], "parents": st["parents"], "tokens": st["tokens"], "finished": st["f_out"]}
    R, W, N, V = c["R"], c["W"], c["N"], c["V"]
    x = st["logits"].double().view(R, W, V)
    top = x.amax(-1, keepdim=True)
    total = x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True)) + st["scores"].double()[..., None]
    done = st["finished"].bool()
    alone = torch.full((V,), -math.inf, device=x.device, dtype=torch.float64)
    alone[st["eos"]] = 0
    total = torch.where(done[..., None], alone + st["scores"].double()[..., None], total).view(R, W * V)
    best, at = torch.sort(total, dim=-1, descending=True, stable=True)       # equal ones: the lowest index first
    best, at = best[:, :N], at[:, :N]
    none = best == -math.inf
    parents = torch.where(none, -1, at // V)
    tokens = torch.where(none, -1, at % V)
    over = (done.gather(1, parents.clamp(min=0)) | (tokens == st["eos"])) & ~none
    return {"scores": best.float(), "parents": parents.to(torch.int32), "tokens": tokens.to(torch.int32), "finished": over.to(torch.uint8)}


def _run_reorder(st):
    """The first child of a beam keeps its row; the others take, in order, the rows of the beams
    without children and a copy of their parent's state and tokens."""
    c = st["case"]
    R, W = c["R"], c["W"]
    if own:
        import paged_kv_linear_gb300 as hyb
        hyb.check(hyb.hyb_beam_reorder(st["parents"], st["bt"], st["lens"], st["pre"], st["slots"], st["types"], len(st["types"]), st["io"], R, W, c["suffix"],
                                       c["Hv"] * c["D"] * c["D"], st["d"], st["ws"], st["ws"].numel()))
        return {"tables": st["bt"], "lens": st["lens"], "slots": st["slots"], "caches": [x for kv in st["caches"] for x in kv], "pools": st["pools"]}
    dev, bs = st["slots"].device, c["block"]
    par = st["parents"].long()
    same = par[:, :, None] == par[:, None, :]
    first = ~(same & torch.ones(W, W, device=dev, dtype=torch.bool).tril(-1)).any(-1)
    childless = ~(par[:, None, :] == torch.arange(W, device=dev)[:, None]).any(-1)
    # rows of childless beams in order, at the front
    free = torch.where(childless, torch.arange(W, device=dev), W).sort(-1).values
    nth = ((~first).cumsum(-1) - 1).clamp(min=0)
    seat = torch.where(first, par, free.gather(1, nth).clamp(max=W - 1))
    base = W * torch.arange(R, device=dev)[:, None]
    seat, par = (base + seat).flatten(), (base + par).flatten()
    bt, slots, lens = st["bt"], st["slots"], st["lens"]
    move = (~first).flatten().nonzero().flatten()
    for pool in st["pools"]:
        pool[slots[seat[move]].long()] = pool[slots[par[move]].long()]
    if bt is not None:
        P = st["pre"].repeat_interleave(W)[move].long()
        at = P[:, None] + torch.arange(c["suffix"], device=dev)
        which = (at < lens[par[move]][:, None]).nonzero()
        pos = at[which[:, 0], which[:, 1]]
        src, dst = (bt[rows[move][which[:, 0]], pos // bs].long() for rows in (par, seat))
        for cache in [x for kv in st["caches"] for x in kv]:
            cache[dst, :, pos % bs] = cache[src, :, pos % bs]
        bt.copy_(bt[seat])
    slots.copy_(slots[seat])
    lens.copy_(lens[par])
    return {"tables": bt, "lens": lens, "slots": slots, "caches": [x for kv in st["caches"] for x in kv], "pools": st["pools"]}


# ---------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "prefix":
        D, Hk, Hq, bs = case["D"], case["Hk"], case["Hq"], case["block"]
        lens, first = st["lens"].tolist(), st["cu"].tolist()
        if sum(lens) * Hq * D > 1 << 37 or st["B"] > 600:
            return None
        out = torch.empty(st["B"], Hq, D, dtype=torch.float64, device="cuda")

        def flat(cache, row, lo, hi):        # tokens [lo, hi) of a table row: [Hk, hi - lo, D]
            lo0 = lo // bs
            x = cache[st["bt"][row, lo0:(hi + bs - 1) // bs].long()].double().transpose(0, 1).flatten(1, 2)
            return x[:, lo - lo0 * bs:hi - lo0 * bs]

        for g in range(len(first) - 1):
            P = st["prefixes"][g]
            kp, vp = flat(st["kc"], first[g], 0, P), flat(st["vc"], first[g], 0, P)
            for b in range(first[g], first[g + 1]):
                n = lens[b]
                lo = max(0, n - case["window"]) if case["window"] else 0
                own_lo = max(P, lo)
                parts = [(kp[:, lo:], vp[:, lo:])] if lo < P else []
                parts.append((flat(st["kc"], b, own_lo, n), flat(st["vc"], b, own_lo, n)))
                q = st["q"][b].double().view(Hk, Hq // Hk, D)
                s = torch.cat([torch.bmm(q, k.transpose(1, 2)) for k, _ in parts], -1) / math.sqrt(D)
                w = torch.softmax(s, -1)
                o, done = 0, 0
                for _, v in parts:
                    o = o + torch.bmm(w[..., done:done + v.shape[1]], v)
                    done += v.shape[1]
                out[b] = o.reshape(Hq, D)
        return out
    if case["op"] == "select":
        R, W, N, V = case["R"], case["W"], case["N"], case["V"]
        scores, parents, tokens, over = [], [], [], []
        s_in, done = st["scores"].tolist(), st["finished"].tolist()
        for r in range(R):
            found = []
            for w in range(W):
                if s_in[r][w] == -math.inf:
                    continue
                if done[r][w]:
                    found.append((-s_in[r][w], w, st["eos"]))
                    continue
                x = st["logits"][r * W + w].double()
                lse = torch.logsumexp(x, 0).item()
                least = torch.topk(x, min(N, V)).values[-1]
                near = (x >= least).nonzero().flatten()
                near = sorted(zip((-x[near]).tolist(), near.tolist()))[:N]
                found += [(-(s_in[r][w] - lse) + y, w, v) for y, v in near if y < math.inf]
            found = sorted(found)[:N]
            found += [(math.inf, -1, -1)] * (N - len(found))
            scores.append([-f[0] for f in found])
            parents.append([f[1] for f in found])
            tokens.append([f[2] for f in found])
            over.append([int(w >= 0 and (bool(done[r][w]) or v == st["eos"])) for _, w, v in found])
        dev = "cuda"
        return {"scores": torch.tensor(scores, dtype=torch.float64, device=dev), "parents": torch.tensor(parents, dtype=torch.int32, device=dev),
                "tokens": torch.tensor(tokens, dtype=torch.int32, device=dev), "finished": torch.tensor(over, dtype=torch.uint8, device=dev)}
    R, W, bs = case["R"], case["W"], case["block"]
    par, lens, slots = st["parents"].tolist(), st["lens"].tolist(), st["slots"].tolist()
    tables = st["bt"].tolist() if st["bt"] is not None else None
    new_lens, new_slots, new_tables, copies = [], [], [], []
    for r in range(R):
        unused = [w for w in range(W) if w not in par[r]]
        taken = set()
        for w in par[r]:
            old, kept = r * W + w, w not in taken
            seat = old if kept else r * W + unused.pop(0)
            taken.add(w)
            if not kept:
                copies.append((old, seat))
            new_lens.append(lens[old])
            new_slots.append(slots[seat])
            if tables:
                new_tables.append(tables[seat])
    pools, caches = [x.double() for x in st["pools"]], []
    for x in pools:
        for old, seat in copies:
            x[slots[seat]] = x[slots[old]]
    tokens = [(tables[old][p // bs], tables[seat][p // bs], p % bs) for old, seat in copies for p in range(case["prefix"], lens[old])] if tables else []
    src, dst, off = (torch.tensor(t, device="cuda") for t in zip(*tokens)) if tokens else (None, None, None)
    for x in [x for kv in st["caches"] for x in kv]:
        y = x.double()
        if tokens:
            y[dst, :, off] = y[src, :, off]
        caches.append(y)
    as_int = {"dtype": torch.int32, "device": "cuda"}
    return {"tables": torch.tensor(new_tables, **as_int) if tables else None, "lens": torch.tensor(new_lens, **as_int), "slots": torch.tensor(new_slots, **as_int),
            "caches": caches, "pools": pools}
