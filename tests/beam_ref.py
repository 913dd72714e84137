"""Plain 64-bit forms of shared-prefix decode attention, beam selection and beam reordering, from
the definitions in include/hyb.h, on torch tensors of any device. Shares no code with the library.

Tolerances of the checks built on them (derived, not tuned). u = 2^-24 is fp32's rounding.
  * Attention. With w the softmax weights, an output is a sum of w_p v_p, and an error of a weight's
    relative size r costs at most r * mag, mag = sum w_p |v_p|. Weights are off by their
    score's error (a sum of D products in fp32, at most D u a with a = scale * sum |q_i k_i|, and the same for
    the sum of the weights: twice that), by the exponential (2^-22), and for bf16 by
    being rounded to bf16 for the tensor core, 2^-8. Sums of n terms in fp32: 4 u sqrt(n) where they are rounded,
    and (n / 16) 2^-23 more where the tensor core cuts them (bf16). Then half a step of the output's type.
  * Selection. The sum over the vocabulary has terms off by 2^-22 (exponential) and 20 u (the
    argument, as weighted) and some 24 roundings on a term's way through the sum: 48 u <
    2^-18 of the sum, so 2^-18 of the score in absolute terms, and its final rounding, u relative.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def attention(q, kc, vc, bt, lens, cu, pre, scale, window=0):
    """-> (out, mag, a, n): [B][Hq][D] twice and the rows' largest a and their keys. Rows of no group: NaN. Bad block
    ids (negative): their tokens are left out."""
    B, Hq, D = q.shape
    Hk, bs = kc.shape[1], kc.shape[2]
    rep = Hq // Hk
    out = torch.full((B, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    mag, a = torch.zeros_like(out), torch.zeros(B, Hq, 1, dtype=torch.float64, device=q.device)
    num = torch.zeros(B, 1, 1, dtype=torch.float64, device=q.device)
    for g in range(len(pre)):
        for b in range(cu[g], cu[g + 1]):
            n = max(0, lens[b])
            at = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
            rows = torch.where(at < pre[g], cu[g], b)
            blk = bt[rows, at // bs].long() if n else at
            at, blk = at[blk >= 0], blk[blk >= 0]
            if not len(at):
                out[b] = 0
                continue
            k, v = (x[blk, :, at % bs].double().repeat_interleave(rep, 1) for x in (kc, vc))       # [n, Hq, D]
            x = q[b].double()
            s = torch.einsum("hd,phd->hp", x, k) * scale
            w = torch.softmax(s, -1)
            out[b] = torch.einsum("hp,phd->hd", w, v)
            mag[b] = torch.einsum("hp,phd->hd", w, v.abs())
            a[b] = (torch.einsum("hd,phd->hp", x.abs(), k.abs()) * abs(scale)).amax(-1, keepdim=True)
            num[b] = len(at)
    return out, mag, a, num


def check_attention(got, ref, dtype, what=""):
    out, mag, a, n = ref
    D = got.shape[-1]
    rel = 2 * D * U * a + 2.0 ** -22 + 4 * U * n.sqrt()
    if dtype == torch.bfloat16:
        rel = rel + 2.0 ** -8 + n / 16 * 2.0 ** -23
    lim = HALF[dtype] * out.abs() * (1 + 2.0 ** -6) + rel * mag * (1 + 2.0 ** -6) + 1e-30
    live = ~out.isnan()
    err = (got.double() - out).abs()
    assert got[live].isfinite().all(), what
    bad = (err > lim) & live
    worst = torch.where(live, err / lim, 0).max().item()
    assert not bad.any(), f"{what}: {worst:.2f} of the limit at {bad.nonzero()[0].tolist()}"
    if dtype == torch.bfloat16:
        # roundings of many weights are independent: a row's error stays a few steps of bf16 of the row's largest value
        size = torch.where(live, out, 0).abs().amax(-1)
        assert (torch.where(live, err, 0).amax(-1) <= 2.0 ** -6 * size + 1e-30).all(), what
    return worst


def select(logits, scores, finished, eos, N):
    """logits [R][W][V], scores [R][W] -> (scores, parents, tokens, finished) as lists."""
    R, W, V = logits.shape
    res = []
    for r in range(R):
        found = []
        for w in range(W):
            s = float(scores[r, w])
            if not math.isfinite(s):
                continue
            if finished is not None and finished[r, w]:
                found.append((-s, w, eos))
                continue
            x = logits[r, w].double()
            if x.isnan().any() or (x == math.inf).any() or (x == -math.inf).all():
                continue
            x = x - torch.logsumexp(x, 0)
            order = torch.sort(x, descending=True, stable=True).indices[:N].tolist()
            found += [(-(s + float(x[v])), w, v) for v in order if float(x[v]) > -math.inf]
        found = sorted(found)[:N]
        found += [(math.inf, -1, -1)] * (N - len(found))
        res.append([(-t, w, v, int(w >= 0 and ((finished is not None and bool(finished[r, w])) or v == eos))) for t, w, v in found])
    return tuple([[c[i] for c in row] for row in res] for i in range(4))


def check_select(got, ref, what=""):
    s, p, t, f = (x.cpu() for x in got)
    assert p.tolist() == ref[1], what
    assert t.tolist() == ref[2], what
    assert f.tolist() == ref[3], what
    want = torch.tensor(ref[0], dtype=torch.float64)
    none = want == -math.inf
    assert (s.double()[none] == -math.inf).all(), what
    lim = 2.0 ** -18 + U * want.abs()
    assert ((s.double() - want).abs()[~none] <= lim[~none]).all(), what


def seats(parents):
    """One request: (row that each beam gets, beam to copy from or None)."""
    W = len(parents)
    free = [w for w in range(W) if w not in parents]
    heir, rows, copy = {}, [], []
    for i, p in enumerate(parents):
        if p >= 0 and p not in heir:
            heir[p] = i
            rows.append(p)
            copy.append(None)
        else:
            rows.append(free.pop(0))
            copy.append(p if p >= 0 else None)
    return rows, copy
