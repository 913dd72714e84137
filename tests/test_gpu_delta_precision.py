"""How near the gated delta rule's tensor-core prefill (bf16, D = 128) comes to the 64-bit recurrence where
an error of its operands would add up: keys that repeat, states that are only slowly lost, outputs."""
import math

import numpy as np
import pytest
import torch

import layer_ops_ref as R
from test_gpu_delta import EPS, Case, host, prefill

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = 64          # rows of a chunk


def one_request(hyb, c):
    out = torch.empty(c.T, c.Hv, c.D, device="cuda", dtype=c.dt)
    prefill(hyb, c, out, torch.tensor([0, c.T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), None)
    return out


@pytest.mark.parametrize("dims", [1, 2])
@pytest.mark.parametrize("T", [64, 1024])
def test_keys_of_few_dimensions(hyb, dims, T):
    """Keys of one or two dimensions, beta 1, no decay: the corrections' system is as far from the
    identity as it gets, and what its inverse W is off by adds up over the rows of a chunk. (One key:
    every entry of A is the same number near 1, and what cutting its tf32 terms loses has one sign in
    all 2016 entries below the diagonal.) Each chunk replaces the keys' dimensions of the state and
    changes no others, so the error is the last chunk's. Allowed, as norms over all heads:
      * 1.5 times what the recurrence is off by in fp32 on the same numbers (fp32 rows take it). The 1.5
        is for chance: 16 heads x 128 columns carry the error, a spread of 2 %.
      * the tensor core's fp32 sums, which cut to 24 bits instead of rounding: each cut takes half a
        unit on average, at most u = 2^-24 of the sum. With S the state at the chunk's start, R = V - K S
        and X = W R, the sums are of full size from the first half's largest terms on: 16 cuts of K S
        (4 products, then 12), 14 of X (2 and 12), 8 of the change K^T X (2 and 6). In the state that is
        u (16 |K^T W K S| + 22 |K^T X|).
    So nothing is left for W."""
    H = 16
    c = Case(30 + dims, T, H, H, 128, torch.bfloat16, 1, gate="none")
    if dims == 1:                          # a dense key for each head, the same at every row
        c.k = c.k[:1].expand(T, -1, -1).contiguous()
    else:
        c.k[..., 2:] = 0
    c.beta.fill_(1.0)
    start = c.pool.clone()
    last = T - C
    S = c.ref(slice(0, last), host(start)[0])[1] if last else host(start)[0]
    want = c.ref(slice(last, T), S)[1]
    k, v = host(c.k)[last:], host(c.v)[last:]
    k = k / np.sqrt((k * k).sum(-1, keepdims=True) + EPS)
    cuts = 0.0
    for h in range(H):
        K = k[:, h]
        W = np.linalg.inv(np.eye(C) + np.tril(K @ K.T, -1))
        removed, change = K.T @ W @ K @ S[h], K.T @ W @ (v[:, h] - K @ S[h])
        cuts += (U * (16 * np.linalg.norm(removed) + 22 * np.linalg.norm(change))) ** 2
    one_request(hyb, c)
    got = host(c.pool)[0]
    c.pool.copy_(start)
    c.q, c.k, c.v, c.dt = c.q.float(), c.k.float(), c.v.float(), torch.float32
    one_request(hyb, c)
    here, fp32 = (np.linalg.norm(x - want) / np.linalg.norm(want) for x in (got, host(c.pool)[0]))
    cuts = math.sqrt(cuts) / np.linalg.norm(want)
    print(f"dims {dims} T {T}: {here:.2e}, fp32 recurrence {fp32:.2e}, cuts {cuts:.2e}")
    assert here <= 1.5 * fp32 + cuts


@pytest.mark.parametrize("gate", [-1e-2, -1e-3, -3e-4, -1e-4, -1e-5])
def test_slow_decay_does_not_drift(hyb, gate):
    """With beta 0 a state only fades, by the same e^(64 g) in every chunk. Applied as S + (e^(64 g) -
    1) S a chunk rounds the state once (at most u of an element, of either sign: in squares over the
    chunks), and e^(64 g) - 1 is off by 3 u of itself (its argument by u, the function by 2 u), alike
    in all of them. e^(64 g) rounded would be off by up to u (more with the function's own error),
    alike in all of them: 128 u here."""
    T = 8192
    n = T // C
    c = Case(32, T, 1, 1, 128, torch.bfloat16, 1, gate="none")
    c.g.fill_(gate)
    c.beta.zero_()
    S0 = host(c.pool)[0, 0]
    one_request(hyb, c)
    ref = S0 * math.exp(float(c.g[0, 0]) * T)
    err = np.linalg.norm(host(c.pool)[0, 0] - ref) / np.linalg.norm(ref)
    lim = U * (math.sqrt(n) + 3 * n * abs(math.expm1(C * float(c.g[0, 0]))))
    print(f"gate {gate}: {err:.2e} of {lim:.2e}")
    assert err <= lim


def test_outputs_next_to_the_rounded_value(hyb):
    """Outputs are products of two bf16 terms each of S, X and P, so some come out on the other side of
    a bf16 rounding than the exact value. How many is a matter of those terms alone:
      * a number less its two terms, each rounded to nearest, is off by the product of two roundings:
        uniform in half a unit of 8 bits, 2^-7 / sqrt(12) of the number's power of two, and with the
        mantissa's own spread (mean of its inverse square 0.541) 2^-9.24 of the number each, so
        e = 2^-18.47 in the mean of squares. The product of second terms that is left out is another e.
      * an element o = scale (e^G q S + P X) is then off by s = scale e sqrt(e^2G sum (q_i S_i)^2 +
        3 sum (P X)^2) in the mean of squares, and normally distributed as a sum of many: 0.8 s in the
        mean. It ends on the other side with a probability of that by the unit of 8 bits at o.
    The limit is 1.4 times that mean: the recurrence's own fp32 share is a tenth of it, chance (some
    thousand elements) 2 %, terms of one sign only twice to four times as large."""
    T, H, D = 512, 8, 128
    c = Case(33, T, H, H, D, torch.bfloat16, 1, gate="none")
    c.g = -0.05 * torch.rand(T, H, generator=c.gen, device="cuda")
    S = host(c.pool)[0]
    q, k, v, g, beta = (host(x) for x in (c.q, c.k, c.v, c.g, c.beta))
    got = host(one_request(hyb, c))
    q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + EPS) for x in (q, k))
    scale, e = D ** -0.5, 2.0 ** -18.47
    other, expected = 0, 0.0
    for t0 in range(0, T, C):
        r = slice(t0, t0 + C)
        ref, S1, _, _ = c.ref(r, S)
        for h in range(H):
            G = np.cumsum(g[r, h])
            fade = np.tril(np.exp(np.minimum(G[:, None] - G[None, :], 0)))
            K, Q = k[r, h], q[r, h] * np.exp(G)[:, None]
            A = np.tril(beta[r, h][:, None] * fade * (K @ K.T), -1)
            X = np.linalg.solve(np.eye(C) + A, beta[r, h][:, None] * (v[r, h] - np.exp(G)[:, None] * (K @ S[h])))
            P = fade * (q[r, h] @ K.T)
            o = scale * (Q @ S[h] + P @ X)
            assert np.abs(o - ref[:, h]).max() < 1e-12
            s = scale * e * np.sqrt((Q * Q) @ (S[h] * S[h]) + 3 * (P * P) @ (X * X))
            unit = 2.0 ** (np.floor(np.log2(np.abs(o))) - 7)
            expected += np.minimum(0.8 * s / unit, 1).sum()
            other += (got[r, h] != R.bf16(o.astype(np.float32))).sum()
        S = S1
    print(f"{other} of {T * H * D}, {expected:.0f} expected")
    assert other <= 1.4 * expected
