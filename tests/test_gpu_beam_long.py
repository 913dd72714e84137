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
            y = y - torch.logsumexp(y, 0)
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
