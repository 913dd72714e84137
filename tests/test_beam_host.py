"""Refusals of shared-prefix attention, beam selection and beam reordering before anything is
launched (no GPU), and pins of their 64-bit test forms."""
import ctypes as C
import math

import pytest
import torch

import beam_ref as R

F = 1 << 20      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def hyb():
    from paged_kv_linear_gb300 import _build
    _build.build()
    import paged_kv_linear_gb300 as hyb
    return hyb


def test_struct_sizes_match_the_header(hyb):
    assert C.sizeof(hyb.hyb_prefix_dims_t) == 20 and C.sizeof(hyb.hyb_beam_dims_t) == 32


def test_prefix_refused(hyb):
    inv, uns, ok = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_OK
    ws = 1 << 30

    def call(d=None, p=None, B=6, ws=F, nb=ws, a=(F,) * 8):
        d = hyb.dims(**{**dict(num_heads=4, head_dim=128, num_blocks=10, max_blocks_per_seq=64), **(d or {})})
        p = hyb.prefix_dims(**{**dict(num_q_heads=8, num_groups=2, max_group=4, max_prefix_len=512, max_suffix_len=64), **(p or {})})
        st = hyb.hyb_paged_attn_decode_shared_prefix(*a, B, p, d, ws, nb, 0)
        if st != ok:
            n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(B, p, d)
            assert n == 0 or a != (F,) * 8 or ws != F or nb < n
        return st

    assert call(B=0, a=(None,) * 8, ws=None, nb=0, p=dict(max_group=0)) == ok
    assert call(p=dict(num_groups=0), a=(None,) * 8, ws=None, nb=0) == ok
    assert call(B=-1) == inv
    for name in ("num_groups", "max_group", "max_prefix_len", "max_suffix_len"):
        assert call(p={name: -1}) == inv, name
    assert call(p=dict(num_q_heads=0)) == inv and call(p=dict(num_q_heads=6)) == inv and call(p=dict(num_q_heads=-4)) == inv
    assert call(p=dict(max_prefix_len=1025)) == inv and call(p=dict(max_suffix_len=1025)) == inv     # 64 blocks of 16
    assert call(p=dict(max_group=7)) == inv                                                          # of 6 requests
    assert call(d=dict(max_blocks_per_seq=1 << 21), p=dict(max_prefix_len=(1 << 24) + 1)) == uns
    assert call(B=65536, p=dict(max_group=4)) == uns and call(B=65535, p=dict(num_q_heads=256)) == uns
    assert call(p=dict(num_groups=65542)) == uns
    assert call(d=dict(head_dim=48, scale=1.0)) == uns and call(d=dict(dtype=hyb.HYB_F16)) == inv and call(d=dict(block_size=24)) == uns
    assert call(d=dict(head_dim=256, dtype=hyb.HYB_F32)) == uns
    assert call(d=dict(window=-1)) == inv and call(d=dict(scale=math.nan)) == inv
    for i in range(8):
        assert call(a=(F,) * i + (None,) + (F,) * (7 - i)) == inv, i
        assert call(a=(F,) * i + (F + 2,) + (F,) * (7 - i)) == inv, i
    n = hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(6, hyb.prefix_dims(8, 2, 4, 512, 64), hyb.dims(4, 128, 10, 64))
    assert n > 0
    assert call(ws=None) == inv and call(ws=F + 8) == inv and call(nb=n - 1) == inv
    d, p = hyb.dims(4, 128, 10, 64), hyb.prefix_dims(8, 2, 4, 512, 64)
    for pp, dd in ((None, d), (p, None), (None, None)):
        assert hyb.hyb_paged_attn_decode_shared_prefix(*(F,) * 8, 6, pp, dd, F, ws, 0) == inv
        assert hyb.hyb_paged_attn_decode_shared_prefix_workspace_size(6, pp, dd) == 0


def test_select_refused(hyb):
    inv, uns, ok = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_OK

    def call(R=3, ws=F, nb=1 << 30, a=(F, F, F, F, F, F + 4096, None), **kw):
        d = hyb.beam_dims(**{**dict(num_beams=4, num_out=8, vocab=1000), **kw})
        return hyb.hyb_beam_select(*a, R, d, ws, nb, 0)

    assert call(R=0, a=(None,) * 7, ws=None, nb=0) == ok
    assert call(R=-1) == inv
    for name in ("num_beams", "num_out", "vocab"):
        assert call(**{name: 0}) == inv and call(**{name: -3}) == inv
    assert call(num_out=5, vocab=1) == inv                       # more than there are candidates
    assert call(num_beams=129) == uns and call(num_out=129) == uns
    assert call(num_beams=1, vocab=(1 << 30) + 1) == uns
    assert call(num_beams=100, vocab=1 << 25) == uns and call(R=1 << 19) == uns
    assert call(dtype=hyb.HYB_F16) == inv and call(eos_token=1000) == inv and call(eos_token=-2) == inv
    assert call(row_stride=999) == inv and call(row_stride=-1) == inv and call(row_stride=1 << 41) == uns
    for i in (0, 1, 2, 4, 5):
        a = [F, F, F, F, F, F + 4096, None]
        assert call(a=a[:i] + [None] + a[i + 1:]) == inv, i
        assert call(a=a[:i] + [a[i] + 2] + a[i + 1:]) == inv, i
    assert call(a=(F, F, F, F, F, F + 4096, F)) == inv           # finished without an eos token
    assert call(a=(F, F, F, F, F, F, None)) == inv               # in place with another number of beams
    assert call(a=(F, F, F, F, F, F + 4096, F), eos_token=1) == inv
    n = hyb.hyb_beam_select_workspace_size(3, hyb.beam_dims(4, 8, 1000))
    assert n > 0 and hyb.hyb_beam_select_workspace_size(0, hyb.beam_dims(4, 8, 1000)) == 0
    assert call(ws=None) == inv and call(ws=F + 8) == inv and call(nb=n - 1) == inv
    assert hyb.hyb_beam_select(F, F, F, F, F, F + 4096, None, 3, None, F, 1 << 30, 0) == inv
    assert hyb.hyb_beam_select_workspace_size(3, None) == 0


def test_reorder_refused(hyb):
    inv, uns, ok = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_OK
    full = hyb.layer_io(k_cache=F, v_cache=2 * F)
    lin = hyb.layer_io(state_pool=3 * F, num_state_slots=9)

    def call(parents=F, bt=F, lens=F, pre=F, slots=F, types=(0, 1), io=(full, lin), L=None, R=2, W=4, most=64, size=128, ws=F, nb=1 << 20, **kw):
        d = hyb.dims(**{**dict(num_heads=4, head_dim=128, num_blocks=10, max_blocks_per_seq=64), **kw})
        return hyb.hyb_beam_reorder(parents, bt, lens, pre, slots, types, len(types) if L is None else L, io, R, W, most, size, d, ws, nb, 0)

    assert call(R=0, parents=None, bt=None, lens=None, pre=None, slots=None, ws=None, nb=0) == ok
    assert call(R=-1) == inv and call(W=0) == inv and call(W=-1) == inv and call(most=-1) == inv and call(L=-1) == inv
    assert call(W=129) == uns and call(R=20000) == uns
    assert call(parents=None) == inv and call(bt=None) == inv and call(lens=None) == inv and call(slots=None) == inv
    for name in ("parents", "bt", "lens", "pre", "slots"):
        assert call(**{name: F + 2}) == inv, name
    assert call(types=(0, 3)) == inv and call(types=(2, 1)) == inv and call(types=(1, 0)) == inv
    assert call(io=(hyb.layer_io(k_cache=F, v_cache=F), lin)) == inv
    assert call(io=(hyb.layer_io(k_cache=F, v_cache=3 * F), lin)) == inv
    assert call(io=(hyb.layer_io(k_cache=F + 8, v_cache=2 * F), lin)) == inv
    assert call(io=(hyb.layer_io(k_cache=F), lin)) == inv
    assert call(io=(hyb.layer_io(k_cache=F, v_cache=2 * F, window=5), lin)) == inv
    assert call(io=(full, hyb.layer_io(state_pool=3 * F))) == inv
    assert call(io=(full, hyb.layer_io(state_pool=3 * F + 8, num_state_slots=9))) == inv
    assert call(size=0) == inv and call(size=126) == inv and call(size=1 << 40) == uns
    assert call(window=4) == inv and call(block_size=24) == uns and call(num_heads=0) == inv
    assert hyb.hyb_beam_reorder_workspace_size(2, 4) == 0
    assert hyb.hyb_beam_reorder(F, F, F, F, F, (0, 1), 2, (full, lin), 2, 4, 64, 128, None, F, 1 << 20, 0) == inv


def test_logits_of_another_stride_refused_by_the_binding(hyb):
    class Fake:
        is_cuda = True
        shape = (3, 100)

        def __init__(self, strides):
            self.s = strides

        def dim(self):
            return 2

        def stride(self):
            return self.s

        def data_ptr(self):
            return F

    assert hyb._logits(Fake((128, 1)), 128) == F
    for s in ((100, 1), (128, 2)):
        with pytest.raises(hyb.HybError):
            hyb._logits(Fake(s), 128)


# ----------------------------------------------------------------- pins of the 64-bit forms
def test_attention_pins():
    torch.manual_seed(0)
    bs, Hk, D = 16, 2, 8
    kc, vc = torch.randn(6, Hk, bs, D), torch.randn(6, Hk, bs, D)
    q = torch.randn(3, 4, D)
    bt = torch.tensor([[4, 1, 0], [-1, 2, 3], [-1, 5, -1]])
    # 20 common tokens: the block of the last four is each row's own
    for c in (kc, vc):
        c[2, :, :4] = c[5, :, :4] = c[1, :, :4]
    out, mag, _, n = R.attention(q, kc, vc, bt, [40, 33, 20], [0, 3], [20], 0.5)
    assert n.flatten().tolist() == [40, 33, 20]
    for b, blocks in enumerate([[4, 1, 0], [4, 2, 3], [4, 5]]):
        k, v = (torch.cat([x[i] for i in blocks], 1)[:, :[40, 33, 20][b]].double().repeat_interleave(2, 0) for x in (kc, vc))
        want = torch.nn.functional.scaled_dot_product_attention(q[b].double()[:, None], k, v, scale=0.5)[:, 0]
        assert torch.allclose(out[b], want) and (mag[b] >= out[b].abs()).all()
    # one key: its value; none: zeros; rows of no group: NaN
    out, *_ = R.attention(q, kc, vc, bt, [1, 0, 5], [0, 2], [20], 0.5)
    assert torch.allclose(out[0], vc[4, :, 0].double().repeat_interleave(2, 0)) and (out[1] == 0).all() and out[2].isnan().all()
    # a window of one: the newest token's value
    out, *_ = R.attention(q, kc, vc, bt, [40, 33, 20], [0, 3], [20], 0.5, window=1)
    assert torch.allclose(out[1], vc[3, :, 0].double().repeat_interleave(2, 0))


def test_select_pins():
    x = torch.tensor([[[0.0, 1.0, 1.0], [5.0, -math.inf, 4.0]]])
    s, p, t, f = R.select(x, torch.tensor([[0.0, -1.0]]), None, -1, 6)
    assert p == [[0, 0, 1, 0, 1, -1]] and t == [[1, 2, 0, 0, 2, -1]] and s[0][5] == -math.inf
    assert abs(sum(math.exp(v) for v, w in zip(s[0], p[0]) if w == 0) - 1) < 1e-12
    assert abs(sum(math.exp(v + 1) for v, w in zip(s[0], p[0]) if w == 1) - 1) < 1e-12
    s, p, t, f = R.select(x, torch.tensor([[-0.5, -9.0]]), torch.tensor([[1, 0]]), 2, 2)
    assert s[0][0] == -0.5 and (p, t, f) == ([[0, 1]], [[2, 0]], [[1, 0]])
    assert R.select(x, torch.tensor([[-math.inf, -math.inf]]), None, -1, 1)[1] == [[-1]]


def test_seat_pins():
    assert R.seats([0, 1, 2]) == ([0, 1, 2], [None] * 3)
    assert R.seats([2, 2, 0]) == ([2, 1, 0], [None, 2, None])
    assert R.seats([1, 1, 1, -1]) == ([1, 0, 2, 3], [None, 1, 1, None])
