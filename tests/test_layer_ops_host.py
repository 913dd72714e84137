"""Refusals of the gated delta rule's and the query/key preparation's entry points, before
anything is launched (no GPU), and pins of their 64-bit test forms."""
import ctypes as C

import numpy as np
import pytest

import layer_ops_ref as R

F = 1 << 20      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def hyb():
    from paged_kv_linear_gb300 import _build
    _build.build()
    import paged_kv_linear_gb300 as hyb
    return hyb


def test_struct_sizes_match_the_header(hyb):
    assert C.sizeof(hyb.hyb_delta_dims_t) == 48 and C.sizeof(hyb.hyb_rope_dims_t) == 48


def test_delta_dims_refused(hyb):
    inv, uns = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED
    ok = dict(num_qk_heads=2, num_v_heads=4, head_dim=128)

    def both(want, **kw):
        d = hyb.delta_dims(**{**ok, **kw})
        assert hyb.hyb_gated_delta_step(F, F, F, F, F, F, F, 4, F, 2, d, 0) == want, kw
        assert hyb.hyb_gated_delta_chunked_prefill(F, F, F, F, F, F, F, F, 4, F, None, 2, 64, 32, d, F, 1 << 16, 0) == want, kw
        assert hyb.hyb_gated_delta_chunked_prefill_workspace_size(2, 64, d) == 0

    both(inv, num_qk_heads=0)
    both(inv, num_v_heads=0)
    both(inv, num_v_heads=3)                       # no multiple of the query/key heads
    both(inv, head_dim=0, scale=1.0)
    for D in (8, 48, 96, 512):
        both(uns, head_dim=D, scale=1.0)
    both(uns, num_qk_heads=1, num_v_heads=65536)
    both(inv, dtype=hyb.HYB_F16)
    both(inv, dtype=7)
    both(inv, scale=float("nan"))
    both(inv, qk_norm_eps=-1.0)
    both(inv, qk_norm_eps=float("inf"))
    both(inv, qk_norm_eps=float("nan"))
    both(inv, q_stride=248)                        # less than a row
    both(inv, k_stride=260)                        # no multiple of 16 bytes
    both(inv, v_stride=-512)


def test_delta_arguments_refused(hyb):
    inv, uns, ok = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_OK
    d = hyb.delta_dims(2, 4, 128)
    step = lambda a=(F,) * 7, NS=4, sl=F, B=2: hyb.hyb_gated_delta_step(*a, NS, sl, B, d, 0)
    for i in range(7):
        assert step(a=(F,) * i + (None,) + (F,) * (6 - i)) == inv, i
        assert step(a=(F,) * i + (F + 2,) + (F,) * (6 - i)) == inv, i
    assert step(sl=None) == inv and step(sl=F + 2) == inv and step(NS=0) == inv and step(B=-1) == inv
    assert step(B=65536) == uns and step(B=0, a=(None,) * 7, sl=None) == ok
    n = hyb.hyb_gated_delta_chunked_prefill_workspace_size(2, 64, d)
    assert n > 0
    assert hyb.hyb_gated_delta_chunked_prefill_workspace_size(0, 64, d) == 0
    pre = lambda cu=F, B=2, T=64, ml=32, ws=F, nb=n, sl=F, NS=4: hyb.hyb_gated_delta_chunked_prefill(
        F, F, F, F, F, F, cu, F, NS, sl, None, B, T, ml, d, ws, nb, 0)
    assert pre(cu=None) == inv and pre(cu=F + 2) == inv and pre(T=-1) == inv
    assert pre(ml=-1) == inv and pre(ml=65) == inv
    assert pre(ws=None) == inv and pre(ws=F + 4) == inv and pre(nb=n - 1) == inv
    assert pre(B=65536) == uns and pre(NS=0) == inv and pre(sl=None) == inv
    assert pre(B=0, ws=None, nb=0) == ok
    # more chains than the work split counts
    many = hyb.delta_dims(1, 65535, 128)
    assert hyb.hyb_gated_delta_step(*(F,) * 7, 4, F, 65535, many, 0) == uns
    # rows may be missing only where there are none
    rows = lambda T: hyb.hyb_gated_delta_chunked_prefill(None, F, F, F, F, F, F, F, 4, F, None, 2, T, 0, d, F, n, 0)
    assert rows(1) == inv


def test_rope_refused(hyb):
    inv, uns, ok = hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_OK

    def call(d=None, r=None, **kw):
        a = dict(q_out=F, k_out=None, q=F, k=F, v=F, pos=F, slot=F, f=F, qw=F, kw=F, T=4, kc=F, vc=F + 4096)
        a.update(kw)
        d = hyb.dims(**{**dict(num_heads=4, head_dim=128, num_blocks=10, max_blocks_per_seq=4), **(d or {})})
        r = hyb.rope_dims(**{**dict(num_q_heads=8, rot_dim=128), **(r or {})})
        return hyb.hyb_qk_norm_rope_append(a["q_out"], a["k_out"], a["q"], a["k"], a["v"], a["pos"], a["slot"], a["f"], a["qw"], a["kw"], a["T"], a["kc"], a["vc"], r, d, 0)

    assert call(T=0) == ok
    assert call(T=-1) == inv
    assert call(d=dict(head_dim=48, scale=1.0)) == uns and call(d=dict(head_dim=512, scale=1.0)) == uns
    assert call(d=dict(block_size=24)) == uns and call(d=dict(num_heads=0)) == inv and call(d=dict(dtype=hyb.HYB_F16)) == inv
    assert call(r=dict(rot_dim=-8)) == inv and call(r=dict(rot_dim=136)) == inv and call(r=dict(rot_dim=12)) == uns
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(r=dict(eps=eps)) == inv
    assert call(r=dict(weight_offset=float("nan"))) == inv and call(r=dict(attn_factor=float("inf"))) == inv
    assert call(r=dict(q_stride=1016)) == inv and call(r=dict(k_stride=516)) == inv and call(r=dict(v_stride=-1)) == inv
    for name in ("q_out", "q", "k", "v", "pos", "slot", "f", "kc", "vc"):
        assert call(**{name: None}) == inv, name
    for name in ("q_out", "q", "k", "v", "kc", "vc", "slot"):
        assert call(**{name: F + 4}) == inv, name
    for name in ("pos", "f", "qw", "kw"):
        assert call(**{name: F + 2}) == inv, name
    assert call(vc=F) == inv                                       # one pool as K and V
    assert call(kc=None, vc=None, slot=None) == inv                # k would go nowhere
    assert call(r=dict(num_q_heads=0)) == inv                      # q_out without queries
    assert call(q_out=F, q=F, r=dict(q_stride=2048)) == inv        # in place on rows of another stride
    assert call(k_out=F, k=F, r=dict(k_stride=2048)) == inv
    assert call(r=dict(num_q_heads=-1)) == inv


def test_rows_of_another_stride_refused_by_the_binding(hyb):
    class Fake:                                                    # what _rows asks of a tensor
        is_cuda = True
        shape = (3, 4, 128)

        def __init__(self, strides):
            self.s = strides

        def stride(self):
            return self.s

        def data_ptr(self):
            return F

    assert hyb._rows(Fake((2048, 128, 1)), 2048) == F
    for s in ((1024, 128, 1), (2048, 256, 1), (2048, 128, 2)):
        with pytest.raises(hyb.HybError):
            hyb._rows(Fake(s), 2048)


def test_missing_dims_refused(hyb):
    """Through the binding too, as its other calls do: a status, not a Python error."""
    inv = hyb.HYB_ERR_INVALID_ARG
    assert hyb.hyb_gated_delta_step(*(F,) * 7, 4, F, 2, None, 0) == inv
    assert hyb.hyb_gated_delta_chunked_prefill(*(F,) * 8, 4, F, None, 2, 64, 32, None, F, 1 << 16, 0) == inv
    d, r = hyb.dims(4, 128, 10, 4), hyb.rope_dims(8, 128)
    for rr, dd in ((None, d), (r, None), (None, None)):
        assert hyb.hyb_qk_norm_rope_append(F, None, *(F,) * 8, 4, F, F + 4096, rr, dd, 0) == inv


def test_more_rows_than_the_kernels_count_refused(hyb):
    d = hyb.delta_dims(2, 4, 128)
    for dims in (d, hyb.delta_dims(2, 4, 64), hyb.delta_dims(2, 4, 16, hyb.HYB_F32)):
        for T in (2 ** 31 - 64, 2 ** 31 - 1):
            for max_len in (8, T):
                assert hyb.hyb_gated_delta_chunked_prefill(*(F,) * 8, 4, F, None, 2, T, max_len, dims, F, 1 << 16, 0) == hyb.HYB_ERR_UNSUPPORTED


# ----------------------------------------------------------------- pins of the 64-bit forms
def test_delta_rule_pins():
    rs = np.random.RandomState(0)
    q, k, v = rs.randn(1, 1, 4), rs.randn(1, 1, 4), rs.randn(1, 1, 4)
    # a zero state and one token: beta k v^T
    o, S, _, _ = R.delta_rule(q, k, v, np.array([[-0.5]]), np.array([[0.25]]), np.zeros((1, 4, 4)), 2.0, 0.0)
    assert np.allclose(S[0], 0.25 * np.outer(k[0, 0], v[0, 0])) and np.allclose(o[0, 0], 2 * q[0, 0] @ S[0])
    # beta 1 and a unit key: the state answers that key with v, whatever it held
    o, S, _, _ = R.delta_rule(k, k, v, np.array([[-0.1]]), np.array([[1.0]]), rs.randn(1, 4, 4), 1.0, 1e-30)
    assert np.allclose(o[0, 0], v[0, 0])
    # beta 0: only the decay
    S0 = rs.randn(1, 4, 4)
    _, S, _, _ = R.delta_rule(q, k, v, np.array([[-0.3]]), np.array([[0.0]]), S0, 1.0, 0.0)
    assert np.allclose(S, np.exp(-0.3) * S0)


def test_norm_rope_pins():
    rs = np.random.RandomState(1)
    x = rs.randn(2, 1, 8)
    f = np.array([1.0, 0.1])
    for inter in (False, True):
        y = R.norm_rope(x, None, 0, 1e-6, np.array([0, 3]), f, 1.0, 4, inter)
        assert np.allclose(y[0], x[0]) and np.allclose(y[1, 0, 4:], x[1, 0, 4:])
        i = (0, 1) if inter else (0, 2)
        z = complex(x[1, 0, i[0]], x[1, 0, i[1]]) * np.exp(3j)
        assert np.allclose([y[1, 0, i[0]], y[1, 0, i[1]]], [z.real, z.imag])
    y = R.norm_rope(x, np.zeros(8), 1.0, 0.0, np.array([0, 0]), f, 1.0, 0, False)
    assert np.allclose((y ** 2).mean(-1), 1)
    assert np.array_equal(R.bf16(np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1.5])), [1.0, 1 + 2.0 ** -6, 1.5])
