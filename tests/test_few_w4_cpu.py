"""CPU checks of the few-token and 4-bit calls: the oracle's 4-bit format on hand-made rows, and
that every call refuses bad arguments before anything is enqueued (fake addresses, never
dereferenced)."""
import ctypes

import numpy as np
import pytest

import oracle
import sparse_moe_expert_fp32_b200 as moe
import synth

A = 4096  # an aligned address that nothing reads


def _bf16(v):
    """fp32 values that bf16 holds exactly -> their bits."""
    u = np.asarray(v, np.float32).view(np.uint32)
    assert not (u & 0xFFFF).any()
    return (u >> 16).astype(np.uint16)


# ------------------------------------------------------------------------- the format's oracle

def test_f64_to_bf16_rounds_half_to_even():
    one = 1.0
    ulp = 2.0 ** -7
    v = np.array([one + ulp / 2, one + 3 * ulp / 2, one + 0.49 * ulp, -one - 3 * ulp / 2, 0.0, 2.0 ** -133])
    want = [one, one + 2 * ulp, one, -one - 2 * ulp, 0.0, 2.0 ** -133]
    assert oracle.f64_to_bf16(v).tolist() == want


def test_quantize_rows_by_hand():
    # amax 7 -> scale 1: halves round to even, the rest to the nearest integer
    w = np.zeros((1, 32), np.float32)
    w[0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, 0.75]
    codes, s = oracle.quantize_w4_rows(_bf16(w), 32)
    assert s.tolist() == [[1.0]]
    assert (codes[0, :8].astype(int) - 8).tolist() == [7, -7, 0, 2, 2, 0, -2, 1]
    assert (codes[0, 8:] == 8).all()


def test_quantize_zero_row_and_short_group():
    w = np.zeros((2, 40), np.float32)
    w[1, 39] = -3.5
    codes, s = oracle.quantize_w4_rows(_bf16(w), 32)
    assert s.shape == (2, 2) and s[0].tolist() == [0, 0] and s[1].tolist() == [0, 0.5]
    assert (codes[0] == 8).all() and codes[1, 39] == 1


def test_packing_places_each_element():
    # one element differs from 8 at a time: its byte and nibble follow the stated rule
    for e in (0, 1, 2, 7, 8, 31, 32, 100, 127, 128, 300):
        codes = np.full((1, 301), 8, np.uint8)
        codes[0, e] = 13
        b = oracle.pack_w4_rows(codes)
        assert b.shape == (1, 192)
        i, t, j = e % 8, e // 8 % 4, e // 32 % 4
        nib = i // 2 + 4 * (i % 2)
        at = 64 * (e // 128) + 16 * t + 4 * j + nib // 2
        want = np.full(192, 0x88, np.uint8)
        want[at] = 0xD8 if nib % 2 else 0x8D
        assert np.array_equal(b[0], want)


@pytest.mark.parametrize("K,group,nb,ns", [(1, 32, 64, 8), (128, 128, 64, 8), (129, 128, 128, 8),
                                           (256, 32, 128, 8), (257, 32, 192, 16),
                                           (2560, 64, 1280, 40), (1 << 20, 32, 1 << 19, 1 << 15)])
def test_row_sizes(K, group, nb, ns):
    assert moe.moe_w4_row_bytes(K) == nb
    assert moe.moe_w4_row_scales(K, group) == ns


@pytest.mark.parametrize("K,group", [(0, 32), (-1, 32), ((1 << 20) + 1, 32), (64, 16), (64, 0), (64, -32)])
def test_row_sizes_refused(K, group):
    with pytest.raises(moe.MoeError):
        moe.moe_w4_row_scales(K, group)


# ------------------------------------------------------------------------- refusals

def _few(s, x=A, w=None, out=A, ws=A, n=1 << 40, ids=None, p=None, gap=None, experts=None):
    L = moe.lib()
    w = moe.moe_weights(A, 0, A, A, A, A, A) if w is None else w
    if experts is None:
        return L.moe_layer_forward_few(ctypes.byref(s), x, ctypes.byref(w), out, ids, p, gap, ws, n, None)
    return L.moe_layer_forward_few_w4(ctypes.byref(s), x, ctypes.byref(w), ctypes.byref(experts), out,
                                      ids, p, gap, ws, n, None)


W4 = dict(q_gate_up=A, s_gate_up=A, q_down=A, s_down=A, group=32)


def _experts(**kw):
    d = dict(W4, **kw)
    return moe.moe_w4_experts(d["q_gate_up"], d["s_gate_up"], d["q_down"], d["s_down"], d["group"])


@pytest.mark.parametrize("w4", [False, True])
def test_few_layer_refuses(w4):
    e = _experts() if w4 else None
    tiny = synth.CONFIGS["tiny"]
    s = moe.shape_of(tiny, T=8)
    before = moe.moe_launch_count()
    assert _few(moe.shape_of(tiny, T=9), experts=e) == moe.MOE_ERR_UNSUPPORTED
    assert _few(moe.make_shape(8, 8256, 16, 4, 128, 128), experts=e) == moe.MOE_ERR_UNSUPPORTED
    assert _few(moe.make_shape(1, 65600, 16, 4, 128, 128), experts=e) == moe.MOE_ERR_UNSUPPORTED
    assert _few(moe.make_shape(1, 100, 16, 4, 128, 128), experts=e) == moe.MOE_ERR_UNSUPPORTED
    assert _few(moe.make_shape(1, 256, 16, 17, 128, 128), experts=e) == moe.MOE_ERR_UNSUPPORTED
    assert _few(moe.make_shape(-1, 256, 16, 4, 128, 128), experts=e) == moe.MOE_ERR_INVALID_ARG
    for bad in (dict(x=None), dict(x=A + 2), dict(out=None), dict(out=A + 4), dict(ws=None),
                dict(ws=A + 8), dict(ids=A + 4), dict(p=A + 4), dict(gap=A + 4)):
        assert _few(s, experts=e, **bad) == moe.MOE_ERR_INVALID_ARG, bad
    for i in (0, 4, 5, 6) if w4 else (0, 2, 3, 4, 5, 6):
        v = [A, 0, A, A, A, A, A]
        for bad in (0, A + 2):
            v[i] = bad
            assert _few(s, w=moe.moe_weights(*v), experts=e) == moe.MOE_ERR_INVALID_ARG, (i, bad)
    n = moe.moe_workspace_bytes(s)
    assert _few(s, n=n - 1, experts=e) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert _few(moe.shape_of(tiny, T=0), n=n, experts=e) == moe.MOE_OK  # no tokens: nothing to do
    assert moe.moe_launch_count() == before


@pytest.mark.parametrize("bad", [dict(q_gate_up=None), dict(s_gate_up=None), dict(q_down=None),
                                 dict(s_down=None), dict(q_gate_up=A + 8), dict(s_down=A + 2),
                                 dict(group=0), dict(group=16), dict(group=256), dict(group=-32)])
def test_few_w4_refuses_experts(bad):
    s = moe.shape_of(synth.CONFIGS["tiny"], T=1)
    assert _few(s, experts=_experts(**bad)) == moe.MOE_ERR_INVALID_ARG


def test_few_w4_needs_no_bf16_bank_and_no_experts_is_refused():
    s = moe.shape_of(synth.CONFIGS["tiny"], T=0)
    w = moe.moe_weights(A, 0, 0, 0, A, A, A)
    assert _few(s, w=w, experts=_experts()) == moe.MOE_OK
    assert moe.lib().moe_layer_forward_few_w4(ctypes.byref(s), A, ctypes.byref(w), None, A, None, None,
                                              None, A, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG


def _mv(T=1, N=16, K=64, group=32, xt=moe.MOE_BF16, x=A, ldx=64, q=A, s=A, yt=moe.MOE_F32, y=A, ldy=16):
    return moe.lib().moe_matvec_w4(T, N, K, group, xt, x, ldx, q, s, yt, y, ldy, None)


def test_matvec_refuses():
    before = moe.moe_launch_count()
    I, U = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    for kw, want in ((dict(T=-1), I), (dict(N=-1), I), (dict(K=0), I), (dict(group=48), I),
                     (dict(xt=moe.MOE_F32), I), (dict(xt=7), I), (dict(yt=moe.MOE_F16), I), (dict(yt=5), I),
                     (dict(T=17), U), (dict(K=(1 << 20) + 1), U), (dict(N=(1 << 31) + 1), U),
                     (dict(x=None), I), (dict(x=A + 1), I), (dict(y=None), I), (dict(y=A + 2), I),
                     (dict(q=None), I), (dict(q=A + 4), I), (dict(s=None), I), (dict(s=A + 2), I),
                     (dict(T=2, ldx=63), I), (dict(T=2, ldy=15), I), (dict(T=0), moe.MOE_OK),
                     (dict(N=0), moe.MOE_OK)):
        assert _mv(**kw) == want, kw
    assert moe.moe_launch_count() == before


def test_quantize_and_dequantize_refuse():
    L, I, U = moe.lib(), moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    before = moe.moe_launch_count()
    for a, want in (((-1, 64, 32, A, A, A), I), ((1, 0, 32, A, A, A), I), ((1, 64, 31, A, A, A), I),
                    ((1, (1 << 20) + 1, 32, A, A, A), U), (((1 << 31) + 1, 64, 32, A, A, A), U),
                    ((1, 64, 32, None, A, A), I), ((1, 64, 32, A + 2, A, A), I), ((1, 64, 32, A, None, A), I),
                    ((1, 64, 32, A, A + 1, A), I), ((1, 64, 32, A, A, A + 2), I),
                    ((0, 64, 32, None, None, None), moe.MOE_OK)):
        assert L.moe_quantize_w4(*a, None) == want, a
        q = a[:3] + (a[4], a[5], moe.MOE_BF16, a[3])
        assert L.moe_dequantize_w4(*q, None) == want, q
    assert L.moe_dequantize_w4(1, 64, 32, A, A, moe.MOE_F16, A, None) == I
    assert moe.moe_launch_count() == before


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 64, dtype=torch.bfloat16)  # host memory: not a device tensor
    y, q, s = torch.zeros(1, 16), torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 8, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):
        moe.moe_matvec_w4(x, q, s, y, 32)
    with pytest.raises(moe.MoeError):
        moe.moe_matvec_w4(x[0], q, s, y, 32)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_w4(torch.zeros(16, 64), q, s, 32)  # fp32 weights
    with pytest.raises(moe.MoeError):
        moe.moe_dequantize_w4(q, s, torch.zeros(16, 64), 32)
    cfg = synth.CONFIGS["tiny"]
    w = {n: torch.zeros(1, dtype=torch.bfloat16) for n in ("w_gate_up", "w_down", "ws_gate_up", "ws_down",
                                                           "w_shared_gate")}
    w["w_router"] = torch.zeros(1)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_forward_few(moe.shape_of(cfg, T=1), x, w, y, q)
