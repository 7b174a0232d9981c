"""CPU checks of the few-token layer's geometry rule, which the host works out from the shape and the
device's number of SMs before anything is enqueued."""
import ctypes

import pytest

import sparse_moe_expert_fp32_b200 as moe


def _fits(shape, group, sms):
    """moe::few_supported(shape, experts, sms) of the library; group 0: bf16 experts."""
    f = ctypes.CDLL(moe.LIB_PATH)["_ZN3moe13few_supportedERK9moe_shapePK14moe_w4_expertsi"]
    f.restype = ctypes.c_bool
    s, q = moe.make_shape(*shape), moe.moe_w4_experts(0, 0, 0, 0, group)
    return f(ctypes.byref(s), ctypes.byref(q) if group else None, sms)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_every_shape_within_the_stated_limits_fits_a_whole_device(group):
    for T in range(0, 9):
        for H in sorted({64, 128, 192, 2560, 4160, 65536 // max(T, 1) // 64 * 64}):
            for E, k in ((1, 1), (33, 32), (512, 10), (1024, 32)):
                for I in (64, 192, 640, 1088, 2048, 16384, 65536):
                    for Is in (64, 640, 4096, 65536):
                        assert _fits((T, H, E, k, I, Is), group, 148), (T, H, E, k, I, Is)


@pytest.mark.parametrize("group", [0, 32])
def test_limits_do_not_depend_on_the_device(group):
    assert not _fits((9, 64, 8, 2, 64, 64), group, 148)
    assert not _fits((8, 8256, 8, 2, 64, 64), group, 148)
    assert not _fits((1, 65600, 8, 2, 64, 64), group, 148)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("shape,sms,ok", [
    # 1025 router rows: a block of 36 has up to 29, in 2 chunks each, and 8 tokens: 29 * 2 * 4 * 8 = 1856 partial sums
    ((8, 8192, 1024, 10, 128, 128), 36, False),
    ((8, 8192, 1024, 10, 128, 128), 72, True),   # 15 rows: 960
    # one chunk a row: 52 rows by 8 tokens are more logits than the 384 threads that add them up
    ((8, 64, 1024, 10, 64, 64), 20, False),
    ((8, 64, 1024, 10, 64, 64), 22, True),       # 47 rows: 376 logits, 1504 partial sums
    ((8, 64, 1024, 10, 64, 64), 21, False),      # 49
    ((1, 64, 1024, 10, 64, 64), 16, True),       # 65 rows of one token
    ((1, 65536, 1024, 10, 64, 64), 40, False),   # 26 rows in 17 or more chunks
])
def test_a_part_of_a_device_that_cannot_hold_the_router_is_refused(shape, sms, ok, group):
    assert _fits(shape, group, sms) == ok


@pytest.mark.parametrize("group", [0, 32])
def test_no_tokens_need_no_addresses_of_theirs(group):
    """T == 0 is valid; a framework's tensor without elements has a null address."""
    L, A = moe.lib(), 4096
    s, w = moe.make_shape(0, 128, 8, 2, 64, 64), moe.moe_weights(A, 0, A, A, A, A, A)
    before = moe.moe_launch_count()
    head = (ctypes.byref(s), None, ctypes.byref(w))
    tail = (None, None, None, None, A, moe.moe_workspace_bytes(s), None)
    if group:
        q = moe.moe_w4_experts(A, A, A, A, group)
        assert L.moe_layer_forward_few_w4(*head, ctypes.byref(q), *tail) == moe.MOE_OK
    else:
        assert L.moe_layer_forward_few(*head, *tail) == moe.MOE_OK
    assert moe.moe_launch_count() == before
