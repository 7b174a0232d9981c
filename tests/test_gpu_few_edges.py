"""The few-token layer at the edges of fp32: SwiGLU where the gate closes, infinite weights.

One token, x a unit vector and one expert (routing weight 1), so that gate and up are single weights,
known exactly, and with one weight in each row of W_down an output is one element of h.
"""
import pytest

torch = pytest.importorskip("torch")

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytestmark = pytest.mark.skip(reason="needs a CUDA device")

import sparse_moe_expert_fp32_b200 as moe  # noqa: E402

U = 2.0 ** -24
BF16 = torch.bfloat16
N = 64  # H and I


def _layer(gate, up):
    """Layer of one expert with gate[c] and up[c] in channel c, W_down the identity; the shared
    expert's matrices are zero."""
    s = moe.make_shape(1, N, 1, 1, N, N)
    x = torch.zeros(1, N, dtype=BF16, device="cuda")
    x[0, 0] = 1
    w = {n: torch.zeros(*sh, dtype=BF16, device="cuda") for n, sh in
         (("w_gate_up", (1, 2 * N, N)), ("w_down", (1, N, N)), ("ws_gate_up", (2 * N, N)), ("ws_down", (N, N)),
          ("w_shared_gate", (N,)))}
    w["w_router"] = torch.zeros(1, N, device="cuda")
    w["w_gate_up"][0, :len(gate), 0] = torch.tensor(gate, dtype=torch.float64).to(BF16).cuda()
    w["w_gate_up"][0, N:N + len(up), 0] = torch.tensor(up, dtype=torch.float64).to(BF16).cuda()
    w["w_down"][0] = torch.eye(N, device="cuda").to(BF16)
    return s, x, w


def _run(s, x, w, group=0):
    """(out [H], gate|up bank, down bank as the layer reads them, in 64 bits)."""
    ws, out = moe.alloc_workspace(s), torch.full((1, N), 77.0, device="cuda")
    if group:
        q = moe.quantize_w4_experts(s, w, group)
        moe.moe_layer_forward_few_w4(s, x, w, q, out, ws)
        banks = []
        for n in ("gate_up", "down"):
            b = torch.empty_like(w["w_" + n], dtype=torch.float32)
            moe.moe_dequantize_w4(q["q_" + n], q["s_" + n], b, group)
            banks.append(b[0].double())
    else:
        moe.moe_layer_forward_few(s, x, w, out, ws)
        banks = [w["w_gate_up"][0].double(), w["w_down"][0].double()]
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK
    return out[0].double(), *banks


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 32, 128])
def test_closed_gates(group):
    """h = SiLU(gate) up for gates whose exponential leaves fp32's range, and where gate times up does.

    Tolerance: exp, the division and the four products of h and of its way to the output are within
    24 u of h; below -87 exp(gate) is a subnormal, off by at most 4 steps of 2^-149 with the quotient's
    rounding; below -104 it is 0, and h as small as that."""
    pairs = [(-1.0, 1e30), (-60, 1e30), (-85, 1e35), (-87, 1e30), (-87.5, 1e30), (-88, 1e30), (-88.5, -1e33),
             (-89, 1e35), (-89, 1e38), (-95, 1e37), (-100, 1e37), (-100, -3e38), (-103, 1e38), (-108, 1e38),
             (-110, 3e38), (-1e4, 1e37), (-1e10, -1e30), (-1e20, 1e20), (-1e30, 1e30), (-1e37, 3e38),
             (88.0, 3.0), (89, 1e30), (100, -1e30), (1e4, 1e30), (1e20, 1e10), (0.0, 1e30), (-50, 0.0)]
    s, x, w = _layer(*zip(*pairs))
    out, gu, dn = _run(s, x, w, group)
    gate, up = gu[:N, 0], gu[N:, 0]
    h = gate / (1 + torch.exp(-gate)) * up
    want = dn @ h
    small = torch.where(gate > -104, 4 * 2.0 ** -149 * (gate * up).abs(), h.abs())
    tol = 24 * U * h.abs() + torch.where(gate < -87, small, 0.0)
    err = (out - want).abs()
    assert (err <= dn.abs() @ tol).all(), [(p, float(o), float(v)) for p, o, v in zip(pairs, out, want)]

@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_h_keeps_24_bits(group):
    """h goes to the down product in three pieces of 8 bits. Its way there and to the output is within
    24 u (exp 4, division 4, the sum and the products 1 each, the pieces' sum and, for 4-bit weights,
    their scales 5); without the third piece it would be up to 512 u off."""
    g = torch.Generator().manual_seed(3)
    gate, up = torch.randn(N, generator=g) * 2, torch.randn(N, generator=g)
    s, x, w = _layer(gate.tolist(), up.tolist())
    out, gu, dn = _run(s, x, w, group)
    gate, up = gu[:N, 0], gu[N:, 0]
    h = gate / (1 + torch.exp(-gate)) * up
    step = torch.exp2(torch.floor(torch.log2(h.abs())) - 15)  # two pieces: 16 bits
    short = torch.trunc(h / step) * step
    tol = 24 * U * (dn @ h).abs()
    assert ((out - dn @ h).abs() <= tol).all()
    assert ((dn @ (short - h)).abs() > 2 * tol).sum() > N // 2  # what this test is to see


@pytest.mark.gpu
def test_infinite_down_weights_times_short_h():
    """An infinite weight times a finite h is an infinity, whichever of h's bits are zero, and NaN for
    h = 0; other rows are as they were. (SiLU(128) is 128 in fp32: h has one significant bit.)"""
    inf = float("inf")
    s, x, w = _layer([128.0] * 16, [1.0, -1.0, 0.0] + [1.0] * 13)
    w["w_down"][0, 20, 0], w["w_down"][0, 21, 1], w["w_down"][0, 22, 0] = inf, inf, -inf
    w["w_down"][0, 23, 2] = inf                               # h = 0
    w["w_down"][0, 24, 3], w["w_down"][0, 24, 4] = inf, -inf  # of either sign
    w["w_down"][0, 25, 5] = float("nan")
    w["ws_gate_up"][0, 0], w["ws_gate_up"][N, 0], w["ws_down"][26, 0] = 128, 1, inf  # the shared expert
    out, gu, dn = _run(s, x, w)
    want = dn @ (gu[:N, 0] * gu[N:, 0])
    want[26] = inf
    assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(want, 7.0))
    assert torch.equal(out.isnan(), want.isnan()) and out.isnan().sum() == 3


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("H,T", [(64, 1), (64, 8), (128, 3)])
def test_blocks_without_output_rows_do_not_wait_for_the_others(H, T, group):
    """H is below the number of blocks: some have no output row and leave early. A block that still looked
    at the grid's counters when the last one puts them back to zero would wait until its limit (seconds),
    and the status would say so."""
    g = torch.Generator(device="cuda").manual_seed(H + T)
    s = moe.make_shape(T, H, 32, 4, 64, 64)
    x = torch.randn(T, H, device="cuda", generator=g).to(BF16)
    w = {n: (torch.randn(*sh, device="cuda", generator=g) * 0.05).to(BF16) for n, sh in
         (("w_gate_up", (32, 128, H)), ("w_down", (32, H, 64)), ("ws_gate_up", (128, H)), ("ws_down", (H, 64)),
          ("w_shared_gate", (H,)))}
    w["w_router"] = torch.randn(32, H, device="cuda", generator=g) * 0.05
    ws, out = moe.alloc_workspace(s), torch.empty(T, H, device="cuda")
    if group:
        q = moe.quantize_w4_experts(s, w, group)
        call = lambda: moe.moe_layer_forward_few_w4(s, x, w, q, out, ws)  # noqa: E731
    else:
        call = lambda: moe.moe_layer_forward_few(s, x, w, out, ws)  # noqa: E731
    call()
    want = out.clone()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(3000):
        call()
    b.record()
    b.synchronize()
    assert torch.equal(out, want)
    assert moe.moe_device_status(ws) == (moe.MOE_OK, 0)
    assert a.elapsed_time(b) < 1500  # ms; a wait that runs out takes 2000 by itself


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 32])
def test_a_barrier_that_runs_out_is_reported_and_leaves_the_workspace_ready(group):
    """The counter of the first grid barrier (the workspace's 17th word) starts one below zero, so that it
    never gets to the number of blocks (a block adds one to it before it looks). Every block's wait ends at
    its limit, the status says so, and the next call on the same workspace is right."""
    T, H, E, k, I = 3, 256, 16, 4, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    s = moe.make_shape(T, H, E, k, I, I)
    x = torch.randn(T, H, device="cuda", generator=g).to(BF16)
    w = {n: (torch.randn(*sh, device="cuda", generator=g) * 0.05).to(BF16) for n, sh in
         (("w_gate_up", (E, 2 * I, H)), ("w_down", (E, H, I)), ("ws_gate_up", (2 * I, H)), ("ws_down", (H, I)),
          ("w_shared_gate", (H,)))}
    w["w_router"] = torch.randn(E, H, device="cuda", generator=g) * 0.05
    ws = moe.alloc_workspace(s)
    raw = torch.full((T * H + 2048,), 7.0, device="cuda")
    out = raw[1024:1024 + T * H].view(T, H)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    q = moe.quantize_w4_experts(s, w, group) if group else None

    def call():
        if group:
            moe.moe_layer_forward_few_w4(s, x, w, q, out, ws, topk_ids=ids)
        else:
            moe.moe_layer_forward_few(s, x, w, out, ws, topk_ids=ids)

    call()
    want = out.clone(), ids.clone()
    ws.view(torch.int32)[16] = -1
    call()
    status, flags = moe.moe_device_status(ws)
    assert status == moe.MOE_ERR_DEVICE_TIMEOUT and flags == 2
    assert ((ids >= 0) & (ids < E)).all()
    assert (raw[:1024] == 7).all() and (raw[1024 + T * H:] == 7).all()
    for _ in range(3):
        call()
        assert torch.equal(out, want[0]) and torch.equal(ids, want[1])
    assert moe.moe_device_status(ws) == (moe.MOE_OK, 0)
