"""The few-token layer on the GPU, with bf16 and with 4-bit experts, against the layer in 64 bits.

Tolerance (u = 2^-24), from the kernel's arithmetic: products are exact; a tensor instruction adds 16 of
them to its accumulator with at most 2 u of the magnitudes lost an addition, at most 8 instructions share
an accumulator (8 * 17 * 2 u = 272 u), and a row's parts are added in fp32 (at most K / 32 + 38 additions
of u each). With c(K) = 310 + K / 32:
  |dg| <= c(H) u G, |du| <= c(H) u Up     (G, Up: the sums of |x w|)
  |dh| <= 1.1 |u| |dg| + |silu(g)| |du| + 16 u |h|     (|silu'| < 1.1; exp, division, products; p)
  |dout| <= sum_e |Wd| (dh + c(K_all) u |h|)            (h with its routing weight in it)
where the routing weight itself is within 16 u (exp and a sum of at most 32).
Expert ids have to be equal: the logits' sums are 64-bit on both sides.
"""
import random

import pytest

torch = pytest.importorskip("torch")

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytestmark = pytest.mark.skip(reason="needs a CUDA device")

import sparse_moe_expert_fp32_b200 as moe  # noqa: E402
import synth  # noqa: E402

U = 2.0 ** -24
BF16 = torch.bfloat16
#        T, H,    E,    k,  I,   Is
SHAPES = {
    "t1": (1, 256, 16, 4, 128, 128),
    "t2_smallest": (2, 64, 1, 1, 64, 64),
    "t3": (3, 320, 24, 3, 192, 64),
    "t8_tiny": (8, 256, 16, 4, 128, 128),
    "t8_all_experts": (8, 128, 8, 8, 64, 192),
    "t5_more_experts_than_ctas": (5, 192, 333, 10, 64, 64),
    "t8_limits": (8, 512, 1024, 32, 64, 64),
    "t7_wide_h": (7, 5120, 12, 2, 64, 128),
    "t8_widest": (8, 8192, 10, 3, 128, 64),
    "t1_widest": (1, 65536, 4, 2, 64, 64),
    "t4_flash": (4, 2560, 40, 10, 640, 640),
    "t6_deep": (6, 128, 20, 5, 2048, 1024),
}
FORMS = {"bf16": 0, "w4_32": 32, "w4_64": 64, "w4_128": 128}


def _layer(shape, seed, bias=True, sigma=0.05):
    T, H, E, k, I, Is = shape
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*sh, dt=BF16, sd=sigma):
        return (torch.randn(*sh, device="cuda", generator=g) * sd).to(dt)

    w = {"w_router": n(E, H, dt=torch.float32), "w_gate_up": n(E, 2 * I, H), "w_down": n(E, H, I),
         "ws_gate_up": n(2 * Is, H), "ws_down": n(H, Is), "w_shared_gate": n(H)}
    if bias:
        w["router_bias"] = n(E, dt=torch.float32, sd=0.5)
    return moe.make_shape(*shape), n(T, H, sd=1.0), w


def _dense(q, s, K, group):
    lead = q.shape[:-1]
    out = torch.empty(lead + (K,), device="cuda")
    moe.moe_dequantize_w4(q, s, out, group)  # pinned bit for bit by the pre-pass tests
    return out.double()


def _run(s, x, w, experts=None, ws=None, stream=None, out=None):
    ws = moe.alloc_workspace(s) if ws is None else ws
    out = torch.full((s.T, s.H), 77.0, device="cuda") if out is None else out
    ids = torch.full((s.T, s.k), -1, dtype=torch.int32, device="cuda")
    p = torch.full((s.T, s.k), -1.0, device="cuda")
    gap = torch.full((s.T,), -1.0, device="cuda")
    if experts is None:
        moe.moe_layer_forward_few(s, x, w, out, ws, topk_ids=ids, topk_w=p, gap=gap, stream=stream)
    else:
        w = {n: v for n, v in w.items() if n not in ("w_gate_up", "w_down")}
        moe.moe_layer_forward_few_w4(s, x, w, experts, out, ws, topk_ids=ids, topk_w=p, gap=gap, stream=stream)
    st, flags = moe.moe_device_status(ws, stream)
    assert st == moe.MOE_OK, (st, flags)
    return out, ids, p, gap


def _banks(s, w, group):
    """(experts argument, gate|up bank, down bank as fp64 getters)."""
    if not group:
        return None, lambda e: w["w_gate_up"][e].double(), lambda e: w["w_down"][e].double()
    q = moe.quantize_w4_experts(s, w, group)
    return (q, lambda e: _dense(q["q_gate_up"][e], q["s_gate_up"][e], s.H, group),
            lambda e: _dense(q["q_down"][e], q["s_down"][e], s.I, group))


def _reference(s, x, w, gate_up, down):
    """(out, ids, p, gap, tolerance of out) in fp64."""
    x = x.double()
    logits = x @ w["w_router"].double().T
    if w.get("router_bias") is not None:
        logits = logits + w["router_bias"].double()
    top, order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, p = order[:, :s.k], torch.softmax(top[:, :s.k], 1)
    gap = top[:, s.k - 1] - top[:, s.k] if s.k < s.E else torch.full((s.T,), float("inf"), device="cuda",
                                                                    dtype=torch.float64)
    n_all = (s.T * s.k * s.I + s.Is) / 32
    ch, cd = (310 + s.H / 32) * U, (310 + n_all) * U
    out, tol = torch.zeros_like(x), torch.zeros_like(x)

    def expert(t, wgu, wd, weight):
        n = wgu.shape[0] // 2
        g, u = wgu[:n] @ x[t], wgu[n:] @ x[t]
        G, Up = wgu[:n].abs() @ x[t].abs(), wgu[n:].abs() @ x[t].abs()
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * u.abs() * ch * G + silu.abs() * ch * Up + 16 * U * h.abs()
        out[t] += weight * (wd @ h)
        tol[t] += weight * (wd.abs() @ (dh + (cd + 16 * U) * h.abs()))

    for e in torch.unique(ids).tolist():
        wgu, wd = gate_up(e), down(e)
        for t, j in torch.nonzero(ids == e).tolist():
            expert(t, wgu, wd, p[t, j])
    wgu, wd = w["ws_gate_up"].double(), w["ws_down"].double()
    sg = torch.sigmoid(x @ w["w_shared_gate"].double())
    # the gate's own sum: |d sigmoid| <= |dz| / 4 and sigmoid >= its value; relative |dz|
    dz = (310 + s.H / 32) * U * (x.abs() @ w["w_shared_gate"].double().abs())
    for t in range(s.T):
        expert(t, wgu, wd, sg[t])
        n = wgu.shape[0] // 2
        h = (wgu[:n] @ x[t]) * torch.sigmoid(wgu[:n] @ x[t]) * (wgu[n:] @ x[t])
        tol[t] += sg[t] * dz[t] * (wd.abs() @ h.abs())
    return out, ids, p, gap, tol


def _check(got, ref, tokens=None):
    out, ids, p, gap = got
    rout, rids, rp, rgap, tol = ref
    at = list(range(out.shape[0])) if tokens is None else tokens
    assert torch.equal(ids[at].long(), rids[at])
    assert ((p[at].double() - rp[at]).abs() <= 64 * U * rp[at] + 1e-30).all()
    fine = torch.isfinite(rgap[at])
    assert torch.equal(fine, torch.isfinite(gap[at]))
    assert ((gap[at].double() - rgap[at])[fine].abs() <= 2 * U * rgap[at][fine] + 1e-12).all()
    err = (out[at].double() - rout[at]).abs()
    assert (err <= tol[at]).all(), float((err / tol[at].clamp_min(1e-300)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_layer(name, form):
    s, x, w = _layer(SHAPES[name], seed=len(name))
    experts, gu, dn = _banks(s, w, FORMS[form])
    _check(_run(s, x, w, experts), _reference(s, x, w, gu, dn))


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("shape", [
    (8, 8192, 9, 3, 1088, 320),    # few and small stages; a row of 8.5 blocks of 128
    (2, 32768, 3, 2, 192, 64),     # many passes of output rows
    (5, 4160, 30, 7, 704, 448),    # rows and half blocks that divide nothing
    (8, 2560, 40, 10, 640, 640),   # two experts a stage, or one for want of units of h
    (1, 128, 300, 32, 64, 64),     # one output row a block, four experts a stage
    (6, 64, 1024, 32, 64, 64),     # fewer output rows than blocks
    (1, 2560, 11, 10, 64, 4096),   # a shared expert deeper than the routed ones
], ids=str)
def test_layer_where_the_stages_change_shape(shape, form):
    s, x, w = _layer(shape, seed=sum(shape))
    experts, gu, dn = _banks(s, w, FORMS[form])
    _check(_run(s, x, w, experts), _reference(s, x, w, gu, dn))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_layer_of_drawn_shapes(seed):
    r = random.Random(seed)
    T, E = r.randint(1, 8), r.choice([1, 5, 40, 130])
    shape = (T, 64 * r.randint(1, 60), E, r.randint(1, min(E, 32)), 64 * r.randint(1, 18), 64 * r.randint(1, 18))
    s, x, w = _layer(shape, seed=seed, bias=r.random() < 0.5)
    for form in ("bf16", r.choice(["w4_32", "w4_64", "w4_128"])):
        experts, gu, dn = _banks(s, w, FORMS[form])
        _check(_run(s, x, w, experts), _reference(s, x, w, gu, dn))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_32"])
@pytest.mark.parametrize("T", range(1, 9))
def test_every_batch_size_and_no_bias(T, form):
    s, x, w = _layer((T, 384, 48, 6, 128, 256), seed=T, bias=False)
    experts, gu, dn = _banks(s, w, FORMS[form])
    _check(_run(s, x, w, experts), _reference(s, x, w, gu, dn))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_64"])
def test_all_tokens_on_the_same_experts(form):
    s, x, w = _layer((8, 256, 32, 4, 192, 128), seed=1)
    w["router_bias"][:] = -torch.arange(32.0).cuda() * 100
    experts, gu, dn = _banks(s, w, FORMS[form])
    got = _run(s, x, w, experts)
    assert (got[1] == torch.arange(4, dtype=torch.int32, device="cuda")).all()
    _check(got, _reference(s, x, w, gu, dn))


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index():
    s, x, w = _layer((8, 128, 64, 7, 64, 64), seed=2, bias=False)
    w["w_router"][:] = w["w_router"][torch.arange(64) // 8 * 8]  # groups of eight equal experts
    _check(_run(s, x, w), _reference(s, x, w, *_banks(s, w, 0)[1:]))
    w["w_router"][:] = 0  # all logits zero, of either sign
    w["router_bias"] = torch.zeros(64, device="cuda")
    w["router_bias"][::2] = -0.0
    got = _run(s, x, w)
    assert (got[1] == torch.arange(7, dtype=torch.int32, device="cuda")).all()
    assert (got[3] == 0).all()


@pytest.mark.gpu
def test_near_ties_are_decided_as_in_64_bits():
    """Experts whose logits differ by less than fp32 sums resolve."""
    s, x, w = _layer((8, 2560, 64, 10, 64, 64), seed=3, bias=False)
    w["w_router"][:] = w["w_router"][:1]
    g = torch.Generator(device="cuda").manual_seed(5)
    at = torch.randint(0, 2560, (64,), device="cuda", generator=g)
    e = torch.arange(64, device="cuda")
    w["w_router"][e, at] *= 1 + 2.0 ** -20 * torch.randn(64, device="cuda", generator=g)
    _check(_run(s, x, w), _reference(s, x, w, *_banks(s, w, 0)[1:]))


@pytest.mark.gpu
def test_masked_experts():
    """Experts closed by a bias of -inf, or of the type's lowest value, are not chosen."""
    s, x, w = _layer((8, 192, 40, 5, 64, 64), seed=4)
    w["router_bias"][:20] = float("-inf")
    w["router_bias"][20:30] = torch.finfo(torch.float32).min
    got = _run(s, x, w)
    assert (got[1] >= 30).all()
    _check(got, _reference(s, x, w, *_banks(s, w, 0)[1:]))
    # fewer open experts than k: the closed ones come with a weight of zero
    w["router_bias"][20:37] = float("-inf")
    out, ids, p, gap = _run(s, x, w)
    assert torch.isfinite(out).all() and (p[:, 3:] == 0).all() and ((ids >= 0) & (ids < 40)).all()
    assert (ids[:, :3] >= 37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_32"])
def test_non_finite_weights_stay_with_their_tokens(form):
    s, x, w = _layer((8, 256, 40, 3, 64, 64), seed=6)
    experts, gu, dn = _banks(s, w, FORMS[form])
    ref = _reference(s, x, w, gu, dn)
    bad = int(ref[1][0, 0])
    hit = (ref[1] == bad).any(1)
    assert hit.any() and not hit.all()
    if experts is None:
        w["w_gate_up"][bad, 5] = float("nan")
        w["w_down"][bad, :, 3] = float("inf")
    else:
        experts["s_gate_up"][bad, 5] = float("nan")
        experts["s_down"][bad] = float("inf")
    got = _run(s, x, w, experts)
    assert not torch.isfinite(got[0][hit]).any()
    _check(got, ref, torch.nonzero(~hit).view(-1).tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_token_stays_alone(value):
    s, x, w = _layer((5, 256, 40, 3, 64, 64), seed=7)
    ref = _reference(s, x, w, *_banks(s, w, 0)[1:])
    x[2, 17] = value
    out, ids, p, gap = _run(s, x, w)
    assert ((ids >= 0) & (ids < 40)).all()
    assert not torch.isfinite(out[2]).any()
    _check((out, ids, p, gap), ref, [0, 1, 3, 4])


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_128"])
def test_zero_token_and_large_values(form):
    s, x, w = _layer((3, 256, 16, 4, 128, 128), seed=8)
    x[0] = 0
    x[1] *= 2.0 ** 20
    x[2] *= 2.0 ** -20
    experts, gu, dn = _banks(s, w, FORMS[form])
    got = _run(s, x, w, experts)
    assert (got[0][0] == 0).all()
    _check(got, _reference(s, x, w, gu, dn))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_32"])
def test_equal_calls_give_equal_bits_and_one_workspace_serves_all_batches(form):
    big, x, w = _layer((8, 512, 64, 8, 192, 64), seed=9)
    experts, gu, dn = _banks(big, w, FORMS[form])
    ws = moe.alloc_workspace(big)
    first = {}
    for _ in range(3):
        for T in (8, 1, 5):
            s = moe.make_shape(T, *[getattr(big, n) for n in ("H", "E", "k", "I", "Is")])
            got = _run(s, x[:T], w, experts, ws=ws)
            for a, b in zip(first.setdefault(T, got), got):
                assert torch.equal(a, b)
    for T, got in first.items():  # a token's result does not depend on the batch around it in its choice
        assert torch.equal(got[1], first[8][1][:T])


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_32"])
def test_captured_replayed_and_concurrent_calls(form):
    s, x, w = _layer((4, 512, 64, 8, 192, 64), seed=10)
    experts, gu, dn = _banks(s, w, FORMS[form])
    want = _run(s, x, w, experts)[0]
    ws = moe.alloc_workspace(s)
    outs = [torch.zeros_like(want) for _ in range(4)]

    def call(o, ws, stream=None):
        if experts is None:
            moe.moe_layer_forward_few(s, x, w, o, ws, stream=stream)
        else:
            moe.moe_layer_forward_few_w4(s, x, w, experts, o, ws, stream=stream)

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # two graphs that share a workspace
    torch.cuda.synchronize()
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o, ws)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # two calls at once, each with its own workspace
    side = [torch.cuda.Stream() for _ in range(2)]
    rooms = [moe.alloc_workspace(s) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o, r in zip(side, outs[2:], rooms):
            call(o, r, st)
    torch.cuda.synchronize()
    assert torch.equal(outs[2], want) and torch.equal(outs[3], want)
    x.copy_(torch.randn_like(x.float()).to(BF16))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], _run(s, x, w, experts)[0]) and not torch.equal(outs[0], want)
    assert moe.moe_device_status(ws)[0] == moe.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "w4_64"])
def test_guard_bands(form):
    s, x, w = _layer((3, 320, 24, 3, 192, 64), seed=11)
    experts, _, _ = _banks(s, w, FORMS[form])
    n = moe.moe_workspace_bytes(s)
    sizes = {"out": 4 * 3 * 320, "ids": 4 * 9, "p": 4 * 9, "gap": 4 * 3, "ws": n}
    raw = {k: torch.full((v + 8192,), 0xA5, dtype=torch.uint8, device="cuda") for k, v in sizes.items()}
    mid = {k: raw[k][4096:4096 + v] for k, v in sizes.items()}
    moe.moe_workspace_init(mid["ws"])
    a = (s, x, w) if experts is None else (s, x, w, experts)
    f = moe.moe_layer_forward_few if experts is None else moe.moe_layer_forward_few_w4
    f(*a, mid["out"].view(torch.float32), mid["ws"], topk_ids=mid["ids"].view(torch.int32),
      topk_w=mid["p"].view(torch.float32), gap=mid["gap"].view(torch.float32))
    torch.cuda.synchronize()
    for k, v in sizes.items():
        assert (raw[k][:4096] == 0xA5).all() and (raw[k][4096 + v:] == 0xA5).all(), k


@pytest.mark.gpu
def test_one_workspace_for_few_tokens_and_whole_batches_in_turn():
    """A serving loop's mix: single tokens and a batch through the other layer, one workspace."""
    s, x, w = _layer((8, 256, 16, 4, 128, 128), seed=12)
    big = moe.make_shape(64, 256, 16, 4, 128, 128)
    xb = torch.randn(64, 256, device="cuda").to(BF16)
    ws = moe.alloc_workspace(big)
    want_few, want_big = _run(s, x, w)[0], torch.empty(64, 256, device="cuda")
    moe.moe_layer_forward(big, xb, w, want_big, moe.alloc_workspace(big))
    for _ in range(3):
        out = torch.empty(64, 256, device="cuda")
        moe.moe_layer_forward(big, xb, w, out, ws)
        assert torch.allclose(out, want_big, rtol=1e-4, atol=1e-4)  # atomics: the order is not fixed
        assert torch.equal(_run(s, x, w, ws=ws)[0], want_few)


@pytest.mark.gpu
def test_4_bit_set_in_a_row():
    """Load time to token: quantise the bank, run the few-token layer on it, read the bank back and
    run a whole batch on it, and take one expert's matrix through the product."""
    s, x, w = _layer((4, 256, 16, 4, 128, 128), seed=13)
    q = moe.quantize_w4_experts(s, w, 32)
    got = _run(s, x, w, q)
    back = dict(w, w_gate_up=torch.empty_like(w["w_gate_up"]), w_down=torch.empty_like(w["w_down"]))
    moe.moe_dequantize_w4(q["q_gate_up"], q["s_gate_up"], back["w_gate_up"], 32)
    moe.moe_dequantize_w4(q["q_down"], q["s_down"], back["w_down"], 32)
    # the same layer on the bf16 values: each rounded by half a step of 2^-8 at most, so the
    # results differ by a few such steps of the magnitudes in the sums
    big = moe.make_shape(64, 256, 16, 4, 128, 128)
    xb = torch.cat([x, torch.randn(60, 256, device="cuda").to(BF16)])
    out = torch.empty(64, 256, device="cuda")
    moe.moe_layer_forward(big, xb, back, out, moe.alloc_workspace(big))
    ref = _reference(s, x, back, lambda e: back["w_gate_up"][e].double(), lambda e: back["w_down"][e].double())
    # tol is 310 u and more of the magnitudes: 2^-8 is 2^16 u
    assert ((got[0] - out[:4]).double().abs() <= ref[4] * (3 * 2.0 ** 16 / 310)).all()
    e = int(got[1][0, 0])
    y = torch.empty(4, 2 * 128, device="cuda")
    moe.moe_matvec_w4(x, q["q_gate_up"][e], q["s_gate_up"][e], y, 32)
    wd = _dense(q["q_gate_up"][e], q["s_gate_up"][e], 256, 32)
    assert ((y.double() - x.double() @ wd.T).abs() <= 200 * U * (x.double().abs() @ wd.abs().T)).all()


@pytest.mark.gpu
def test_synthetic_layer_of_the_repository():
    """One token of the Flash-Next-shaped layer, as the generator makes it, in both forms."""
    cfg = synth.CONFIGS["flash_decode"].replace(T=1)
    dev = synth.device_inputs(cfg, seed=0)
    s = moe.shape_of(cfg)
    w = {n: dev[n] for n in ("w_router", "w_gate_up", "w_down", "ws_gate_up", "ws_down", "w_shared_gate")}
    for group in (0, 32):
        experts, gu, dn = _banks(s, w, group)
        _check(_run(s, dev["x"], w, experts), _reference(s, dev["x"], w, gu, dn))


@pytest.mark.gpu
def test_binding_refuses_tensors_that_do_not_fit():
    s, x, w = _layer((2, 128, 8, 2, 64, 64), seed=14)
    ws = moe.alloc_workspace(s)
    out = torch.empty(2, 128, device="cuda")
    q = moe.quantize_w4_experts(s, w, 32)
    before = moe.moe_launch_count()
    calls = [(x.float(), w, out), (x[:1], w, out), (x, w, out.half()), (x, w, out[:, :64]), (x.cpu(), w, out),
             (x, dict(w, w_down=w["w_down"][:7]), out), (x, dict(w, w_router=w["w_router"].half()), out),
             (x, dict(w, ws_down=w["ws_down"].cpu()), out), (x, dict(w, router_bias=w["router_bias"][:7]), out)]
    for a in calls:
        with pytest.raises(moe.MoeError):
            moe.moe_layer_forward_few(s, *a, ws)
    for bad in (dict(q, group=64, s_down=q["s_down"][:1]), dict(q, q_down=q["q_down"][:7]), dict(q, group=16),
                dict(q, s_gate_up=q["s_gate_up"].float())):
        with pytest.raises(moe.MoeError):
            moe.moe_layer_forward_few_w4(s, x, w, bad, out, ws)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_forward_few(s, x, w, out, ws[:1024])
    assert moe.moe_launch_count() == before
