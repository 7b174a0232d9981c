"""4-bit weights on the GPU: the pre-pass bit for bit against the oracle, the matrix-vector product
against 64-bit sums, their refusals' neighbours (strides, ragged ends, odd lengths), captured and
concurrent calls.

Tolerance of the product (u = 2^-24): the kernel multiplies exact operands and adds in fp32. A tensor
instruction adds 16 products to its accumulator, each addition off by at most 2 u of the magnitudes
added (truncation), and at most 8 instructions share an accumulator: 8 * 17 * 2 u = 272 u. A part's sum
is scaled and added to a running sum (u each, at most K / 32 times), and at most 32 such sums are added
at the end. So |y - ref| <= (306 + K / 32) u * sum |x w|, and y's own rounding (half a step) on top.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytestmark = pytest.mark.skip(reason="needs a CUDA device")

import oracle  # noqa: E402
import sparse_moe_expert_fp32_b200 as moe  # noqa: E402

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _matrix(rows, K, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(rows, K, generator=g) * 0.02
    if spread and rows > 1:  # row magnitudes from 2^-20 to 2^20, a zero row, a row of halves
        w *= torch.exp2(torch.randint(-20, 21, (rows, 1), generator=g).float())
        w[rows // 2] = 0
        w[-1] = torch.randint(-14, 15, (K,), generator=g) * 0.5
        w[-1, 0] = 7
    return w.to(BF16)


def _dense(q, s, K, group):
    """The stored matrix in fp64, element by element from the format's definition."""
    e = torch.arange(K, device=q.device)
    i, t, j, b = e % 8, e // 8 % 4, e // 32 % 4, e // 128
    nib = i // 2 + 4 * (i % 2)
    byte = q[:, 64 * b + 16 * t + 4 * j + nib // 2].int()
    c = torch.where(nib % 2 == 1, byte >> 4, byte & 15) - 8
    return c.double() * s[:, e // group].double()


# ------------------------------------------------------------------------- pre-pass

@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 32), (5, 33), (7, 128), (4, 129), (9, 640), (33, 250),
                                    (2, 1000), (3, 2560), (2, 8191), (300, 64)])
def test_quantize_bit_exact(rows, K, group):
    w = _matrix(rows, K, rows * 1000 + K)
    nb, ns = moe.moe_w4_row_bytes(K), moe.moe_w4_row_scales(K, group)
    q = torch.full((rows, nb), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, ns), 3.0, dtype=BF16, device="cuda")
    moe.moe_quantize_w4(w.cuda(), q, s, group)
    codes, scales = oracle.quantize_w4_rows(_bits(w), group)
    assert np.array_equal(q.cpu().numpy(), oracle.pack_w4_rows(codes))
    want = np.zeros((rows, ns))
    want[:, :scales.shape[1]] = scales
    assert np.array_equal(s.double().cpu().numpy(), want)
    back32 = torch.empty(rows, K, device="cuda")
    back16 = torch.empty(rows, K, dtype=BF16, device="cuda")
    moe.moe_dequantize_w4(q, s, back32, group)
    moe.moe_dequantize_w4(q, s, back16, group)
    values = oracle.dequantize_w4_rows(codes, scales, group)
    assert np.array_equal(back32.double().cpu().numpy(), values)
    assert np.array_equal(back16.double().cpu().numpy(), oracle.f64_to_bf16(values))


@pytest.mark.gpu
def test_quantize_every_quotient_near_a_tie():
    """All bf16 values of four binades against all scales of one binade's significands: every
    rounding decision the format can meet, exact ties among them."""
    sig = torch.arange(128, 256).float()  # 8-bit significands
    amax = (sig * 2.0 ** -7)  # one group maximum each
    vals = torch.cat([sig * 2.0 ** (e - 7) for e in (-4, -3, -2, -1, 0)])
    rows = []
    for a in amax:
        v = vals[vals.abs() <= a]
        v = torch.cat([v, -v])
        v = torch.nn.functional.pad(v, (0, -len(v) % 127)).view(-1, 127)
        rows.append(torch.cat([torch.full((len(v), 1), float(a)), v], 1))
    w = torch.cat(rows).to(BF16)
    q, s = moe.quantize_w4(w.cuda(), 128)
    codes, scales = oracle.quantize_w4_rows(_bits(w), 128)
    assert np.array_equal(q.cpu().numpy(), oracle.pack_w4_rows(codes))
    assert np.array_equal(s[:, :1].double().cpu().numpy(), scales)


@pytest.mark.gpu
def test_quantize_tiny_huge_and_non_finite():
    w = torch.zeros(6, 64)
    w[0] = torch.linspace(-1, 1, 64) * 1e-37  # scale near the bottom of bf16's normal range
    w[1] = torch.linspace(-1, 1, 64) * 1e-39  # bf16 subnormals
    w[2] = torch.linspace(-1, 1, 64) * 3e38
    w[3, :32] = torch.linspace(-1, 1, 32)
    w[3, 40] = float("inf")
    w[4, 5] = float("nan")
    w[5] = -1
    w = w.to(BF16)
    q, s = moe.quantize_w4(w.cuda(), 32)
    fine = [0, 1, 2, 5]
    codes, scales = oracle.quantize_w4_rows(_bits(w[fine]), 32)
    assert np.array_equal(q[fine].cpu().numpy(), oracle.pack_w4_rows(codes))
    assert np.array_equal(s[fine][:, :2].double().cpu().numpy(), scales)
    back = torch.empty(6, 64, device="cuda")
    moe.moe_dequantize_w4(q, s, back, 32)
    assert torch.isfinite(back[3, :32]).all() and torch.isnan(back[3, 32:]).all()
    assert torch.isnan(back[4, :32]).all() and (back[4, 32:] == 0).all()


@pytest.mark.gpu
def test_quantize_a_bank_leaves_the_rest_alone():
    w = _matrix(12, 320, 5).view(3, 4, 320).cuda()
    nb, ns = moe.moe_w4_row_bytes(320), moe.moe_w4_row_scales(320, 64)
    qbuf = torch.full((12 * nb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((12 * ns + 8,), 9.0, dtype=BF16, device="cuda")
    moe.moe_quantize_w4(w, qbuf[:12 * nb], sbuf[:12 * ns], 64)
    q, s = moe.quantize_w4(w, 64)
    assert q.shape == (3, 4, nb) and s.shape == (3, 4, ns)
    assert torch.equal(qbuf[:12 * nb], q.view(-1)) and torch.equal(sbuf[:12 * ns], s.view(-1))
    assert (qbuf[12 * nb:] == 0xA5).all() and (sbuf[12 * ns:] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 130), (4, 257), (2, 1023), (130, 641)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_ragged_rows_stay_within_their_buffers(rows, K, dt):
    w = _matrix(rows, K, K).cuda()
    raw = torch.full((rows * K + 64,), float("nan"), dtype=BF16, device="cuda")  # behind w: must not get into it
    raw[:rows * K] = w.view(-1)
    nb, ns = moe.moe_w4_row_bytes(K), moe.moe_w4_row_scales(K, 32)
    qbuf = torch.full((rows * nb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((rows * ns + 8,), 9.0, dtype=BF16, device="cuda")
    moe.moe_quantize_w4(raw[:rows * K].view(rows, K), qbuf[:rows * nb], sbuf[:rows * ns], 32)
    q, s = qbuf[:rows * nb].view(rows, nb), sbuf[:rows * ns].view(rows, ns)
    codes, scales = oracle.quantize_w4_rows(_bits(w), 32)
    assert np.array_equal(q.cpu().numpy(), oracle.pack_w4_rows(codes))
    back = torch.full((rows * K + 64,), 5.0, dtype=dt, device="cuda")
    moe.moe_dequantize_w4(q, s, back[:rows * K].view(rows, K), 32)
    assert torch.equal(back[:rows * K].view(rows, K).double(), _dense(q, s, K, 32).to(dt).double())
    assert (back[rows * K:] == 5).all() and (qbuf[rows * nb:] == 0xA5).all() and (sbuf[rows * ns:] == 9).all()


# ------------------------------------------------------------------------- product

def _check(x, q, s, K, group, y, ref_w=None):
    w = _dense(q, s, K, group) if ref_w is None else ref_w
    ref = x.double() @ w.T
    mag = x.double().abs() @ w.abs().T
    tol = (306 + K / 32) * U * mag
    if y.dtype is not F32:
        tol = tol + torch.finfo(y.dtype).eps / 2 * (ref.abs() + tol)
        tol = tol + (2.0 ** -25 if y.dtype is F16 else 0.0)  # half a step of fp16's subnormals
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-300)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("xt,yt", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("T,N,K,group", [
    (1, 1, 1, 32), (1, 16, 64, 32), (2, 17, 127, 32), (3, 147, 129, 64), (8, 149, 128, 128), (9, 33, 640, 32),
    (16, 2560, 640, 64), (5, 4099, 2501, 64), (1, 5000, 2560, 32), (7, 300, 8192, 128), (16, 65, 4225, 32),
    (16, 9500, 256, 128), (4, 64, 16500, 128), (16, 600, 9000, 64), (1, 150000, 64, 32),
    (15, 80001, 320, 32), (13, 700, 13001, 128), (1, 40, 70000, 64)])
def test_matvec(T, N, K, group, xt, yt):
    g = torch.Generator().manual_seed(T * 7 + N + K)
    x = torch.randn(T, K, generator=g).to(xt).cuda()
    q, s = moe.quantize_w4((torch.randn(N, K, generator=g) * 0.02).to(BF16).cuda(), group)
    y = torch.full((T, N), 7.0, dtype=yt, device="cuda")
    moe.moe_matvec_w4(x, q, s, y, group)
    _check(x, q, s, K, group, y)


@pytest.mark.gpu
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (8, 8), (64, 5)])
def test_matvec_strided_rows_and_untouched_gaps(pad, off, xt):
    T, N, K, group = 5, 211, 417, 32
    g = torch.Generator().manual_seed(3)
    xb = torch.randn(T, K + pad + off, generator=g).to(xt).cuda()
    xb[:, off + K:] = float("nan")  # what lies between the rows must not be read into them
    xb[:, :off] = float("nan")
    q, s = moe.quantize_w4((torch.randn(N, K, generator=g) * 0.02).to(BF16).cuda(), group)
    yb = torch.full((T + 1, N + pad + off), 5.0, device="cuda")
    y = yb[:T, off:off + N]
    moe.moe_matvec_w4(xb[:, off:off + K], q, s, y, group)
    _check(xb[:, off:off + K], q, s, K, group, y)
    assert (yb[T] == 5).all() and (yb[:, :off] == 5).all() and (yb[:, off + N:] == 5).all()


@pytest.mark.gpu
def test_matvec_every_code_and_scale_sign():
    """Codes that the pre-pass does not write (0 stands for -8) and negative scales."""
    N, K, group = 40, 384, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randint(0, 256, (N, moe.moe_w4_row_bytes(K)), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randn(N, moe.moe_w4_row_scales(K, group), device="cuda", generator=g).to(BF16)
    x = torch.randn(3, K, device="cuda", generator=g).to(F16)
    y = torch.empty(3, N, device="cuda")
    moe.moe_matvec_w4(x, q, s, y, group)
    _check(x, q, s, K, group, y)


@pytest.mark.gpu
def test_matvec_non_finite_stays_in_its_row():
    N, K = 70, 256
    q, s = moe.quantize_w4(_matrix(N, K, 2, spread=False).cuda(), 32)
    s[3, 2] = float("nan")
    s[44, 0] = float("inf")
    x = torch.randn(6, K, device="cuda").to(BF16)
    x[4, 100] = float("inf")
    y = torch.empty(6, N, device="cuda")
    moe.moe_matvec_w4(x, q, s, y, 32)
    rows = [r for r in range(N) if r not in (3, 44)]
    toks = [0, 1, 2, 3, 5]
    assert torch.isnan(y[:, 3]).all()
    assert not torch.isfinite(y[toks][:, 44]).any()
    w = _dense(q, s, K, 32)[rows]
    _check(x[toks], q, s, K, 32, y[toks][:, rows], w)


@pytest.mark.gpu
def test_matvec_same_bits_captured_and_on_two_streams():
    T, N, K, group = 4, 3000, 1280, 64
    q, s = moe.quantize_w4(_matrix(N, K, 4, spread=False).cuda(), group)
    x = torch.randn(T, K, device="cuda").to(BF16)
    y = torch.empty(T, N, device="cuda")
    moe.moe_matvec_w4(x, q, s, y, group)
    ys = [torch.empty_like(y) for _ in range(3)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for st, o in zip(side, ys):
        moe.moe_matvec_w4(x, q, s, o, group, stream=st)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_matvec_w4(x, q, s, ys[2], group)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, o) for o in ys)
    x.copy_(torch.randn(T, K, device="cuda").to(BF16))
    graph.replay()
    moe.moe_matvec_w4(x, q, s, y, group)
    torch.cuda.synchronize()
    assert torch.equal(y, ys[2])


@pytest.mark.gpu
def test_matvec_refuses_tensors_that_do_not_fit():
    q, s = moe.quantize_w4(_matrix(32, 128, 4, spread=False).cuda(), 32)
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    y = torch.zeros(2, 32, device="cuda")
    bad = [(x.float(), q, s, y), (x, q.cpu(), s, y), (x, q[:31], s, y), (x, q, s[:31], y), (x, q, s.float(), y),
           (x, q, s, y.double()), (x, q, s, y.half()), (x[:1], q, s, y), (x.t(), q, s, y), (x, q, s, y.cpu()),
           (x[:, ::2], q, s, y), (x, q.t(), s, y), (x[:1].expand(2, 128), q, s, y)]
    before = moe.moe_launch_count()
    for args in bad:
        with pytest.raises(moe.MoeError):
            moe.moe_matvec_w4(*args, 32)
    with pytest.raises(moe.MoeError):
        moe.moe_matvec_w4(torch.zeros(17, 128, dtype=BF16, device="cuda"), q, s,
                          torch.zeros(17, 32, device="cuda"), 32)
    assert moe.moe_launch_count() == before
    moe.moe_matvec_w4(x[:0], q, s, y[:0], 32)  # no rows: nothing to do
    assert moe.moe_launch_count() == before
