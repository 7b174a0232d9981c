"""4-bit weights on the GPU: the pre-pass on a stream that is not the current one."""
import pytest

torch = pytest.importorskip("torch")

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytestmark = pytest.mark.skip(reason="needs a CUDA device")

import sparse_moe_expert_fp32_b200 as moe  # noqa: E402

BF16 = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_quantize_on_another_stream_takes_no_memory_that_is_still_read(handle):
    """Freed on the current stream while its last reader waits there: such a block may be given out again
    there, but not to the pre-pass on another stream, which would write it at once."""
    rows, K, group = 4096, 4096, 32
    w = (torch.randn(rows, K, device="cuda") * 0.02).to(BF16)
    want = moe.quantize_w4(w, group)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.full((t.numel() * t.element_size(),), 0x5A, dtype=torch.uint8, device="cuda") for t in want]
    kept = [torch.zeros_like(t) for t in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    for k, o in zip(kept, old):
        k.copy_(o)
    del old, o
    q, s = moe.quantize_w4(w, group, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all((k == 0x5A).all() for k in kept)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    experts = {"w_gate_up": w.view(2, 2048, 4096)}
    shape = moe.make_shape(1, 4096, 2, 1, 1024, 64)
    experts["w_down"] = w.view(-1)[:2 * 4096 * 1024].view(2, 4096, 1024)
    bank = moe.quantize_w4_experts(shape, experts, group, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(bank["q_gate_up"].view_as(q), q)
