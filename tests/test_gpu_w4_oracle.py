"""The 4-bit few-token layer against the CPU oracle from end to end: bf16 banks, quantised by the library
on one side and by the oracle on the other. Tolerance: that of test_gpu_few.py."""
import pytest

torch = pytest.importorskip("torch")

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytestmark = pytest.mark.skip(reason="needs a CUDA device")

import oracle  # noqa: E402
import sparse_moe_expert_fp32_b200 as moe  # noqa: E402
import synth  # noqa: E402
import test_gpu_few as few  # noqa: E402


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 8])
def test_layer_against_the_oracle(T, group):
    cfg = synth.CONFIGS["tiny"].replace(T=T)
    host, dev = synth.host_inputs(cfg, seed=T), synth.device_inputs(cfg, seed=T)
    ref = oracle.forward_inputs(host, w4=oracle.W4Experts(host.gate_up, host.down, group))
    s = moe.shape_of(cfg)
    q, gate_up, down = few._banks(s, dev, group)
    out, ids, p, gap = few._run(s, dev["x"], dev, q)
    tol = few._reference(s, dev["x"], dev, gate_up, down)[4]
    assert (ref["gap"] > 1e-5).all()  # no near tie among these tokens
    assert torch.equal(ids.cpu().long(), torch.from_numpy(ref["ids"]).long())
    err = (out.double() - torch.from_numpy(ref["out"]).cuda()).abs()
    assert (err <= tol).all(), float((err / tol).max())
