"""Results of the 4-bit product over its weights are refused, on a GB300."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_results_over_weights_are_refused():
    import trellis_quantized_weight_gb300 as tq
    codes = torch.zeros(64, 64, dtype=torch.int32, device="cuda")
    scales, biases = torch.ones(64, 16).bfloat16().cuda(), torch.ones(64, 16).bfloat16().cuda()
    x = torch.ones(4, 512).bfloat16().cuda()
    for out in (codes.view(torch.bfloat16)[:2].view(4, 64), scales[:16].view(4, 64), biases[48:].view(4, 64)):
        with pytest.raises(tq.TrellisError):
            tq.gemm_q4(x, codes, scales, biases, out=out)
    x8, s8 = tq.rms_norm_q8(x, torch.ones(512).bfloat16().cuda())
    both = torch.ones(256 + 4, dtype=torch.float32, device="cuda")
    with pytest.raises(tq.TrellisError):
        tq.gemm_q4(x8, codes, scales, biases, x_scales=both[:4], out=both[2:130].view(torch.bfloat16).view(4, 64))
    assert torch.all(tq.gemm_q4(x, codes, scales, biases).float() == 512)
