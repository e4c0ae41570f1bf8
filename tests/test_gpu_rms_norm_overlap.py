"""Outputs of the norm over its inputs: in place where that is allowed, refused elsewhere, on a GB300."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_shifted_and_strided_buffers_are_refused():
    import trellis_quantized_weight_gb300 as tq
    w = torch.ones(640).bfloat16().cuda()
    buf = torch.randn(4001, 640).bfloat16().cuda()
    x, r = buf[:-1], torch.randn(4000, 640).bfloat16().cuda()
    wide = torch.randn(4000, 1280).bfloat16().cuda()
    strided = wide[:, :640]
    inside = wide.view(-1)[:4000 * 640].view(4000, 640)             # from the same address, but whole rows
    for bad in (lambda: tq.rms_norm(x, w, out=buf[1:]), lambda: tq.rms_norm(x, w, residual=r, residual_out=buf[1:]),
                lambda: tq.rms_norm(r, w, residual=x, residual_out=buf[1:]), lambda: tq.rms_norm(strided, w, out=inside),
                lambda: tq.rms_norm(strided, w, residual=r, residual_out=inside), lambda: tq.rms_norm_q8(x, w, residual=r, residual_out=buf[1:]),
                lambda: tq.rms_norm(r[:1], w, out=w.view(1, 640))):
        with pytest.raises(tq.TrellisError):
            bad()


def test_outputs_beside_the_rows_of_a_wider_array():
    """What lies between the rows of x, or behind them, is free to be written."""
    import trellis_quantized_weight_gb300 as tq
    w = torch.ones(64).bfloat16().cuda()
    buf = torch.randn(3, 4096).bfloat16().cuda()
    x = buf[:, :64]
    want = tq.rms_norm(x.contiguous(), w)
    between = buf[0, 64:256].view(3, 64)
    assert tq.rms_norm(x, w, out=between) is between and torch.equal(between, want)
    behind = buf[2, 64:256].view(3, 64)
    tq.rms_norm(x, w, out=behind)
    assert torch.equal(behind, want)
    one = buf[1:2, :64]
    tq.rms_norm(one, w, out=one)                                     # a single row is contiguous whatever its stride
    assert torch.equal(one, want[1:2])
