"""The decoding command's steps: a token's residual stream begins with its own row, on a GB300."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_token_does_not_carry_the_streams_of_those_before(monkeypatch, capsys):
    """After the last token the stream is that token's row and its attention half's output, each added once: what the tokens
    before it left in the stream would be there too."""
    from trellis_quantized_weight_gb300 import attention_block

    class Stream(torch.cuda.Stream):                # of the other pool
        def __new__(cls, *a, **kw):
            return super().__new__(cls, *a, **{**kw, "priority": -1})
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    seen = {}
    step, half = attention_block.Layer.step, attention_block.AttentionBlock.step

    def layer_step(self, x, residual, *a, **kw):
        seen["x"], seen["residual"] = x, residual
        return step(self, x, residual, *a, **kw)

    def half_step(self, *a, **kw):
        seen["y"] = half(self, *a, **kw)
        return seen["y"]
    monkeypatch.setattr(attention_block.Layer, "step", layer_step)
    monkeypatch.setattr(attention_block.AttentionBlock, "step", half_step)
    attention_block.main(["--requests", "3", "--prompt", "40", "--samples", "2", "--steps", "12", "--hidden", "512", "--inner", "768",
                          "--q-heads", "4", "--kv-heads", "1", "--head-dim", "64", "--page", "16"])
    torch.cuda.synchronize()
    assert seen["x"].shape == (6, 512)
    assert torch.equal(seen["residual"], (seen["x"].float() + seen["y"].float()).bfloat16())
