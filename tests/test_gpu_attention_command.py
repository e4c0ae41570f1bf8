"""The attention block's command on a GB300: its rotary table covers the positions that it runs."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,steps", [(40, 3), (32760, 20)])
def test_the_table_covers_every_position(prompt, steps, monkeypatch, capsys):
    from trellis_quantized_weight_gb300 import attention_block
    made, last = [], []
    table, append = attention_block.rope_table, attention_block.kv_append

    def note(cache, k, v, starts, kv_len, pages, **kw):
        last.append(kv_len)                                # the same tensor, counted up by every step
        assert pages.shape[1] * cache[0].shape[2] >= prompt + steps + 1
        return append(cache, k, v, starts, kv_len, pages, **kw)
    monkeypatch.setattr(attention_block, "rope_table", lambda n, *a, **kw: made.append(n) or table(n, *a, **kw))
    monkeypatch.setattr(attention_block, "kv_append", note)
    attention_block.main(["--requests", "2", "--prompt", str(prompt), "--steps", str(steps), "--hidden", "512", "--q-heads", "4",
                          "--kv-heads", "1", "--head-dim", "64", "--page", "16"])
    assert made == [int(last[-1].max())] and made[0] == prompt + steps + 1
    assert "us a step" in capsys.readouterr().out
