"""The calls of one layer of a step go to one stream (no GPU: the calls are fakes)."""
import pytest

from long_context_sparse_moba_gb300 import paged
from long_context_sparse_moba_gb300.paged import PagedCache


@pytest.mark.parametrize("stream", [None, "side"])
@pytest.mark.parametrize("freqs", [None, "freqs"])
def test_one_stream(monkeypatch, stream, freqs):
    seen = []

    def fake(name, result):
        return lambda *a, stream=None, **kw: (seen.append((name, stream, kw)), result)[1]

    monkeypatch.setattr(paged.ops, "rope", fake("rope", ("q", "k")))
    monkeypatch.setattr(paged.ops, "paged_append", fake("append", None))
    monkeypatch.setattr(paged.ops, "paged_attn", fake("attn", "results"))
    c = PagedCache(1, 4, 1, 64, page_size=16, block_size=64, device="cpu")
    batch = c.extend({c.new(): 3})
    kw = {} if stream is None else {"stream": stream}
    assert c.attend(0, batch, "q", "k", "v", 2, freqs=freqs, with_idx=True, **kw) == "results"
    assert [s[0] for s in seen] == (["rope"] if freqs else []) + ["append", "attn"]
    assert all(s[1] == stream for s in seen), seen
    assert seen[-1][2] == {"with_idx": True}
