"""The scratch of a call is sized for its tensors' device, not for the current one: it
goes by the number of SMs (no GPU: the library is a fake)."""
import torch

from long_context_sparse_moba_gb300 import ops


def test_workspace_is_sized_on_the_tensors_device(monkeypatch):
    current, asked = [0], []

    class Lib:
        @staticmethod
        def moba_paged_attn_workspace_size(*a):
            asked.append(current[0])
            return 512

        @staticmethod
        def moba_paged_attn(*a):
            assert a[-2] == 512 and current[0] == 1
            return 0

    def call(device, stream, fn):
        current[0] = device
        try:
            return fn(0)
        finally:
            current[0] = 0

    monkeypatch.setattr(ops, "lib", lambda: Lib)
    monkeypatch.setattr(ops, "_call", call)
    monkeypatch.setattr(ops, "_device", lambda t, name: 1)
    monkeypatch.setattr(ops, "_tensor", lambda *a: None)
    monkeypatch.setattr(ops, "_paged", lambda *a: (4, 2, 16, 64, 1, 4, 0))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pools, ints = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    ops.paged_attn(q, pools, pools, None, ints, ints, ints, 3, 64, 4)
    assert asked == [1]
