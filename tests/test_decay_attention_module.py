"""DecayAttention's parameters and buffer under casts and moves, on the CPU."""

import pytest
import torch

X = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.mixers")


@pytest.mark.parametrize("cast", [lambda m: m.bfloat16(), lambda m: m.to(torch.bfloat16), lambda m: m.to("cpu", torch.bfloat16),
                                  lambda m: torch.nn.Sequential(m).bfloat16()[0], lambda m: m.double().bfloat16(),
                                  lambda m: m.bfloat16().float().bfloat16()])
def test_decays_stay_float32(cast):
    m = X.DecayAttention(32, 4, 16, dtype=torch.float32)
    g = m.log_decay.clone()
    m = cast(m)
    assert m.query.dtype == torch.bfloat16 and m.log_decay.dtype == torch.float32 and torch.equal(m.log_decay, g)
    assert list(m.state_dict()) == ["query", "key", "value", "out", "log_decay"] and m._buffers["log_decay"] is m.log_decay


def test_decays_move_with_the_module():
    m = X.DecayAttention(32, 4, 16, dtype=torch.float32)
    sd = {n: t.clone() for n, t in m.state_dict().items()}
    m.to("meta")
    assert m.log_decay.is_meta and m.query.is_meta
    m.to_empty(device="cpu").bfloat16()
    assert m.log_decay.dtype == torch.float32 and m.log_decay.device.type == "cpu"
    m.load_state_dict(sd)
    assert torch.equal(m.log_decay, sd["log_decay"])
    with torch.device("meta"):
        n = X.DecayAttention(32, 4, 16, log_decay=[-1.0] * 4, device="meta")
    assert n.bfloat16().log_decay.dtype == torch.float32
