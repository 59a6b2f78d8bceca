"""The binding of include/gdn_hybrid.h on the host (no GPU): arguments that no status code of the library can catch."""
import types

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def linear(T=5):
    """q, k, v and alpha of 2 key and 4 value heads, in host memory."""
    return torch.zeros(T, 2, 64, dtype=BF), torch.zeros(T, 2, 64, dtype=BF), torch.zeros(T, 4, 64, dtype=BF), torch.ones(4)


def test_host_tensors_are_refused():
    """A kernel must never get a host address: tensors that agree in everything but lie in host memory are refused, with the
    caller's stream as well."""
    q, k, v, a = linear()
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_linear_prefill(q, k, v, a, [0, 5], ws=ws)
    states, o = torch.zeros(5, 4, 64, 64), torch.zeros(5, 4, 64, dtype=BF)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_linear_step(q, k, v, a, states)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_linear_step(q, k, v, a, states, o=o, stream=types.SimpleNamespace(cuda_stream=0))
    pq, pk = torch.zeros(2, 1, 8, 64, dtype=BF), torch.zeros(10, 2, 64, dtype=BF)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_prefix_attention(pq, pk, pk, ws=ws)


@pytest.mark.parametrize("slot", [2 ** 32, 2 ** 32 + 1, -2 ** 32 - 1, 2 ** 31, -2 ** 31 - 1])
def test_initial_slots_past_32_bits_are_refused(slot):
    """A slot that 32 bits do not hold must not come out as another one (2^32 as slot 0)."""
    q, k, v, a = linear()
    with pytest.raises(ValueError, match="S0_index"):
        gdn.gdn_linear_prefill(q, k, v, a, [0, 3, 5], S0=torch.zeros(3, 4, 64, 64), S0_index=[0, slot],
                               ws=torch.zeros(256, dtype=torch.uint8))


def test_step_without_queries_is_refused():
    """A step always reads out."""
    _, k, v, a = linear()
    with pytest.raises(ValueError, match="q"):
        gdn.gdn_linear_step(None, k, v, a, torch.zeros(5, 4, 64, 64))
