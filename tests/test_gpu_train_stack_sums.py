"""The key and value gradients of a donor that several layers of the stack
read: its buffers hold their sums, added in the order of the backward pass."""
import pytest

import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def harness():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_attention_quant_gb300 import harness
    return harness


@pytest.mark.parametrize("blocks", [[64, 20, 12], [300, 1, 200]])
def test_donors_hold_their_readers_sums(harness, blocks):
    """Every layer's read backward again, into buffers of its own that it does
    not add to: the donor's buffers are their fp32 sums, from the last layer
    that reads its keys and values to the donor itself, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(61)

    def d_outs(i, sp, rows):
        t = torch.randn(rows, sp.n_q_heads, sp.head_dim, generator=gen, device="cuda") * 0.01
        return t.bfloat16().view(torch.int16)

    stack = harness.TrainGradStackCase(blocks, d_outs)
    for _ in range(2):                                   # the second step starts from the first one's sums
        stack.step()
    torch.cuda.synchronize()
    layers = stack.layers
    assert len(layers) == W.N_LAYERS and all(c.grad_status() == 0 for c in layers)
    readers = {}
    for i in reversed(range(W.N_LAYERS)):
        readers.setdefault(W.stack_cache_layer(i), []).append(i)
    assert len(readers) == W.N_DONORS and max(len(r) for r in readers.values()) > 2
    for donor, order in readers.items():
        held = layers[donor].dk_hat.clone(), layers[donor].dv_hat.clone()
        assert order[-1] == donor and all(layers[i].dk_hat is layers[donor].dk_hat for i in order)
        dk = dv = None
        for i in order:
            c = layers[i]
            c.dk_hat, c.dv_hat, c.adds = torch.full_like(held[0], 7.0), torch.full_like(held[1], 7.0), False
            c.read_backward()
            dk = c.dk_hat if dk is None else dk + c.dk_hat
            dv = c.dv_hat if dv is None else dv + c.dv_hat
        torch.cuda.synchronize()
        assert torch.equal(dk, held[0]) and torch.equal(dv, held[1]), donor
