"""KronAdapters as a module: what conversions of the whole model leave of its scales (CPU only: nothing is launched)."""
import copy

import pytest

torch = pytest.importorskip("torch")


def model(**kw):
    import kronecker_factored_structured_amd as K
    torch.manual_seed(0)
    return K.KronAdapters(torch.nn.Linear(8, 12), 8, 12, rank=3, adapters=4, alpha=0.7, **kw)


def test_scales_stay_float32():
    """alpha / rank is a float32 factor of the products, whatever the parameters' type: conversions of the module, or of one
    that holds it, leave it as it is."""
    want = torch.full((4,), 0.7 / 3)
    for convert in (lambda m: m.bfloat16(), lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16().float(), lambda m: m.double(), lambda m: m.half(),
                    lambda m: torch.nn.Sequential(m).bfloat16()[0], lambda m: copy.deepcopy(m).to("cpu", torch.bfloat16)):
        m = convert(model())
        assert m.scales.dtype == torch.float32 and torch.equal(m.scales, want)
        assert "scales" in m.state_dict() and [k for k, _ in m.named_buffers()] == ["scales"]
    assert model().bfloat16().down.dtype == torch.bfloat16 and model().bfloat16().projection.weight.dtype == torch.bfloat16
    assert model().to("meta", torch.bfloat16).scales.is_meta
    m = model(dtype=torch.bfloat16)
    m.scales.mul_(2)
    assert torch.equal(m.to(torch.bfloat16).scales, want * 2)      # (its own values, not those it was made with)


def test_state_of_another_type():
    m = model()
    m.load_state_dict({k: v.bfloat16() for k, v in model().state_dict().items()})
    assert m.scales.dtype == torch.float32 and torch.equal(m.scales, torch.full((4,), 0.7 / 3).bfloat16().float())
