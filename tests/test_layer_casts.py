"""The layers under the casts and moves every module has: the projections take the type, the members the kernels read in
32 bits keep theirs, bit for bit, with their gradients."""
import copy

import pytest
import torch

from linear_attention_delta_gdn_b200.layer import DecayLinearAttentionLayer, Gdn2Layer

CASTS = {"bfloat16": lambda m: m.to(torch.bfloat16), "half": lambda m: m.half(), "double": lambda m: m.double(),
         "there and back": lambda m: m.bfloat16().float(), "device and type": lambda m: m.to("cpu", torch.bfloat16),
         "like a tensor": lambda m: m.to(torch.zeros(1, dtype=torch.bfloat16)), "in a model": lambda m: torch.nn.Sequential(m).bfloat16()[0]}


def layers():
    torch.manual_seed(1)
    return [(DecayLinearAttentionLayer(32, 3, 16, 16, sections=(3, 5), dtype=torch.float32), ("W_qk", "W_v", "W_out")),
            (Gdn2Layer(32, 2, 16, 16, dtype=torch.float32), ("W_in", "W_out"))]


@pytest.mark.parametrize("cast", CASTS)
def test_casts_keep_the_float32_members(cast):
    for layer, projections in layers():
        for p in layer.parameters():
            p.grad = torch.randn_like(p)
        was, grads = copy.deepcopy(layer.state_dict()), {n: p.grad.clone() for n, p in layer.named_parameters()}
        same = {n: getattr(layer, n) for n, _ in layer.named_parameters()}
        got = CASTS[cast](layer)
        assert got is layer
        for n in layer._float32:
            t = getattr(layer, n)
            assert t.dtype == torch.float32 and torch.equal(t, was[n]), n
            if n in grads:
                assert isinstance(t, torch.nn.Parameter) and t.requires_grad and t is same[n]
                assert t.grad.dtype == torch.float32 and torch.equal(t.grad, grads[n]), n
        to = {"half": torch.float16, "double": torch.float64, "there and back": torch.float32}.get(cast, torch.bfloat16)
        assert all(getattr(layer, n).dtype == to for n in projections)
        if "axes" in was:
            assert layer.axes.dtype == torch.int32 and torch.equal(layer.axes, was["axes"])
        assert set(layer.state_dict()) == set(was)


def test_moves_without_a_cast_stay_moves():
    for layer, _ in layers():
        layer.to("meta")
        assert all(t.device.type == "meta" for t in list(layer.parameters()) + list(layer.buffers()))
        layer.to_empty(device="cpu")
        assert all(t.device.type == "cpu" for t in list(layer.parameters()) + list(layer.buffers()))
        assert all(getattr(layer, n).dtype == torch.float32 for n in layer._float32)
    for layer, projections in layers():
        layer.to("meta", torch.bfloat16)
        assert all(getattr(layer, n).device.type == "meta" and getattr(layer, n).dtype == torch.float32 for n in layer._float32)
        assert all(getattr(layer, n).dtype == torch.bfloat16 for n in projections)


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_a_cast_layer_runs_as_one_built_that_way(packed):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.manual_seed(2)
    a = DecayLinearAttentionLayer(64, 2, 32, 32, dtype=torch.float32)
    b = DecayLinearAttentionLayer(64, 2, 32, 32, dtype=torch.bfloat16)
    b.load_state_dict(a.state_dict())
    a, b = a.to("cuda").to(torch.bfloat16), b.cuda()
    x = torch.randn(*((70,) if packed else (2, 35)), 64, device="cuda", dtype=torch.bfloat16)
    kw = {}
    if packed:
        kw = dict(positions=torch.arange(70, dtype=torch.int32, device="cuda"), Tmax=40,
                  cu_seqlens=torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda"))
    out = []
    for layer in (a, b):
        y, S = layer(x, **kw)
        (y.float().sum() + S.sum()).backward()
        out.append([y, S] + [p.grad for p in layer.parameters()])
    assert all(p.dtype == q.dtype and torch.equal(p, q) for p, q in zip(*out))
