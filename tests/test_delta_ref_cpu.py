"""The delta-rule reference itself: its gradients against central differences, closed forms
and split chaining."""
import pytest
import torch

import delta_ref as ref


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "s0"])
def test_gradient_is_the_difference_quotient(name):
    x = ref.inputs(1, 5, 1, 2, torch.float64, seed=3)
    grads = ref.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], 0.3, x["s0"], x["dsT"])
    gen = torch.Generator().manual_seed(5)
    for _ in range(3):
        along = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)

        def loss(eps):
            y = dict(x)
            y[name] = x[name].double() + eps * along
            o, sT = ref.forward(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.3, y["s0"])
            return float((o * x["do"].double()).sum() + (sT * x["dsT"].double()).sum())

        h = 1e-5
        num = (loss(h) - loss(-h)) / (2 * h)
        ana = float((grads["d" + name] * along).sum())
        assert abs(num - ana) <= 1e-7 * (1 + abs(ana))


def test_one_token_closed_form():
    x = ref.inputs(2, 1, 1, 1, torch.float64, seed=1, state=False)
    o, s = ref.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5)
    u = x["beta"][:, 0, :, None] * x["v"][:, 0]
    torch.testing.assert_close(s, x["k"][:, 0, :, :, None] * u[:, :, None])
    torch.testing.assert_close(o[:, 0], 0.5 * (x["q"][:, 0] * x["k"][:, 0]).sum(-1, keepdim=True) * u)


def test_a_unit_key_with_gate_one_recalls_its_value():
    x = ref.inputs(1, 3, 1, 1, torch.float64, seed=2)
    one = torch.ones_like(x["beta"])
    _, s = ref.forward(x["q"], x["k"], x["v"], x["g"], one, 1.0, x["s0"])
    torch.testing.assert_close(torch.einsum("hi,hij->hj", x["k"][0, -1], s[0]), x["v"][0, -1])


def test_split_and_packed_chain():
    x = ref.inputs(1, 9, 2, 4, torch.float64, seed=4)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, s = ref.forward(*a, 0.125, x["s0"])
    o1, s1 = ref.forward(*[t[:, :4] for t in a], 0.125, x["s0"])
    o2, s2 = ref.forward(*[t[:, 4:] for t in a], 0.125, s1)
    torch.testing.assert_close(torch.cat([o1, o2], 1), o)
    torch.testing.assert_close(s2, s)
    op, sp = ref.forward(*a, 0.125, torch.cat([x["s0"]] * 2), ref.spans_of([4, 5]))
    torch.testing.assert_close(op[:, :4], o1)
    torch.testing.assert_close(sp[0], s1[0])


def test_pool_references():
    pool = torch.arange(6.0)[:, None].repeat(1, 2)
    assert ref.copied(pool, [1, 0, -1, 3, 2], [0, 1, 5, 4, 4])[:, 0].tolist() == [1, 0, 2, 3, 2, 0]
    new, index, n = ref.compacted(pool, [0, 1, 1, 0, 0, 1])
    assert new[:, 0].tolist() == [1, 2, 5, 3, 4, 5] and index == [-1, 0, 1, -1, -1, 2] and n == 3
