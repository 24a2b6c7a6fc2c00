"""The operators together, as a training program and a serving loop use them (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss_and_steps_follow_the_whole_pass(bits):
    from differentiable_cholesky_gb300 import train_steps
    model, losses, sequence = train_steps.train(steps=25, width=64, state_bits=bits, log=lambda s: None)
    assert all(x == x for x in losses) and losses[-1] < losses[0] - 0.3
    with torch.no_grad():
        whole = model.predict(sequence, torch.tensor([0, len(sequence)], device="cuda"))
    states = [torch.zeros((1, 64), device="cuda") for _ in model.blocks]
    steps = torch.cat([model.step(y[None], states) for y in sequence])
    # float32 products in TF32-free torch and some hundreds of roundings a token
    assert (steps - whole).norm().item() <= 1e-4 * whole.norm().item()


def test_gradients_of_the_whole_model_agree_with_differences():
    """A directional derivative of the loss (float32 model: differences with a
    step of 1e-2 of the parameters' size, good to a few parts in 10^3)."""
    from differentiable_cholesky_gb300 import train_steps
    data = train_steps.draw_sequences([60, 30], 6, 3)
    off = torch.tensor([0, 60, 90], device="cuda")
    model = train_steps.Model(6, 32, 2, seed=4)
    params = model.parameters()
    loss, status = model.loss(data, data.roll(-1, 0), off)
    loss.backward()
    assert status.item() == 0
    gen = torch.Generator(device="cuda").manual_seed(5)
    steps = [torch.randn(p.shape, generator=gen, device="cuda", dtype=p.dtype) * 1e-3 for p in params]
    along = sum((p.grad.double() * s.double()).sum() for p, s in zip(params, steps)).item()
    got = []
    with torch.no_grad():
        for sign in (1, -2):
            for p, s in zip(params, steps):
                p.add_(s, alpha=sign)
            got.append(model.loss(data, data.roll(-1, 0), off)[0].item())
    diff = (got[0] - got[1]) / 2
    assert abs(diff - along) <= 0.02 * abs(along) + 1e-5
