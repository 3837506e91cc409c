"""The 64-bit reference of the norms' gradients against central differences of
the 64-bit forward pass (CPU)."""
import pytest
import torch

from . import reference64 as ref


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_gradients_are_the_differences(post, gate):
    rows, H, eps, scale = 4, 24, 1e-6, 0.6
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x = dict(y=rnd(rows, H), h=rnd(rows, H), post_w=rnd(H) if post else None, pre_w=rnd(H),
             gate={"none": None, "channel": rnd(H), "token": rnd(rows, 1)}[gate])
    a, b = rnd(rows, H), rnd(rows, H)

    def loss(x):
        hp, z, _ = ref.forward(x["y"], x["h"], x["post_w"], x["gate"], scale, x["pre_w"], eps)
        return float((z * a).sum() + (hp * b).sum())

    hp = ref.forward(x["y"], x["h"], x["post_w"], x["gate"], scale, x["pre_w"], eps)[0]
    r = ref.backward(a, b, hp, x["y"], x["post_w"], x["gate"], scale, x["pre_w"], eps)
    step = 1e-6
    for name, grad in (("y", "dy"), ("h", "dh"), ("post_w", "dpost"), ("gate", "dgate"), ("pre_w", "dpre")):
        if x[name] is None:
            assert r[grad] is None
            continue
        d = rnd(*x[name].shape)
        fd = (loss(dict(x, **{name: x[name] + step * d})) - loss(dict(x, **{name: x[name] - step * d}))) / (2 * step)
        dot = float((r[grad] * d).sum())
        # truncation about step^2, rounding about 1e-16 * |loss terms| / step
        assert abs(fd - dot) <= 1e-7 * (1 + abs(dot)), name
