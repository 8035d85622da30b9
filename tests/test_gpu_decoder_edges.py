"""The decoder operators at the edges of what they take, against plain
implementations in 64 bits. Bounds as in test_gpu_decoder.py: U = 2^-24 is half
a unit in the last place of fp32."""
import math

import pytest

import test_gpu_decoder as base
from test_gpu_decoder import TYPES, dl, gen, logits_of, near, randn  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = math.inf


# ----------------------------------------------------------------------------
# rotary positions


def test_rotary_most_heads(dl):
    """One token of 2^31 - 1 heads, in place: the last ones are turned, and nothing beside them."""
    heads, pad = 2**31 - 1, 64
    room = torch.full((2 * heads + 2 * pad,), 7.0, dtype=torch.float16, device="cuda")
    x = room[pad:pad + 2 * heads].view(1, heads, 2)
    x[..., 0] = 1
    x[..., 1] = 0
    F = dl.RotaryFrequencies(2, frequencies=[1.0])
    dl.rotary_apply(x, F, first=1, out=x)
    for i, want in enumerate((math.cos(1.0), math.sin(1.0))):
        low, high = x[0, :, i].aminmax()
        near(torch.stack([low, high]), torch.full((2,), want, device="cuda").double(), base.ROTARY_TOL + base.UT["f16"])
    assert bool((room[:pad] == 7).all()) and bool((room[-pad:] == 7).all())


def test_rotary_widest_head(dl):
    """One head of 2^31 - 1 elements, 16 of them rotated: the others are copied to the last."""
    width, pad = 2**31 - 1, 64
    x = torch.empty(width + 1, dtype=torch.float16, device="cuda").normal_(generator=gen(1))
    room = torch.full((width + 1 + pad,), 7.0, dtype=torch.float16, device="cuda")
    # strides of whole packs: the widest ones are used
    view = lambda t: t.as_strided((1, 1, width), (2**31, 2**31, 1))  # noqa: E731
    F = dl.RotaryFrequencies(16)
    dl.rotary_apply(view(x), F, first=3, out=view(room))
    assert torch.equal(room[:16], dl.rotary_apply(x[:16].view(1, 1, 16), F, first=3).view(16))
    assert torch.equal(room[16:width], x[16:width])
    assert bool((room[width:] == 7).all())
