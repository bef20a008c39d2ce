"""Rotation by small angles, one dim of the pair at a time: the sine itself, to
the rounding of its result."""
import numpy as np
import pytest
import torch

from tests.test_gpu_rope import _k

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e7, 1e9])
def test_sines_of_small_angles(base, interleaved):
    pairs = 64
    inv = (base ** (-np.arange(pairs) / pairs)).astype(np.float32)
    pos = np.array([1, 2, 3, 5, 7, -1, -6, 1000, 2**20 + 1, 0])
    x = torch.zeros(len(pos), 2, 2 * pairs, dtype=torch.bfloat16)
    a = torch.arange(pairs) * 2 if interleaved else torch.arange(pairs)
    b = a + 1 if interleaved else a + pairs
    x[:, 0, a] = 1.0
    x[:, 1, b] = 1.0
    out = torch.zeros_like(x).cuda()
    _k().kvq_qk_norm_rope(x.cuda(), None, torch.from_numpy(pos).cuda(), torch.from_numpy(inv).cuda(), out, None, interleaved=interleaved)
    out = out.cpu().double().numpy()
    angle = pos[:, None].astype(np.longdouble) * inv.astype(np.longdouble)
    sin, cos = np.sin(angle).astype(np.float64), np.cos(angle).astype(np.float64)
    # half a step of bf16, 2^-8 of the value.  float32: the sine's argument is rounded twice and its factor
    # once, the series and the products after it within 2^-22, 2^-20 of the value in all.  The angle: its
    # fraction of a turn is cut at 2^-64 per position, which inv_freq > 2^-31 makes 2^-30 of it; what the
    # reduction leaves of a large angle is off by 2^-64 turns times the position and the last place of its
    # conversion, below 2^-40 in absolute terms here
    room = 2.0 ** -8 + 2.0 ** -20 + 2.0 ** -30
    for head, (first, second) in enumerate(((cos, sin), (-sin, cos))):
        for dims, ref in ((a, first), (b, second)):
            got = out[:, head, dims.numpy()]
            assert np.all(np.abs(got - ref) <= room * np.abs(ref) + 2.0 ** -40), head
