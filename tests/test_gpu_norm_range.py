"""Head norms where float32 squares of bf16 values overflow or underflow, and
where a value times its weight does: x / sqrt(mean x^2 + eps) * w all the same."""
import numpy as np
import pytest
import torch

from oracle import rotary
from tests.test_gpu_rope import _inputs, _k, _rows_ok, _slots, _turn

pytestmark = pytest.mark.gpu


def _norm(q, w, eps, **more):
    out = torch.full_like(q, 9.0)
    _k().kvq_qk_norm_rope(q, None, more.pop("positions", None), more.pop("inv_freq", None), out, None, q_weight=w, eps=eps, **more)
    return out


def _check(out, x, w, eps, **host):
    """To the bounds of the rows that float32 holds: a power of two that scales a row is exact."""
    host = {"positions": None, "inv_freq": None, **host}
    x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    # a bf16 result below the normal numbers, or of float32 factors there, is off by 2^-133 at most
    _rows_ok(out, rotary.turn(x, **host, weight=w, eps=eps), rotary.slop(x, w, eps) + 2.0 ** -133)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30, 1e-45, 1e30])
def test_rows_of_any_size(dim, eps):
    """Each row times another power of two, from the subnormal numbers to the largest."""
    eps = float(np.float32(eps))
    gen = torch.Generator().manual_seed(dim)
    x = torch.randn(9, 3, dim, generator=gen).double()
    power = torch.tensor([-126, -100, -64, -20, 0, 50, 64, 100, 125]).double()
    x = (x * 2.0 ** power[:, None, None]).bfloat16()
    assert torch.isfinite(x).all()
    w = (1 + 0.4 * torch.randn(dim, generator=gen)).bfloat16()
    _check(_norm(x.cuda(), w.cuda(), eps), x, w, eps)


@pytest.mark.parametrize("size", [1e20, 1e30, 3e38, 1e-22, 1e-30, 1e-38, 1e-40])
def test_one_value_of_a_row(size):
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 5], x[1, 0, 63] = size, -size
    out = _norm(x.cuda(), torch.ones(64, dtype=torch.bfloat16, device="cuda"), 0.0)
    assert float(out[0, 0, 5]) == 8.0 and float(out[1, 0, 63]) == -8.0 and int((out != 0).sum()) == 2


@pytest.mark.parametrize("size,weight", [(1e10, 1e30), (1e15, 3e36), (1.0, 1e38), (3e38, 1e-30), (1e-12, 1e-30), (1e-30, 1e30)])
def test_weights_that_take_a_product_out_of_float32(size, weight):
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn(5, 2, 128, generator=gen).clamp(-1, 1) * size).bfloat16()
    w = (torch.rand(128, generator=gen) * weight).bfloat16()
    pos, inv = torch.arange(5) * 7, torch.rand(64, generator=gen)
    out = _norm(x.cuda(), w.cuda(), 0.0, positions=pos.cuda(), inv_freq=inv.cuda())
    _check(out, x, w, 0.0, positions=pos.numpy(), inv_freq=inv.numpy())


def test_infinities_nan_and_zeros_stay_what_the_formula_makes_of_them():
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 4], x[2, 0] = float("inf"), float("nan"), 0.0
    out = _norm(x.cuda(), torch.ones(64, dtype=torch.bfloat16, device="cuda"), 0.0).cpu()
    want = torch.ones(4, 2, 64, dtype=torch.bfloat16)
    want[0, 0], want[1, 0], want[2, 0] = 0.0, float("nan"), float("nan")  # x / inf, x / NaN, 0 / 0
    want[0, 0, 3] = float("nan")
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_other_rows_keep_their_bits(dim):
    """A row's result does not depend on what its neighbours hold."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(40, 5, dim, generator=gen).bfloat16().cuda()
    w = (1 + 0.4 * torch.randn(dim, generator=gen)).bfloat16().cuda()
    alone = _norm(x, w, 1e-6)
    odd = torch.zeros(40, 5, dtype=torch.bool)
    odd[::3, 1] = odd[5] = odd[17, 2] = True
    y = x.clone()
    y[odd] = (y[odd].double() * 2.0 ** 90).bfloat16()
    out = _norm(y, w, 1e-6)
    assert torch.equal(out[~odd], alone[~odd])
    _check(out[odd][:, None], y[odd][:, None], w, 1e-6)


def test_keys_on_their_way_into_the_cache():
    k = _k()
    T, H, D = 50, 2, 128
    (_, kk, v), _ = _inputs(T, 1, H, D, seed=3)
    kk = (kk.double() * 2.0 ** torch.randint(-100, 120, (T, H, 1), generator=torch.Generator().manual_seed(1)).cuda()).bfloat16()
    dev, more, host, w = _turn(T, D, 1, True, D, 5000)
    slots, blocks = _slots(T, "middle")
    sd = torch.from_numpy(slots).cuda()
    kd, vd = k.alloc_kv_cache(blocks, H, D, "bf16", fill=0)
    more["eps"] = 0.0
    k.kvq_rope_and_cache(None, kk, v, **dev, slot_mapping=sd, k_cache=kd, v_cache=vd, cache_dtype="bf16", **more)
    ko, vo = torch.zeros_like(kk), torch.zeros_like(kk)
    k.kvq_gather_cache(sd, kd, vd, ko, vo, cache_dtype="bf16")
    _rows_ok(ko, rotary.turn(kk.double().cpu().numpy(), **host, weight=w[1], eps=0.0),
             rotary.slop(kk.double().cpu().numpy(), w[1], 0.0) + 2.0 ** -133)
    assert torch.equal(vo, v)
