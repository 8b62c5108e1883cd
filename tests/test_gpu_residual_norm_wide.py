"""The norms' backward pass over rows of more than 4096 elements, with several rows a block and
every cut of the gate groups, against the 64-bit reference: rows in registers up to 8192
elements, element by element beyond."""
import pytest
import torch

from test_gpu_residual_norm import DT, check, make, moved

import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("C", [8192, 5000, 4102, 5001])
@pytest.mark.parametrize("per", [1, 3, 20, 130, 400])
def test_rows_in_registers(dt, C, per):
    x, y, dr, dn, p = make(400, C, dt, "layer", "rms", per=per, seed=C + per)
    check(x, y, dr, dn, p, dt, f"{dt} {C} per {per}")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "none"), ("layer", "layer"), ("rms", "rms")])
@pytest.mark.parametrize("affine", [True, False])
def test_kinds(dt, post, pre, affine):
    for per in (1, 100):
        x, y, dr, dn, p = make(310, 6000, dt, post, pre, per=per, affine=affine, scale=affine)
        check(x, y, dr, dn, p, dt, f"{dt} {post} {pre} per {per}")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("R", [200, 700])
@pytest.mark.parametrize("per", [1, 3, 64, 65, 100, 700])
def test_element_by_element(dt, R, per):
    """Several tasks, groups cut into several, a short last one."""
    x, y, dr, dn, p = make(R, 8200, dt, "rms", "layer", per=min(per, R), seed=R + per)
    check(x, y, dr, dn, p, dt, f"{dt} {R} per {per}")


@pytest.mark.parametrize("per", [1, 8, 64])
def test_same_bits_every_time(per):
    for dt in DT:
        x, y, dr, dn, p = make(500, 8192, dt, "layer", "rms", per=per)
        p = moved(p, lambda t: t.cuda())
        args = [t.cuda() for t in (dr, dn, x, y)]
        a, b = (mec.residual_norm_backward(*args, **p) for _ in range(2))
        assert all(a[k] is b[k] is None or torch.equal(a[k], b[k]) for k in a)


def test_an_infinite_gate_stays_with_its_group():
    """Slots without a group add nothing to the sums, whatever the first group's gate is."""
    x, y, dr, _, p = make(10, 64, "f32", "layer", "none", per=1)
    p["gate"][0, 3] = float("inf")
    p = moved(p, lambda t: t.cuda())
    g = mec.residual_norm_backward(dr.cuda(), None, x.cuda(), y.cuda(), **p)
    assert float(g["db_post"][3]) == float("inf") * float(dr[0, 3].sign())
    assert bool(g["dw_post"][3].isinf()) and bool(g["dgate"].isfinite().all())
