"""The bound that the fp32 products are held to, on the CPU: what the kernels do stays inside, and
every part that could be lost is seen."""
import pytest

import gated_planes as gp


def _operands(K, seed=1, operands=1):
    return [(gp.planed(6, K, seed=seed + 2 * i), gp.planed(5, K, seed=seed + 2 * i + 1))
            for i in range(operands)]


def _runs(K, operands=1):
    return operands * -(-K // (gp.RUN * gp.STAGE))


def test_planes_are_positive_and_whole():
    x = gp.planed(64, 64, seed=4)
    p = gp.planes(x)
    assert all((q > 0).all() for q in p) and (sum(p) == x.double()).all()
    for q, lo, hi in zip(p, (1, 1.5 * 2.0 ** -9, 1.5 * 2.0 ** -18), (1.25, 2.0 ** -8, 2.0 ** -17)):
        assert lo <= q.min() and q.max() < hi


@pytest.mark.parametrize("operands", [1, 2])
@pytest.mark.parametrize("K", [40, 256, 300, 512, 1024, 2048])
def test_what_the_kernels_do_is_inside(K, operands):
    ops = _operands(K, operands=operands)
    assert gp.off(gp.emulated(ops), gp.exact(ops)) <= gp.bound(_runs(K, operands))


@pytest.mark.parametrize("product", gp.PRODUCTS)
@pytest.mark.parametrize("K", [40, 300, 512, 1024, 2048, 4096])
def test_a_product_left_out_is_seen(K, product):
    ops = _operands(K)
    got = gp.emulated(ops, lambda o, u, p: p == product)
    assert gp.off(got, gp.exact(ops)) > gp.bound(_runs(K) + 8)


@pytest.mark.parametrize("product", gp.PRODUCTS)
@pytest.mark.parametrize("run", [0, 1])
def test_a_product_left_out_of_one_run_is_seen(run, product):
    ops = _operands(512)
    got = gp.emulated(ops, lambda o, u, p: u == run and p == product)
    assert gp.off(got, gp.exact(ops)) > gp.bound(_runs(512))


@pytest.mark.parametrize("product", gp.PRODUCTS)
@pytest.mark.parametrize("K", [256, 1024])
def test_a_product_left_out_of_the_second_operand_is_seen(K, product):
    first, second = _operands(K, operands=2)
    ops = [first, (2 * second[0], second[1])]
    got = gp.emulated(ops, lambda o, u, p: o == 1 and p == product)
    assert gp.off(got, gp.exact(ops)) > gp.bound(_runs(K, 2))


def test_one_sum_without_runs_is_seen():
    ops = _operands(2048)
    assert gp.off(gp.emulated(ops, run_stages=32), gp.exact(ops)) > gp.bound(_runs(2048))
