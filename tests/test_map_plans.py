"""The plans that the GPU tests of several rounds, runs and chunks rely on
(map_plans.py): what each of their cases makes the operators do."""
import pytest

import map_plans as plans


@pytest.mark.parametrize("shape, G, dtype, grad", plans.ROUNDS_ALONE)
def test_single_ctas_take_several_units_and_a_narrower_last_slab(shape, G, dtype, grad):
    assert all(plans.fewest_rounds(p) >= 2 for p in plans.cluster_plans(shape, G, dtype, grad))
    cl, keep, units, gs, slabs = plans.likely_plan(shape, G, dtype, grad)
    assert cl == 1 and keep == 2 and slabs > 1 and G - (slabs - 1) * gs == 1 < gs


@pytest.mark.parametrize("shape, G, dtype, grad", plans.ROUNDS_CLUSTERS)
def test_clusters_take_several_units(shape, G, dtype, grad):
    every = plans.cluster_plans(shape, G, dtype, grad)
    assert every and all(p[0] > 1 and plans.fewest_rounds(p) >= 2 for p in every)


@pytest.mark.parametrize("shape, G, dtype", plans.MANY_CHUNKS)
@pytest.mark.parametrize("grad", [False, True])
def test_joins_of_many_chunks(shape, G, dtype, grad):
    assert not plans.cluster_plans(shape, G, dtype, grad)
    chunks, px, walk = plans.pass_plan(shape, 16 // plans.SIZE[dtype], grad)
    # 64 rows of threads, four chunks each, and a last chunk that is shorter
    assert chunks > 4 * 64 and (shape[1] * shape[2]) % px and walk <= 1024


def test_resizes_walk_runs_with_rows_ahead():
    seen = {}
    for N, geo, C in plans.RESIZES:
        for dtype in plans.SIZE:
            readers, run, ahead = plans.gradient_plan(N, geo, C, dtype)
            assert run > 1 and ahead > 1, (geo, dtype)
            seen.setdefault((readers, plans.SIZE[dtype]), set()).add((run, ahead))
            assert plans.forward_run(N, geo, C, dtype) > 1
    assert set(seen) == {(r, s) for r in (4, 6, 8) for s in (2, 4)}
    assert {run for got in seen.values() for run, _ in got} >= {4, 8, 16, 32}
    assert {plans.forward_run(N, geo, C, t) for N, geo, C in plans.RESIZES for t in plans.SIZE} >= {8, 16}
    assert plans.gradient_plan(*plans.TABLE, "bf16", True)[1:] == (4, 3)
