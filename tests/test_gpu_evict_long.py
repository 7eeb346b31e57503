"""Evictions from rows of more than 262144 slots, which sixteen CTAs share: byte for byte."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_evict import check, evict, weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hkv,keep,recent,kind", [
    (262145, 1, 1000, 10, "random"), (270001, 2, 100000, 512, "ties"), (270001, 2, 270000, 0, "random"),
    (300007, 1, 4096, 4096, "wide"), (300007, 2, 5, 0, "equal"), (524289, 1, 131072, 1, "odd"),
    (1000003, 1, 65536, 256, "ties")])
def test_rows_that_sixteen_ctas_share(n, hkv, keep, recent, kind):
    case = Case([n], hkv, hkv, 8, "bf16", 64, seed=2, q_gain=1.0)
    w = weights_of(kind, 1, hkv, n, seed=n).cuda()
    before = case.pool.clone()
    check(case, before, w, [keep], recent, evict(case, w, [keep], recent))


def test_ragged_rows_beside_one_another():
    lens, keep = [270001, 0, 77, 150000], [50000, 9, 100, 149999]
    case = Case(lens, 2, 2, 8, "f16", 64, seed=3, q_gain=1.0)
    w = weights_of("ties", 4, 2, 270001, seed=3).cuda()
    before = case.pool.clone()
    check(case, before, w, keep, 300, evict(case, w, keep, 300, want_index=False))
