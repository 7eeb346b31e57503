"""Chunks of values as large and as small as bf16 holds beside their sums, under references
that climb tile after tile."""
import pytest
import torch

from tests.scored_reference import Case, slopes
from tests.test_gpu_scored import run

pytestmark = pytest.mark.gpu


def climbing(case, step):
    """Keys of KV head 0 along the first query head's direction, scores `step` more a tile."""
    for b, n in enumerate(case.lens):
        t = torch.arange(n, device="cuda")
        block = case.tables[b].long()[t // case.bs]
        d = case.q[b, -1, 0].float()
        k = d / d.norm() ** 2 * case.dim ** 0.5 * (step * (t // 64))[:, None]
        case.pool[block, 0, 0, 0, t % case.bs] = k.to(case.pool.dtype)


@pytest.mark.parametrize("power", [-70, 90, 105])
@pytest.mark.parametrize("step", [0.0, 3.0, 9.0, 20.0])
@pytest.mark.parametrize("rules", ["none", "cap", "slopes"])
def test_values_of_every_size(rules, step, power):
    case = Case([640, 200, 70], 8, 2, 128, "bf16", 16, 40, seed=41, q_gain=1.0)
    if step:
        climbing(case, step)
    case.pool[:, 1] = (case.pool[:, 1].float() * 2.0 ** power).to(torch.bfloat16)
    r = {"none": {}, "cap": dict(cap=200.0), "slopes": dict(slopes=slopes(8))}[rules]
    case.check(run(case, torch.float32, **r), case.reference(**r))
