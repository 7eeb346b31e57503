"""Capped chunks (two threads a row): block scales, rows of very different size, keys that
raise a row's largest score tile after tile, signs of the scale."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import expand, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rules", [dict(cap=8.0), dict(cap=12.0, docs=True), dict(cap=5.0, window=70)])
@pytest.mark.parametrize("kv,scaled", [("bf16", False), ("f16", False), ("e4m3", False), ("e4m3", True)])
def test_rows_of_every_size(kv, scaled, rules):
    case = Case([333, 64, 90, 0, 700], 8, 2, 128, kv, 16, 48, seed=21, block_scales=scaled)
    size = torch.arange(case.q.numel() // 128, device="cuda") * 5 % 17 - 12    # 2^-12 .. 2^4
    case.q = (case.q.view(-1, 128).float() * torch.exp2(size.float())[:, None]).to(
        case.q.dtype).view(case.q.shape)
    r = expand(case, rules)
    want = case.reference(**r)
    case.check(run(case, torch.float32, **r), want)
    case.check(run(case, **r), want)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("cap", [0.0, 200.0])
def test_references_that_move_in_every_tile(kv, cap):
    # keys along the first query head's direction, longer from tile to tile: the first head's
    # scores climb by some 20 a tile of 64, its neighbours' hardly
    case = Case([640, 200], 8, 2, 128, kv, 64, 40, seed=22, q_gain=1.0)
    for b, n in enumerate(case.lens):
        t = torch.arange(n, device="cuda")
        block = case.tables[b].long()[t // 64]
        d = case.q[b, -1, 0].float()
        k = d / d.norm() ** 2 * 128 ** 0.5 * (20.0 * (t // 64))[:, None] / 3
        if kv == "e4m3":
            rows = (k / case.k_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            rows = k.to(case.pool.dtype)
        case.pool[block, 0, 0, 0, t % 64] = rows
    r = dict(cap=cap) if cap else {}
    want = case.reference(**r)
    case.check(run(case, torch.float32, **r), want)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.4])
def test_scale_sign_and_size(scale):
    for kv in ("bf16", "e4m3"):
        case = Case([130, 217], 8, 2, 128, kv, 16, 40, seed=23, q_gain=1.0)
        case.check(run(case, torch.float32, scale=scale, cap=15.0),
                   case.reference(scale=scale, cap=15.0))
