"""Every shape that draft verification launches (clusters of 16, 8, 4 and 2 CTAs, one
CTA of 1024 or 512 threads), against the 64-bit reference and against one another.
Sizes are stated for 152 SMs."""
import pytest
import torch

from tests.test_gpu_verify import DT, _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


SHAPES = [  # batch, drafts, vocabulary
    (16, 2, 90000), (33, 1, 131071),          # clusters of eight
    (40, 1, 90001), (70, 1, 66000),           # of four, of two
    (100, 1, 41000), (152, 1, 49999),         # one CTA of 1024 threads
    (153, 1, 41001), (160, 1, 65536),         # one of 512, some SMs with two
]


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("B,K,V", SHAPES)
def test_shapes(pkv, B, K, V, dtype, lookup):
    t, q, x, ua, us = _case(B, K, V, dtype, seed=B)
    num = torch.arange(B, dtype=torch.int32, device="cuda") % (K + 2)
    num[num > K] = K
    _check(pkv, t, None if lookup else q, x, ua, us, num)


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("V", [131072, 116985])
def test_the_same_answer_in_every_shape(pkv, V, lookup):
    """160 sequences together, and in batches that other shapes serve."""
    t, q, x, ua, us = _case(160, 1, V, seed=V, sharp=3.0)
    q = None if lookup else q
    tokens, acc = _run(pkv, t, q, x, ua, us)
    for lo, hi in ((0, 100), (60, 136), (5, 45), (100, 116), (159, 160), (3, 4)):
        at = slice(lo, hi)
        a, b = _run(pkv, t[at], None if lookup else q[at], x[at], ua[at], us[at])
        assert torch.equal(a, tokens[at]) and torch.equal(b, acc[at])


def test_rows_without_mass_and_saturated_ones(pkv):
    """In one CTA of 1024 threads and in clusters of eight: the second pass, sums at 16."""
    for B, V in ((100, 41003), (16, 90001)):
        t, q, x, ua, us = _case(B, 1, V, seed=V)
        t[0], t[1], t[2] = 0.0, 1.0, 0.0
        t[2, :, V - 1] = 1e-3
        q[3, 0], q[4, 0] = 1.0, t[4, 0]                      # residuals without mass
        ua[3:5] = 1.0
        _check(pkv, t, q, x, ua, us)
        _check(pkv, t, None, x, ua, us)
