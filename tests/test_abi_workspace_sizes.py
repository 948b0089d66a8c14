"""CPU: a workspace sized for the largest call serves the smaller ones: the sizes
do not fall as a prompt, or a selection's batch, beams, vocabulary or number of
places, grows."""
import ctypes as C
import random

import pytest

from tests.test_abi import lib  # noqa: F401  (a fixture)
from tests.test_abi_ssm_beam import sd


@pytest.fixture
def sizes(lib):  # noqa: F811
    lib.gdn_ssm_prefill_workspace_bytes.restype = C.c_size_t
    lib.gdn_beam_select_workspace_bytes.restype = C.c_size_t
    return (lambda d, T: lib.gdn_ssm_prefill_workspace_bytes(C.byref(d), T),
            lambda *a: lib.gdn_beam_select_workspace_bytes(*a))


def test_prompt_sizes_by_hand(sizes):
    d = sd(batch=1, num_heads=32, num_groups=1, head_dim=64, state_dim=128)
    assert 0 < sizes[0](d, 4096) <= sizes[0](d, 4160)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("P,N", [(32, 32), (64, 128), (128, 128), (64, 256)])
def test_prompt_sizes_grow_with_the_prompt(sizes, P, N, act):
    for B, H, G in ((1, 1, 1), (1, 32, 1), (3, 23, 1), (2, 48, 16), (8, 64, 2), (40, 64, 1)):
        d = sd(batch=B, num_heads=H, num_groups=G, head_dim=P, state_dim=N, act_dtype=act)
        lengths = [*range(1, 1400), *range(1400, 70000, 61), 1 << 20, (1 << 20) + 64, 1 << 22]
        got = [sizes[0](d, T) for T in lengths]
        assert got[0] > 0
        for a, b, T in zip(got, got[1:], lengths[1:]):
            assert a <= b, (B, H, G, T)


def test_select_sizes_by_hand(sizes):
    assert 0 < sizes[1](16, 4, 128000, 4) <= sizes[1](30, 4, 128000, 4)


def test_select_sizes_grow_with_every_argument(sizes):
    r = random.Random(1)
    for _ in range(20000):
        a = [r.choice([1, 2, 3, 16, 30, 100, 513, 1024, 4000]), r.randint(1, 32), int(10 ** r.uniform(2, 6)), r.randint(1, 64)]
        b = list(a)
        k = r.randrange(4)
        b[k] = min(b[k] + r.choice([1, 2, 3, 7, 100, 5000]), [30000, 32, 1 << 25, 64][k])
        assert 0 < sizes[1](*a) <= sizes[1](*b), (a, b)
