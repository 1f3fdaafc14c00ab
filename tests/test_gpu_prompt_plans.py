"""Sequence attention in every plan that the sizes of a call choose: rows and waves of a workgroup in the forward, dQ and
dK/dV, parts of a key head's query heads, with queries of few keys in one and two parts; sequences of one length and packed
ones (GPU). References and tolerances are those of tests/test_gpu_prompt.py."""
import pytest
import torch

from test_gpu_prompt import BF, F32, bounds, check, make

pytestmark = pytest.mark.gpu

# sequences, tokens, heads and window; in parentheses blocks of 32 rows and waves of each, S, where bf16 / 128 channels first
# takes them (64 channels and fp32 take other ones at the same sizes)
CALLS = [(1, 2, (1, 1), 0), (1, 2, (2, 1), 0), (8, 60, (40, 2), 0),          # one tile: alone
         (1, 100, (1, 1), 0), (1, 100, (2, 1), 0), (1, 130, (16, 16), 0),    # few blocks: one by four waves
         (1, 130, (16, 4), 0), (1, 130, (64, 64), 0), (1, 130, (64, 8), 0),  # two by four, and parts
         (1, 130, (64, 8), 70), (4, 100, (24, 24), 0),                       # two by four in two parts
         (16, 130, (8, 8), 0), (16, 130, (8, 2), 0),                         # four alone
         (16, 130, (16, 16), 0), (16, 130, (16, 4), 0),                      # 64 channels: four alone
         (16, 130, (32, 32), 0), (8, 130, (64, 8), 0),                       # fp32: four alone
         (1, 520, (32, 32), 0), (1, 520, (40, 2), 0),                        # by two waves
         (1, 520, (64, 64), 0), (1, 520, (64, 8), 0),                        # 64 channels: by two
         (4, 100, (64, 64), 70), (4, 100, (64, 8), 70),                      # 64 channels: by two in two parts
         (1, 1100, (16, 16), 0), (1, 1100, (16, 2), 300), (1, 1500, (16, 4), 0)]  # long walks by four


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,T,heads,window", CALLS)
def test_plans(dtype, D, N, T, heads, window):
    args = make(N * T, *heads, D, dtype, seed=60)
    check(*(x.view(N, T, -1, D) for x in args), bounds([T] * N), window=window, packed=False)
    cut = [T // 4 if i % 2 else -(T // 4) for i in range(N - N % 2)] + [0] * (N % 2)
    check(*args, bounds([T + c for c in cut]), window=window)


@pytest.mark.parametrize("N", [63, 64])
@pytest.mark.parametrize("heads,D", [((8, 8), 128), ((2, 1), 64)])
def test_as_many_sequences_as_lanes(N, heads, D):
    # the longest list that is taken longest tile first
    lens = [(11 * i) % 90 for i in range(N)]
    check(*make(sum(lens), *heads, D, BF, seed=61), bounds(lens))


@pytest.mark.parametrize("lens,heads,window", [([2100], (64, 64), 0), ([2100], (64, 64), 60), ([5, 3000, 1200], (48, 16), 0)])
def test_turns_of_many_heads(lens, heads, window):
    args = make(sum(lens), *heads, 128, BF, seed=62)
    check(*args, bounds(lens), window=window)
    if len(lens) == 1:
        check(*args, bounds(lens), window=window, packed=False)


@pytest.mark.parametrize("D", [64, 128])
def test_a_long_sequence_of_few_heads(D):
    # two waves a walk, with queries of few keys in two parts in the backward
    check(*make(8192, 8, 1, D, BF, seed=63), [0, 8192], packed=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_long_sequence_beside_short_ones(dtype):
    # plans go by the mean
    lens = [1500] + [5 + i for i in range(23)]
    check(*make(sum(lens), 8, 4, 128, dtype, seed=64), bounds(lens))
    lens = lens[1:] + lens[:1]
    check(*make(sum(lens), 8, 4, 64, dtype, seed=65), bounds(lens), window=400)
