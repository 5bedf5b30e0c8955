"""Checkpoints of groups that routing leaves very uneven: half of all rows in one of them, many
with few or none.  Every row's bits are those of the rows saved and restored as one group."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("counts", [[4000] + [37] * 15, [0] * 15 + [5000], [1, 0, 3000, 0, 2, 900, 1, 1], [1] * 64, [3001] + [0] * 300])
@pytest.mark.parametrize("F,act,dtype", [(1792, "swiglu", BF), (328, "gelu", HF), (8, "none", BF)])
def test_hot_and_cold_groups(counts, F, act, dtype):
    rows, offsets = sum(counts) + 9, [0]
    for c in counts[:-1]:
        offsets.append(offsets[-1] + c)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((2, rows, F), generator=g, device="cuda").to(dtype)
    count, offset = ints([counts, counts[::-1]]), ints([offsets, [0] * len(counts)])
    run = 0
    for i, c in enumerate(counts[::-1]):
        offset[1, i] = run
        run += c
    codes, scales = ep.checkpoint(x, count, offset)
    want = [ep.checkpoint(x[r]) for r in range(2)]
    for r in range(2):
        assert same(codes[r, :run], want[r][0][:run]) and same(scales[r, :run], want[r][1][:run])
    y = ep.checkpoint_restore(codes, scales, count, offset, activation=act, dtype=dtype)
    for r in range(2):
        assert same(y[r, :run], ep.checkpoint_restore(*want[r], activation=act, dtype=dtype)[:run])
