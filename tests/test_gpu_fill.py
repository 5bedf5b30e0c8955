"""torch fills uninitialised memory under deterministic algorithms: what the calls leave
unspecified in their outputs is then the same in every run (NaN), as in torch's own."""
import pytest
import torch

import combine_ep_layout_06_gb300 as ep

pytestmark = pytest.mark.gpu


def rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def outputs():
    """Rows 20 and on belong to no group."""
    x, w = rand(40, 64), rand(1, 32, 64, seed=1)
    count, offset = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (20, 0))
    y, pre = ep.expert_product(x, w, count, offset, save_pre=True)
    dx, _, _ = ep.expert_product_backward(y, x, w, count, offset)
    codes, scales = ep.checkpoint(x, count, offset)
    back = ep.checkpoint_restore(codes, scales, count, offset)
    return dict(y=y, pre=pre, dx=dx, scales=scales, codes=codes.float(), back=back)


def test_uninitialised_rows_are_filled():
    torch.full((1 << 22,), 3.0, device="cuda")              # freed memory is not NaN by chance
    on, fill = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        for name, t in outputs().items():
            assert bool(t[20:].isnan().all()), name
            assert not bool(t[:20].isnan().any()), name
    finally:
        torch.use_deterministic_algorithms(on)
        torch.utils.deterministic.fill_uninitialized_memory = fill
