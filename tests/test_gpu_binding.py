"""What the compiled binding leaves visible to torch: the outputs it allocates."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import fp8_fine_grained_amax_amd as fg
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


class Names(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(func.overloadpacket._qualified_op_name)
        return func(*args, **(kwargs or {}))


def calls():
    x, gamma = torch.ones(2, 256, device=device(), dtype=torch.bfloat16), torch.ones(256, device=device())
    n = fg.fg_norm_quantize(x, gamma)
    return {5: lambda: fg.fg_norm_quantize(x, gamma, with_y=True),               # codes, scales, y, mean, rstd
            3: lambda: fg.fg_norm_bwd(x, n.mean, n.rstd, gamma, x, bias_grad=True),
            2: lambda: fg.fg_orthogonalize(x),                                      # the workspace too
            0: lambda: fg.fg_norm_quantize(x, gamma, out=n)}


def test_dispatch_modes_see_allocations():
    for count, call in calls().items():
        for _ in range(2):
            with Names() as mode:
                call()
            assert mode.seen == ["aten::empty"] * count, count


@pytest.mark.parametrize("fill", [False, True])
def test_profilers_and_the_fill_of_new_memory(fill):
    for count, call in calls().items():
        torch.use_deterministic_algorithms(fill)
        try:
            with torch.autograd.profiler.profile() as p:
                call()
        finally:
            torch.use_deterministic_algorithms(False)
        names = [e.name for e in p.function_events]
        assert names.count("aten::empty") >= count and (count == 0 or ("aten::fill_" in names) == fill), (count, names)


def test_results_are_the_same_when_watched():
    for call in calls().values():
        want = call()
        with Names():
            got = call()
        torch.use_deterministic_algorithms(True)
        try:
            filled = call()
        finally:
            torch.use_deterministic_algorithms(False)
        for a, b, c in zip(*((r if isinstance(r, tuple) else (r,)) for r in (want, got, filled))):
            assert (a is None and b is None and c is None) or (torch.equal(a, b) and torch.equal(a, c))
