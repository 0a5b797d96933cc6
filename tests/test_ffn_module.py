"""The compiled binding of the feed-forward operators loads where the library is built, and refuses before any GPU work."""
import os

import pytest
import torch

import fp8_fine_grained_amax_amd as fg
from fp8_fine_grained_amax_amd import ffn


@pytest.fixture(scope="module")
def module():
    if not os.path.exists(os.path.join(os.path.dirname(ffn.__file__), "_ffn.so")):
        from fp8_fine_grained_amax_amd import build
        build.build()
    return ffn._ffn()


def test_module_is_in_the_package(module):
    assert os.path.dirname(module.__file__) == os.path.dirname(os.path.abspath(ffn.__file__))


def test_arguments_are_counted(module):
    for f in (module.linear, module.act_forward, module.act_backward, module.moe):
        with pytest.raises(TypeError, match="expected"):
            f(1)


@pytest.mark.parametrize("what", [None, 3, "z", torch.zeros(4, 128)])
def test_anything_but_a_gpu_tensor_is_refused(module, what):
    for call in (lambda: fg.fg_fp8_gemm_fprop_epilogue(what, what, what, what),
                 lambda: fg.fg_act_checkpoint_fwd(what, fg.FG_ACT_SILU),
                 lambda: fg.fg_act_checkpoint_bwd(what, what, what, fg.FG_ACT_SILU),
                 lambda: fg.fg_moe_few_tokens(what, what, what, what, what, what, what)):
        with pytest.raises(fg.Fp8fgError):
            call()
