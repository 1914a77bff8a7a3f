"""What the gated delta rule's outputs keep beyond a norm over whole outputs: the same bits with and without a checkpoint, roundings
to bf16 that are those of the fp32 result, decay gradients of heads that forget."""

import numpy as np
import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_deltarule import CASES, _case, _fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_a_checkpoint_changes_no_bit(ss, B, L, H, G, K, V, opt, dtype):
    import torch
    d = _case(B, L, H, G, K, V, dtype, seed=L + K + V, **opt)
    o, _, h = _fwd(ss, d)
    o2, _, h2 = _fwd(ss, d, want_ckpt=False)
    assert torch.equal(o, o2) and torch.equal(h, h2)
