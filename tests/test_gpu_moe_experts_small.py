"""An expert of up to eight tokens has h in two halves whichever launch serves it: its tokens are as exact as the output's own
rounding, also where the call's other experts have hundreds."""
import numpy as np
import pytest
import torch

import model_oracle as mo
from gpu_util import say
from test_gpu_moe_layer import layer, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,eight", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("few", [1, 5, 8])
@pytest.mark.parametrize("tokens,experts,dim,hidden", [(300, 2, 256, 512), (100, 3, 1040, 272), (180, 130, 272, 1040)])
def test_few_tokens_beside_a_crowd(dtype, eight, few, tokens, experts, dim, hidden):
    x, w_in, w_out, ids, weights, s_in, s_out = layer(tokens + few, tokens, experts, 1, dim, hidden, dtype, eight)
    ids[:] = 0
    ids[-few:] = experts - 1
    args = (x, w_in, w_out, ids, weights, s_in, s_out)
    ref, bound = mo.experts(*args)
    got = on_gpu(*args)
    mo.within(got, ref, bound, "all tokens")
    off = np.linalg.norm(mo.f64(got)[-few:] - ref[-few:])
    own = np.linalg.norm(mo.f64(torch.from_numpy(ref[-few:]).to(dtype)) - ref[-few:])
    say("off by %.3f of the output's own rounding" % (off / own))
    assert off <= 1.1 * own, (off, own)
