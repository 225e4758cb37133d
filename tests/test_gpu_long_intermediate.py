"""swiglu_mlp_lora of a few bf16 rows keeps two pieces of h, 22 bits, whatever the length of the
intermediate: past 131072 columns the down projection leaves the streamed form for the tiles."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import rel_err, x_values
from lora_bounds import adapters, codes, device_lora, device_weight
from test_gpu_lora import _mlp, _x

pytestmark = pytest.mark.gpu


# float32 scales, sums and pieces of 22 bits: each below 2^-22 of a value, and together in 1e-6 (one piece: 2^-12.8 = 1.4e-4)
@pytest.mark.parametrize("I", [8192, 278528])
@pytest.mark.parametrize("M", [1, 4, 8])
def test_bits_of_h(M, I):
    H, R = 64, 8
    ws3 = [codes(K, N, 1 + i) for i, (K, N) in enumerate(((H, I), (H, I), (I, H)))]
    lo = adapters(2, R, I, H, 4)
    ids = (np.arange(M) % 3 - 1).astype(np.int32)
    x = _x(M, H, "bf16", 5)
    y = _mlp(x, [device_weight(w) for w in ws3], [None, None, device_lora(lo)], torch.from_numpy(ids).cuda(),
             torch.float32)
    err = rel_err(y, O.swiglu_mlp_lora64(x_values(x), *ws3, None, None, lo, ids))
    print(f"mlp_lora bf16 M={M} I={I} relF={err:.3e}", flush=True)
    assert err <= 1e-6
