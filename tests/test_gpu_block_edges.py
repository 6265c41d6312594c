"""The block-scaled cache's operators at the edges of what include/kvq.h promises."""
import numpy as np
import pytest

import block_ref as R
from test_gpu_block_cache import assert_cache, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,P,D", [(3, 32, 64), (1, 64, 128), (1, 32, 64)])
def test_append_prompts_with_short_tails(kvq, H, P, D):
    """Few kv heads and several pages a CTA, full ones and short tails in turn: the maxima
    that the warps of a full page exchange are its own."""
    rng = np.random.default_rng([H, P, D, 31])
    n = rng.integers(1, 3, 900) * P + rng.integers(1, 17, 900)
    s = R.Step(rng, n, n, H, P, D)
    mag = np.exp2(rng.integers(-12, 13, (s.N, H, 1)))
    kt, vt = (R.bf16(rng.standard_normal((s.N, H, D)) * mag) for _ in range(2))
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kt.double().numpy(), vt.double().numpy()], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt))
    assert err == 0
    assert_cache(c, pools, scales)
