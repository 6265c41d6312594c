"""The block-scaled cache's operators at the edges of what include/kvq.h promises."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block_cache import assert_cache, dev, run_append

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


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend(kvq, s, q, max_q, table=None, ws=None, sm=None, abort=None):
    Hq, D = q.shape[1:]
    out = torch.full((q.shape[0], Hq, D), -77.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = kvq.block_workspace(s.B, max_q, Hq, s.H, D)
    kvq.kvq_block_attn(kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales)), q.cuda(), dev(s.tok_start),
                       dev(s.lens), dev(s.table if table is None else table), out, ws, max_q=max_q,
                       abort_mask=None if abort is None else dev(abort), sm_scale=sm, err_word=err)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), int(err.item())


def compare(got, want, tol):
    err = np.abs(got - want) - tol
    worst = np.unravel_index(np.nanargmax(err), err.shape)
    assert not np.isnan(got).any() and err.max() <= 0, \
        f"at {worst}: got {got[worst]}, want {want[worst]}, bound {tol[worst]}"


@pytest.mark.parametrize("D,max_q", [(64, 1), (64, 6), (128, 1), (128, 3), (128, 6)])
def test_largest_value_scales(kvq, D, max_q):
    """V scales up to the largest fp32, with codes so small that the values are finite: block_ref's
    bound, in which nothing depends on a scale's size."""
    rng = np.random.default_rng([D, max_q, 32])
    s = R.Step(rng, [1, max_q, 1], [200, 90, 640], 2, 16, D)
    s.v &= 0x87  # at most 7 2^-9
    e = rng.integers(124, 128, s.scales.shape[:2])
    s.scales[:, :, 1] = np.ldexp(rng.integers(4, 8, e.shape) / 4.0, e)
    s.scales[::3, :, 1] = np.float32(2.0 ** 127)
    s.scales[1::5, :, 1] = np.finfo(np.float32).max
    q, qx = R.values(rng, s.N, 8, D)
    want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, D ** -0.5, max_q=max_q)
    got, err = attend(kvq, s, q, max_q)
    assert err == 0
    compare(got, want, tol)
