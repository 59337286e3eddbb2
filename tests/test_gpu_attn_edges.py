"""Attention over the FP4 cache (include/rfpx_attn.h) at the edges of what a
caller may hand in, with the rows and tolerances of test_gpu_attn.py."""
import pytest

import block_quantized_expert_amd as bqe
from test_gpu_attn import Case, attend64, check_lse, check_out, torch

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- large scores

@pytest.mark.parametrize("d,scale", [(64, 0.125), (128, 1.0), (128, 128 ** -0.5)])
@pytest.mark.parametrize("low", [2.0 ** 30, 2.0 ** 40, 2.0 ** 90])
def test_many_rows_end_at_any_score(d, scale, low):
    """Scores of 2^30 and more, where the room that k_attn_chunk leaves above a
    row's maximum is lost to rounding: every tile is done with, and the rows of
    ordinary scores in the same waves are right."""
    t = torch()
    # 64 splits with a tile or none in each, and one split of several tiles
    for hk, heads, plan in ((2, 16, 65536), (128, 256, 1024)):
        c = Case([300], [40], hk, d, 64, t.bfloat16, seed=d, capacity=plan)
        g = t.Generator(device="cuda").manual_seed(int(100 * scale))
        q = t.randn((c.rows, heads, d), generator=g, device="cuda") * 1.3
        q[:, 1::2] *= low * (1 + t.rand((c.rows, heads // 2, 1), generator=g, device="cuda"))
        q = q.to(t.bfloat16)
        z = t.zeros((c.rows, heads), device="cuda")
        out = bqe.rfpx_attn_forward(c.cache, c.planned(plan), q, scale, lse=z)
        heads_seen = 16  # of the first kv heads: the plain form takes its time
        (k, v), = c.values()
        c.hk = heads_seen * hk // heads
        c.values = lambda: [(k[:, :c.hk], v[:, :c.hk])]
        ref = attend64(c, q[:, :heads_seen], scale)
        even = {n: x[:, 0:heads_seen:2] for n, x in ref.items() if n not in ("w", "dw")}
        check_out(out[:, 0:heads_seen:2], even, t.bfloat16, slice(0, c.rows))
        check_lse(z[:, 0:heads_seen:2], even, slice(0, c.rows))
