"""slim_attention_decode_q4 under every way that it cuts its work: 4, 8 and 16
waves a workgroup, whole key heads and keys split over workgroups, lengths that
fit the plan and those that do not (max_len only plans the work)."""
import numpy as np
import pytest

from attention_helpers import bound, check, host, reference
from q4_helpers import q4_case
from test_attention_q4_gpu import env, run  # noqa: F401

pytestmark = pytest.mark.gpu

PLANS = (0, 100, 300, 600, 1100, 1500, 3000, 9000, 40000, 200000, 1 << 30)


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("bf16", 128), ("fp16", 256)])
@pytest.mark.parametrize("seqs,q_heads,kv_heads,longest", [(1, 8, 1, 6000), (1, 32, 8, 2500), (4, 8, 8, 1500), (9, 20, 10, 900),
                                                           (20, 16, 16, 400), (33, 8, 8, 400), (40, 16, 16, 200), (70, 8, 8, 200)])
def test_every_plan(env, dtype, dim, seqs, q_heads, kv_heads, longest):
    lens = np.random.default_rng(seqs).integers(0, longest + 1, seqs)
    lens[-1] = longest
    c = q4_case(env[0], 7, dtype, [int(n) for n in lens], q_heads, kv_heads, dim, 64)
    want, want_lse, mass = reference(c)
    most, seen = bound(c, want, mass), ~np.isneginf(want_lse)
    for max_len in (None, *PLANS):
        y, lse = run(env, c, lse=True, max_len=max_len)
        y, lse = host(y), host(lse)
        assert (np.abs(y - want) <= most).all(), f"max_len={max_len}"
        # (The bound of attention_helpers.check.)
        assert np.array_equal(~np.isneginf(lse), seen) and (np.abs(lse[seen] - want_lse[seen]) <= 2.0 ** -12 * (
            1 + np.abs(want_lse[seen]).max())).all(), f"max_len={max_len}: lse"
    y, lse = run(env, c, window=130, sinks=70, lse=True, max_len=longest)
    check(c, y, lse, 130, 70)
