"""Results that every rank gets are the same bits on every rank."""
import numpy as np
import pytest

from gpu_util import BF16, F32
from test_gpu_token_ops import coll, rng, run_logprob, shards  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cuts,dtype", [(300, [0, 700, 1401], F32), (2000, [0, 3000, 9000], BF16), (300, [0, 40000, 131072], BF16),
                                             (500, [0, 100, 200, 300, 400, 500, 600, 700, 801], F32)])
def test_logprob(coll, rows, cuts, dtype):
    g = rng(70, rows, len(cuts), dtype)
    zs, _ = shards(g.normal(0, 3, (rows, cuts[-1])), cuts, dtype)
    o, _ = run_logprob(coll, zs, [int(x) for x in g.integers(0, cuts[-1], rows)], 0.8, 4)
    for k, v in o.items():
        bits = v.cpu().numpy().view(np.uint32)
        differ = int((bits != bits[:1]).sum())
        assert differ == 0, (k, differ)
