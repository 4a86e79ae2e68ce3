"""dsa_latent_frontend for the query alone: lengths that the call looks at are checked, others are not."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa

from test_gpu_latent import Case

pytestmark = pytest.mark.gpu
QUERY_ALONE = dict(c_kv=None, k_rope=None, gamma_kv=None, lat_pool=None, block_table=None)


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


@pytest.mark.parametrize("n_q", [1, 4])
@pytest.mark.parametrize("bad", [0, -5, 257, 2 ** 31 - 1, -2 ** 31])
def test_the_query_alone_reports_bad_lengths(n_q, bad):
    """Without positions the lengths give them; with positions they are not looked at."""
    import torch

    c = Case([100, 70, 200], n_q, "fp8", True, False, seed=6, width=4)
    pool, ref = c.run()
    c.check(pool, ref)
    assert dsa.get_device_error(c.ws) == 0
    good = c.lens.copy()
    for b in range(3):
        c.lens = good.copy()
        c.lens[b] = bad
        _, out = c.run(**QUERY_ALONE)
        assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_CTX, b
        rest = [r for r in range(c.rows) if r // n_q != b]
        assert torch.equal(out[rest], ref[rest])
    c.positions = np.concatenate([np.arange(n - n_q, n) for n in good]).astype(np.int32)
    _, out = c.run(**QUERY_ALONE)
    assert dsa.get_device_error(c.ws) == 0 and torch.equal(out, ref)
