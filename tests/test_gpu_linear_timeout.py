"""The forward product's bounded waits: with a limit far below the time that a
first load takes, both of its kernels end early, say so, and leave the device
usable."""
import numpy as np
import pytest
import torch

import grouped_fp8_weight_gb300 as dg
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def operands(ms, N, K):
    r = np.random.default_rng(N + K)
    code = lambda *s: oracle.e4m3_encode(r.standard_normal(s) * 60)  # noqa: E731
    x, w = code(sum(ms), K), code(len(ms), N, K)
    sx = np.exp(r.standard_normal((sum(ms), -(-K // 128)))).astype(np.float32)
    sw = (0.01 * np.exp(r.standard_normal((len(ms), -(-N // 128), -(-K // 128))))).astype(np.float32)
    return x, sx, w, sw


@pytest.mark.parametrize("ms,N,K", [
    ([600, 100], 512, 2048),      # CTA pairs: full tiles and a rest
    ([100] * 8, 256, 1024),       # CTA pairs: rests
    ([5, 9, 0, 1], 512, 2048),    # single CTAs, K shared in a cluster
    ([20] * 40, 2048, 512),       # single CTAs
])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(ms, N, K, monkeypatch):
    """A tenth of a microsecond: no load comes back from memory in that time."""
    ops = operands(ms, N, K)
    d = [torch.from_numpy(a).to(DEV) for a in ops]
    m = torch.tensor(ms, dtype=torch.int32, device=DEV)
    y = torch.zeros(sum(ms), N, dtype=torch.bfloat16, device=DEV)
    torch.zeros(1 << 27, device=DEV).add_(1.0)        # nothing of the operands in the L2 cache
    dg.dg_sync_check()
    monkeypatch.setenv("DG_WAIT_LIMIT_US", "0.1")
    dg.dg_m_grouped_fp8_linear(*d, y, m)
    with pytest.raises(dg.DGError) as e:
        dg.dg_sync_check()
    assert e.value.status == dg.DG_ERR_TIMEOUT
    dg.dg_sync_check()                                # the record was read and cleared
    monkeypatch.delenv("DG_WAIT_LIMIT_US")
    y.fill_(float("nan"))
    dg.dg_m_grouped_fp8_linear(*d, y, m)
    dg.dg_sync_check()
    want, S = oracle.mgrouped_fp8_linear(*ops, ms)
    err = np.abs(y.float().cpu().double().numpy() - want)
    assert np.all(err <= oracle.linear_bound(want, S))
