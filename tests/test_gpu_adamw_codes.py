"""AdamW's 8-bit moments byte for byte: signs of zeros, moments that are not
finite, and blocks at the bottom of FP32's range."""
import numpy as np
import pytest
import torch

import grouped_fp8_weight_gb300 as dg
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


class State:
    """One tensor with 8-bit moments: codes and scales as given."""

    def __init__(self, g, m, v, sm, sv, p=None):
        n = len(g)
        d = lambda a, dt: torch.from_numpy(np.array(a)).to(DEV, dt)  # noqa: E731
        self.host = [np.array(a) for a in (np.zeros(n) if p is None else p, g, m, v, sm, sv)]
        self.p, self.g = d(self.host[0], torch.float32), d(g, torch.float32)
        self.m, self.v, self.sm, self.sv = (d(a, torch.uint8) for a in (m, v, sm, sv))

    def step(self, t, seed, **hyper):
        plan = dg.dg_adamw_plan([self.p], [self.g], [self.m], [self.v], [self.sm], [self.sv])
        dg.dg_adamw_step(plan, t, seed=seed, **hyper)
        dg.dg_sync_check()

    def check(self, t, seed, lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0):
        """Steps, and compares codes and scale bytes with the oracle's."""
        p, g, m, v, sm, sv = self.host
        F = np.float32
        m0 = oracle.moment_decode(m, sm).astype(F)
        r0 = oracle.moment_decode(v, sv).astype(F)
        with np.errstate(over="ignore", invalid="ignore"):
            m1, _, r1, _, _ = oracle.adamw(p, g.astype(F), m0, r0 * r0, t, lr, beta1, beta2, eps,
                                           weight_decay)
        bits = oracle.element_bits(len(g), seed, 0)
        self.step(t, seed, lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay)
        for code, scale, x, b, keep in ((self.m, self.sm, m1, bits >> np.uint64(16), False),
                                        (self.v, self.sv, r1, bits & np.uint64(0xFFFF), True)):
            c, s = oracle.moment_encode(x, b, keep)
            assert np.array_equal(scale.cpu().numpy(), s)
            got = code.cpu().numpy()
            assert np.array_equal(got, c), np.argwhere(got != c)[:4].tolist()
        return m1


def test_codes_keep_the_sign_of_zero():
    """Moments -0.0 and +0.0, and negative ones that round to zero."""
    n = 300
    m = np.where(np.arange(n) % 2, 0x80, 0x00)
    g = np.where(np.arange(n) % 3, -0.0, 0.0)
    g[0], g[128], g[256:] = 1.0, -1.0, np.where(np.arange(44) % 2, -1e-9, 1e-9)
    g[260] = 1.0
    s = State(g, m, np.zeros(n), np.full(3, 120), np.full(3, 120))
    m1 = s.check(3, 11)
    zero = (m1 == 0) & (np.arange(n) < 256)
    got = s.m.cpu().numpy()
    assert set(got[zero]) == {0x00, 0x80} and np.array_equal(got[zero] == 0x80, np.signbit(m1)[zero])


@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), -float("inf")])
def test_moments_that_are_not_finite_are_one_code(bad):
    r = np.random.default_rng(1)
    n = 400
    g = r.standard_normal(n)
    g[[0, 131, 399]] = bad
    codes = r.integers(1, 127, (2, n))
    codes[0] |= r.integers(0, 2, n) << 7
    s = State(g, codes[0], codes[1], np.full(4, 120), np.full(4, 118))
    s.check(7, 5)
    assert set(s.m.cpu().numpy()[[0, 131, 399]]) == {0x7F}
    assert set(s.v.cpu().numpy()[[0, 131, 399]]) == {0x7F}


def test_a_negative_moment_that_was_not_finite_stays_one_code():
    m = np.full(128, 0x3F)
    m[5], m[6] = 0xFF, 0x7F
    s = State(np.full(128, -0.5), m, np.full(128, 0x3F), np.full(1, 120), np.full(1, 120))
    s.check(2, 3)
    assert set(s.m.cpu().numpy()[[5, 6]]) == {0x7F}


@pytest.mark.parametrize("byte,beta1,seed", [(0, 0.1, 0), (0, 0.1, 1), (1, 0.1, 1), (2, 0.1, 0),
                                             (0, 0.9, 0), (1, 0.9, 0), (0, 0.0, 0), (8, 0.1, 0)])
def test_blocks_whose_scale_times_beta1_is_not_a_normal_number(byte, beta1, seed):
    """b1 (code * scale) in that order: with scales up to 2^-125 b1 * scale alone
    would lose bits that decide codes."""
    F, n = np.float32, 1 << 20
    r = np.random.default_rng(0)
    m = r.integers(1, 127, n) | (r.integers(0, 2, n) << 7)
    scale = np.full(n // 128, byte)
    if beta1 == 0.1 and byte < 3:        # the case decides something
        u = oracle.element_bits(n, seed, 0) >> np.uint64(16)
        codes = oracle.moment_decode(m, np.full(n // 128, 127)).astype(F)
        other = (F(beta1) * F(2.0 ** (byte - 127))) * codes
        mine = F(beta1) * oracle.moment_decode(m, scale).astype(F)
        assert not np.array_equal(oracle.moment_encode(other, u, False)[0],
                                  oracle.moment_encode(mine, u, False)[0])
    s = State(np.zeros(n), m, np.zeros(n), scale, np.zeros(n // 128))
    s.check(4, seed, beta1=beta1)
