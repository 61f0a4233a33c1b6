"""What the 8-bit moments' rounding does over many steps of steady gradients.

One step's rounding of r = sqrt(v) is right on average: E[r'] = r.  The next
step squares what is held, and E[r'^2] = r^2 + s (1 - s) h^2 for a grid step h
and a part s cut off.  A step moves r by |d| r, d = (1 - b2) / 2 (g^2 / v - 1),
so from a grid point s is about |d| r / h and the excess |d| r h.  With E |g^2 / v
- 1| = 4 phi(1) = 0.968 for normal gradients and h / r between 1/16 and 1/8, v
settles where (1 - b2) times its excess is that: 3 to 6 % high, whatever b2.  The
same noise against the pull (1 - b2) gives r a relative variance of a quarter of
0.968 h / r: 12 to 17 %.  m's recursion is linear, so its mean stays right."""
import pytest
import torch

import grouped_fp8_weight_gb300 as dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def value(codes, scales):
    e = scales.int().repeat_interleave(128)[:codes.numel()] - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), e)


def test_second_moment_settles_where_its_rounding_puts_it():
    n, steps, b1, b2, mean = 1 << 16, 9000, 0.9, 0.999, 0.25
    g = torch.Generator(device=DEV).manual_seed(1)
    p, grad = torch.zeros(n, device=DEV), torch.empty(n, device=DEV)
    m = torch.zeros(n, dtype=torch.uint8, device=DEV)
    v = torch.full((n,), 0x38, dtype=torch.uint8, device=DEV)        # r = 1
    sm, sv = (torch.full((n // 128,), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    plan = dg.dg_adamw_plan([p], [grad], [m], [v], [sm], [sv])
    means, seconds, spreads = [], [], []
    scale = (1 - mean ** 2) ** 0.5
    for t in range(steps):
        grad.normal_(generator=g).mul_(scale).add_(mean)             # E[g] = 1/4, E[g^2] = 1
        dg.dg_adamw_step(plan, t + 1, 0.0, b1, b2, seed=t)
        if t >= 7000 and t % 100 == 0:                               # seven time constants of v
            r = value(v, sv)
            means.append(value(m, sm).mean())
            seconds.append(r.square().mean())
            spreads.append((r / r.square().mean().sqrt() - 1).square().mean().sqrt())
    dg.dg_sync_check()
    avg = lambda x: float(torch.stack(x).mean())  # noqa: E731
    # the held m spreads by sqrt((1 - b1) / (1 + b1)) = 0.23 and its roundings by
    # less: 20 times n of them, of which one in about 10 is a new one
    assert abs(avg(means) - mean) < 5 * 0.3 / (20 * n / 10) ** 0.5
    # (a percent for |d| r being more than a small part of h, and for v's spread)
    assert 1.03 - 0.01 < avg(seconds) < 1.06 + 0.01
    assert 0.12 - 0.01 < avg(spreads) < 0.175 + 0.01
