"""The attention over the 8-bit cache held to its documented precision: probabilities to 2^-16 of their size
(16-bit types) or 2^-24 (fp32), fp32 queries to 2^-24, scores and sums in fp32 -- in prompts as in single tokens."""
import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref as ref
from gpu_util import say
from test_gpu_kv8 import F8, HALF_STEP, World, i32

pytestmark = pytest.mark.gpu
# of a probability, by the documentation; the exponential is good to an ulp (2^-23), its argument's rounding
# is one of the score's
KEPT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -16, "f32": 2.0 ** -24}
EXP = 2.0 ** -22


def within(got, gz, o, z, spread, amp, dtype, dims, n, what):
    """Output and lse within what the documentation leaves: a score is a sum over `dims` dims (the others are
    zero) of at most three exact terms a product (3 roundings of 2^-24 each), then its factor; the output sums n values of at most three terms each (a
    rounding a term), l sums n, and they are divided; the output is rounded once."""
    ds = ((3 * dims + 8) * 2.0 ** -24 + (2.0 ** -24 if dtype == "f32" else 0)) * amp
    tol = HALF_STEP[dtype] * o.abs() * 1.01 + (2 * ds[..., None] + KEPT[dtype] + EXP + (4 * n + 4) * 2.0 ** -24) * spread + 1e-30
    worst = ((got - o).abs() / tol).max()
    say("  worst of the tolerance", what, float(worst))
    assert bool(((got - o).abs() <= tol).all()), (what, float(worst))
    fin = torch.isfinite(z)
    assert torch.equal(fin, torch.isfinite(gz)), what
    dz = (gz[fin] - z[fin]).abs()
    # of l: n roundings and the exponential; the logarithm is good to 2^-22 of itself or of 1
    assert bool((dz <= ds[fin] + (n + 4) * 2.0 ** -24 + EXP + 2.0 ** -22 * z[fin].abs() + 2.0 ** -22).all()), (what, float(dz.max()))


def two_keys(T, hq, hk, D, dtype, seed):
    """Rows of which each sees two keys of weight (positions 0 and 1; the others score 200 less and add e^-200),
    with values of opposite signs in all ratios that two mantissas of e4m3 make: in some dims they nearly
    cancel, and what is left shows every bit that a probability lost."""
    w = World([T], 16, hk, D, seed=seed)
    k, v = torch.zeros(2, w.nb, 16, hk, D)
    k[..., 0] = -448.0
    first = int(w.tables[0, 0])
    k[first, :2] = 0.0
    k[first, :2, :, 1:5] = torch.randn(2, hk, 4, generator=w.g) * 60  # few dims: their sum rounds little
    d = torch.arange(D)
    v[first, 0] = 8.0 + d % 8
    v[first, 1] = -(8.0 + d // 8 % 8)
    w.kc, w.vc = k.clamp(-448, 448).to(F8), v.to(F8)
    w.ks.fill_(2.0 ** -6)
    q = w.heads(T, hq, dtype, D ** 0.5 / 4)
    q[:, :, 0] = 200 / 7 * D ** 0.5  # times -448 * 2^-6 * D^-0.5
    return w, q


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk", [(256, 8, 2), (128, 16, 4), (64, 3, 3)])
@pytest.mark.parametrize("T", [1, 300])
def test_probabilities_keep_their_bits(dtype, D, hq, hk, T):
    """As one prompt (many rows) and as single tokens (few rows): the same bound."""
    say("two keys", dtype, D, T)
    n = 300 if T > 1 else 40
    w, q = two_keys(n, hq, hk, D, dtype, D + T)
    if T == 1:
        w.tables = w.tables.repeat(n, 1)
        cu, ctx = None, [n] * n
    else:
        cu, ctx = [0, n], [n]
    out, lse = mr.attend_kv8(q.cuda(), None if cu is None else i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
    o, z, spread, amp = ref.attend(q, None, [2] * n, w.tables[:1].tolist() * n, w.kc, w.vc, w.ks, w.vs)
    assert bool((o.abs() < spread / 32).any())
    first = 2 if cu else 0  # a prompt's first rows do not see both
    within(out.cpu().double()[first:], lse.cpu().double()[first:], *(x[first:] for x in (o, z, spread, amp)), dtype, 4, 2, (dtype, D, T))
