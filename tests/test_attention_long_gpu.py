"""The attention over prompts and its gradients where the other tests do not reach: calls of several
thousand tokens with 16 query and 4 kv heads of 128 (jobs from a list, long loops), and both sides
of the row counts at which the arithmetic changes (512 for the forward's maxima, 4096 for the
gradients' second bf16 terms).

Tolerances: those of the short tests (test_attention_prefill_gpu, test_attention_backward_gpu), whose
main term is 2^-8 of a sum of magnitudes; an fp32 sum of n terms adds n 2^-24 of that sum, which is
n 2^-16 of the main term, so they are taken 1 + n 2^-16 times.

In norm, where all terms are of one size and their signs random: rounding the probabilities (or P
and dS) moves a result by as much as rounding the result itself does, together sqrt(2) times that;
as much again is room for terms that are not of one size: twice the result's own rounding."""
import pytest
import torch

from test_attention_backward_gpu import formula as gradients
from test_attention_backward_gpu import step
from test_attention_prefill_gpu import cu, formula, inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def each(lens, H, kv):
    """Slices: a sequence's tokens, a kv head's query heads, the kv head."""
    at = 0
    for n in lens:
        for h in range(kv if n else 0):
            yield slice(at, at + n), slice(h * (H // kv), (h + 1) * (H // kv)), slice(h, h + 1)
        at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[6000], [3500, 1, 0, 2600, 700, 130]])
def test_thousands_of_tokens(gdn_lib, lens, d):
    gdn, H, kv = gdn_lib, 16, 4
    T = sum(lens)
    q, k, v = inputs(T, T, H, kv, d, seed=T)
    out, lse, dout, got = step(gdn, q, k, v, cu(lens))
    for t, qh, h in each(lens, H, kv):
        n = t.stop - t.start
        o, want, A, size = formula(q[t, qh], k[t, h], v[t, h], d ** -0.5)
        tol = (2.0 ** -8 * 1.01 * (o.abs() + A) + A * (2.0 ** -16 * (1 + size))[..., None]) * \
            (1 + n * 2.0 ** -16)
        assert ((out[t, qh].double().transpose(0, 1) - o).abs() <= tol).all(), (n, h)
        assert ((lse[t, qh].double().t() - want).abs() <= 2.0 ** -16 * (1 + size) + n * 2.0 ** -24).all()
        del o, want, A, size, tol
        want = gradients(q[t, qh], k[t, h], v[t, h], out[t, qh], lse[t, qh], dout[t, qh], d ** -0.5)
        for (g, tol), name, heads in zip(want, ("dq", "dk", "dv"), (qh, h, h)):
            off = (got[name][t, heads].double() - g).abs()
            assert (off <= tol * (1 + n * (H // kv) * 2.0 ** -16)).all(), (name, n, h)
    assert gdn.device_status() == 0


def rounding(x):
    return (x.to(BF16).double() - x).norm()


@pytest.mark.parametrize("d,kv", [(64, 2), (128, 1)])
@pytest.mark.parametrize("n", [100, 127, 128, 129, 300, 1023, 1024, 1025, 1500])
def test_norms_on_both_sides_of_the_row_counts(gdn_lib, n, d, kv):
    """4 n rows: 512 are at n = 128, 4096 at n = 1024."""
    q, k, v = inputs(n, n, 4, kv, d, seed=n)
    out, lse, dout, got = step(gdn_lib, q, k, v, None)
    o = formula(q, k, v, d ** -0.5)[0]
    assert (out.double().transpose(0, 1) - o).norm() <= 2 * rounding(o)
    want = gradients(q, k, v, out, lse, dout, d ** -0.5)
    for (g, _), name in zip(want, ("dq", "dk", "dv")):
        off = (got[name].double() - g).norm()
        assert off <= (1.125 if 4 * n < 4096 else 2) * rounding(g), name
    assert gdn_lib.device_status() == 0
