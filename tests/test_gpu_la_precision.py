"""The bf16 outputs of linear attention (o, dq, dk, dv) are as exact as one rounding of the 64-bit result.

Bound: the weighted scores and the boundary states go into the products in two bf16 terms each. A residual of a bf16
rounding is at most 2^-9 of the value and its own rounding at most 2^-9 of that, so a term pair is off by at most 2^-18, a
sum over them by at most 2^-18 of the sum of magnitudes: well under 2^-13 of an output's norm even where the terms
cancel to 1/32. One rounding to bf16 is off by about 1.6e-3 > 2^-10 in the same norm; errors before it that are eight times smaller
add at most 1/128 to it in the root of squares, so 1.01 times the error of the rounded 64-bit result bounds the
output's, where a second rounding of the same size would give 1.4."""
import pytest
import torch

import layer_reference as ref
from test_gpu_la import inputs, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


def check(got, want, names):
    for n in names:
        once = ref.rel(want[n].to(torch.bfloat16), want[n])
        assert ref.rel(got[n], want[n]) <= 1.01 * once, (n, ref.rel(got[n], want[n]), once)


CASES = [dict(B=2, T=100, Hqk=2, Hv=2, dk=128, dv=128, seed=1, h0=False),     # one chunk: the scores alone
         dict(B=1, T=1, Hqk=2, Hv=2, dk=128, dv=128, seed=2),                # one token: the state and one score
         dict(B=1, T=700, Hqk=2, Hv=2, dk=128, dv=64, seed=3, g_mean=8.0),    # the states of many chunks
         dict(B=1, T=0, Hqk=1, Hv=3, dk=64, dv=128, seed=4, lens=[5, 300, 0, 131]),
         dict(B=1, T=2100, Hqk=1, Hv=1, dk=64, dv=64, seed=5, head=True)]     # split walks


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c['T']}_dk{c['dk']}_dv{c['dv']}")
def test_one_rounding(gdn, case):
    x, gr = inputs(**case)
    o, _ = run_fwd(gdn, x, 0.7)
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), 0.7, gr["dout"], gr["dhT"])
    check(dict(o=o, **run_bwd(gdn, x, gr, 0.7)), want, ("o", "dq", "dk", "dv"))
