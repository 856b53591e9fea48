"""The bound on d_W of up to 64 bf16 rows, on the CPU: g in two bf16 terms keeps it,
in one it does not."""
import pytest
import torch

import vocab_ref as R
from vocab_few_ref import TwoTerms


@pytest.mark.parametrize("n", [1, 7, 33, 64])
@pytest.mark.parametrize("d", [8, 64, 130])
def test_one_term_is_not_enough(n, d):
    t = R.problem(n + d, n, d, 300, "bf16")
    ref = TwoTerms(t["h"], t["w"], "bf16", target=t["target"])
    want, err = ref.d_w(t["d_loss"])
    g = ref.factors(t["d_loss"])[0]
    one = g.bfloat16().double()
    two = one + (g - one).bfloat16().double()
    R.check("two terms", two.t() @ ref.h, want, err)
    with pytest.raises(AssertionError, match="outside"):
        R.check("one term", one.t() @ ref.h, want, err)
