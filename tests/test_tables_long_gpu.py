"""The step's tables of one long prompt among more requests than workgroups, with a
padded tail, against the oracle."""
import pytest

from test_tables_gpu import case, dev, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,at,tokens", [(300, 299, 8192), (513, 0, 8192), (600, 311, 30001),
                                         (1500, 1499, 9000)])
@pytest.mark.parametrize("spare", [-3, 7])
def test_a_long_prompt_among_many(B, at, tokens, spare, dev):
    new, ctx = [b % 3 for b in range(B)], [(37 * b) % 900 for b in range(B)]
    new[at], ctx[at] = tokens, 77
    run(case(new, ctx, 240, pad=5000, spare=spare, seed=B), dev)
