"""Both forms of the decode with shared prefixes, each where the plan is known to
take it; against attention in 64 bits, with the tolerances of
test_gpu_paged_shared.py."""
import pytest

from test_gpu_paged_shared import Shared
from test_shared_plan import planned

pytestmark = pytest.mark.gpu


def run(c, form, num_sms=0):
    assert planned(c.shared_problem(), num_sms or 152) == form
    outs = [c.run_shared(num_sms=num_sms or 152) for _ in range(2)]
    for out, lse, err in outs:
        assert err == 0
        c.check_shared(out, lse)
    assert outs[0][0].equal(outs[1][0]) and outs[0][1].equal(outs[1][1])


@pytest.mark.parametrize("num_sms,form", [(0, (128, 76)), (152, (128, 76)), (15, (128, 7)), (2, (128, 1))])
def test_one_block_of_rows_over_many_pairs(num_sms, form):
    """128 rows over 20,000 tokens: cut into a piece for each pair, and merged."""
    run(Shared([70, 3], 1, 64, [0, 2], [20001], max_prefix_pages=9000, seed=1), form, num_sms)


@pytest.mark.parametrize("s,h", [(1, 40), (2, 64), (1, 128)])
def test_pairs_over_groups_of_all_sizes(s, h):
    c = Shared([5, 200, 0, 64, 1, 128, 513, 9, 63, 65, 300, 31], s, h, [0, 1, 7, 7, 11], [700, 2049, 64, 1000],
               max_prefix_pages=9000, seed=s * h)
    run(c, (128, 76))


def test_many_small_groups_on_single_sms():
    lens = [(37 * b) % 190 for b in range(120)]
    plens = [(531 * g) % 2100 for g in range(40)]
    run(Shared(lens, 1, 16, list(range(0, 121, 3)), plens, max_prefix_pages=1024, seed=3), (64, 152))


@pytest.mark.parametrize("prefix_pages,form", [(64, (64, 152)), (9000, (128, 76))])
def test_room_for_more_groups_than_sequences(prefix_pages, form):
    """Eight sequences in groups of two; the other 60 groups are empty."""
    start = [0, 2, 4, 6] + [8] * 61
    plens = [300, 0, 4000, 129] + [100 * g for g in range(10)] + [0] * 50
    run(Shared([30, 200, 0, 64, 1, 128, 77, 9], 1, 128, start, plens, max_prefix_pages=prefix_pages, seed=4), form)
