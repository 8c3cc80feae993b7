"""Which form of the decode with shared prefixes a plan takes, read from its
workspace: fp32 rows of 512 dims and their log-sum-exps for two pieces a part and
every unit, and 16 bytes for every unit and one more."""
import pytest

import fp4_kv_cache_sparse_gb300 as mla
from fp4_kv_cache_sparse_gb300 import build as lib_build


@pytest.fixture(scope="module", autouse=True)
def built():
    lib_build.build()


def planned(p, num_sms=152):
    """(rows of a unit, parts): 16, 32 or 64 rows on single SMs, 128 on pairs of them."""
    all_rows, rows = p.batch * p.seq_len_q * p.h_q, p.seq_len_q * p.h_q
    found = []
    for nr, parts in ((16, num_sms), (32, num_sms), (64, num_sms), (128, num_sms // 2)):
        units = p.batch * -(-rows // nr) + all_rows // nr + p.groups
        if (2 * parts + units) * nr * (512 + 1) * 4 + (units + 1) * 16 == mla.paged_shared_plan(p, num_sms)[1]:
            found.append((nr, parts))
    assert len(found) == 1
    return found[0]


def problem(groups, sequences, h, prefix_pages, s=1, pages=4):
    batch = groups * sequences
    return mla.PagedSharedProblem.make(batch, s, h, pages, prefix_pages, 1 << 20, groups=groups)


@pytest.mark.parametrize("groups,sequences,h,prefix_pages", [
    (40, 3, 16, 1024), (24, 3, 16, 1024), (30, 3, 16, 1024), (60, 3, 16, 1024), (64, 3, 16, 1024), (20, 4, 16, 1024),
    (76, 4, 16, 256), (152, 4, 16, 128),
])
def test_many_small_groups_stay_on_single_sms(groups, sequences, h, prefix_pages):
    """A group of up to 64 rows is one unit in either form, and a pair's takes longer."""
    assert planned(problem(groups, sequences, h, prefix_pages)) == (64, 152)


@pytest.mark.parametrize("groups,sequences,h,prefix_pages", [
    (1, 64, 128, 256), (10, 5, 40, 1024), (10, 5, 40, 512), (8, 8, 16, 1024), (4, 16, 16, 1024), (16, 1, 128, 512),
    (33, 1, 100, 256),
])
def test_groups_of_many_rows_go_by_pairs(groups, sequences, h, prefix_pages):
    assert planned(problem(groups, sequences, h, prefix_pages)) == (128, 76)


@pytest.mark.parametrize("num_sms,form", [
    (1, (64, 1)), (2, (128, 1)), (3, (64, 3)),           # a pair is two thirds of three SMs
    (5, (128, 2)), (40, (128, 20)), (151, (128, 75)),
])
def test_pairs_of_any_number_of_sms(num_sms, form):
    assert planned(problem(1, 64, 128, 256), num_sms) == form


def test_few_rows_and_short_prefixes():
    assert planned(problem(1, 8, 16, 64)) == (16, 152)
    assert planned(problem(1, 1, 16, 1024)) == (16, 152)
    assert planned(problem(1, 1, 24, 1024)) == (32, 152)
    assert planned(problem(3, 31, 24, 141, s=2, pages=11))[0] in (64, 128)


@pytest.mark.parametrize("groups", [9, 64, 8192])
def test_groups_past_the_sequences_are_empty(groups):
    """Room for more prefixes than there are sequences changes nothing about the units' rows."""
    for h, prefix_pages in ((128, 64), (48, 512), (128, 512)):
        p = mla.PagedSharedProblem.make(8, 1, h, 4, prefix_pages, 1 << 20, groups=groups)
        assert planned(p) == planned(mla.PagedSharedProblem.make(8, 1, h, 4, prefix_pages, 1 << 20, groups=8))
