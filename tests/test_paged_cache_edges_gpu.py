"""GPU tests of the paged cache's edges: page pools that hold what is no page, calls that overlap,
and chains of calls with nothing between them."""
import numpy as np
import pytest
import torch

import head_rank_attention_b200 as hra
from oracle import paged
from test_paged_cache_gpu import Plan, _plan_case

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- page plan
@pytest.mark.parametrize("B,page,wide,chunk,max_tokens,head", [
    (1, 32, 3, 90, 90, 0), (64, 64, 40, 1, 64, 77), (257, 96, 30, 50, 5000, 123456), (1024, 32, 16, 90, 65536, 1 << 33)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_refuses_pages_that_are_none_of_the_pool(B, page, wide, chunk, max_tokens, head, in_place):
    """The last page to be taken is -1, or one past the pool; behind the pages to be taken it does not matter."""
    lens, new, table, ring, free = _plan_case(B, B, page, wide, chunk, max_tokens, head=head)
    good = paged.page_plan(lens, new, table, ring, free, page, max_tokens)
    taken = good["free"][0] - free[0]
    assert good["status"] == [0, 0, 0, 0] and (taken > 0 or B == 64)
    for at, bad, code in ((taken - 1, -1, 6), (taken - 1, len(ring), 6), (0, -2 ** 31, 6), (taken, -1, 0)):
        if code and taken == 0:
            continue
        other = ring.copy()
        other[(free[0] + at) % len(ring)] = bad
        want = paged.page_plan(lens, new, table, other, free, page, max_tokens)
        assert want["status"][0] == code
        plan = Plan(lens, new, table, other, free, page, max_tokens, in_place=in_place)
        hra.page_plan(plan.p)
        plan.check(want)
        if code:
            with pytest.raises(hra.HraError, match="no page of the pool") as e:
                hra.check_plan_status(plan.p)
            assert e.value.status == hra._binding.HRA_ERR_PLAN


def test_a_bad_page_given_back_is_not_handed_out():
    """Request 0 ends with a page that is none of the pool in its row; the page goes to the ring, and
    the step that would hand it to request 1 is refused, lengths and pool as they were."""
    case = ([40, 0], [-1, 32], np.array([[0, 9], [-1, -1]]), np.array([2, 3, -7, -7]), [0, 2])
    plan = Plan(*case, 32, 64, in_place=True)
    hra.page_plan(plan.p)
    hra.check_plan_status(plan.p)
    assert plan.free.tolist() == [1, 4] and plan.ring.tolist() == [2, 3, 0, 9] and plan.table.tolist()[1] == [2, -1]
    plan.new.copy_(torch.tensor([0, 32]))
    hra.page_plan(plan.p)
    plan.new.copy_(torch.tensor([64, 0]))
    hra.page_plan(plan.p)
    assert plan.status.tolist() == [6, 0, 3, 9] and plan.free.tolist() == [2, 4] and plan.lens.tolist() == [0, 64]
