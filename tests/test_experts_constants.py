"""The limits of the layer of experts, as the header, the binding and the library know them."""
import re

import pytest

import rotated_bit_linear_amd as rbl


@pytest.mark.parametrize("name", ["CR_MAX_EXPERTS", "CR_MAX_CHOICES", "CR_MAX_EXPERT_GROUPS", "CR_PLAN_SLOTS_IN_PLACE"])
def test_header_and_binding(name):
    assert int(re.search(rf"#define {name} (\d+)", open(rbl.HEADER).read()).group(1)) == getattr(rbl, name)


@pytest.mark.parametrize("E", [1, 64, 512])
@pytest.mark.parametrize("k", [1, 8, 32])
def test_a_plan_needs_a_workspace_from_there_on(E, k):
    T = rbl.CR_PLAN_SLOTS_IN_PLACE // k
    assert rbl.cr_experts_plan_workspace_bytes(T, k, E) == 0
    assert rbl.cr_experts_plan_workspace_bytes(T + 1, k, E) > 0
