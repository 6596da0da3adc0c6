"""What the paged kernels' sources must keep and no run can show (CPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "full_gqa_learned_b200", "csrc")


def step_source():
    return open(os.path.join(CSRC, "flint_paged_step.cu")).read()


def test_the_plan_shares_no_memory_with_the_tma_ring():
    """Threads read and write the plan's shared memory by plain accesses; bytes
    that TMA then writes would need a proxy fence between the two.  The plan has
    a region of its own, and a static_assert keeps it off the ring."""
    s = step_source()
    call = re.search(r"step_plan<NT>\(p, TL::tile, .*?\);", s, re.S).group(0)
    assert "reinterpret_cast<StepPlanSmem*>(smem + S::plan)" in call
    assert re.search(r"static_assert\(plan >= kStepStages \* kStepStage\b", s)
