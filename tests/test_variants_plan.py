"""Which variant of the state and pass kernels a problem takes (CPU)."""
import _plan


def test_heads_per_workgroup():
    """One head where the workgroups fit the GPU once, more where that saves a round, three for layers."""
    assert _plan.bwd_heads(2, 530, 4, 2) == 1 and _plan.prompt_heads(131, 5, 24, 1) == 1
    assert _plan.bwd_heads(18, 70, 17, 1) == 2 and _plan.prompt_heads(1100, 36, 17, 1) == 2
    for heads in (24, 32, 64, 80):
        assert _plan.bwd_heads(8, 2048, heads, 1) == 3
    assert _plan.prompt_heads(16384, 24, 24, 1) == 3 and _plan.prompt_heads(32769, 1, 24, 2) == 3


def test_chunks_ahead():
    assert _plan.prompt_ahead(32769, 1, 24, 64) == 16 and _plan.prompt_ahead(16384, 24, 24, 128) == 4
    assert _plan.prompt_ahead(5000, 1, 2, 64) == 16 and _plan.prompt_ahead(5000, 30, 2, 64) == 4
