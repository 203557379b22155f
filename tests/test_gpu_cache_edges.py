"""The paged-cache operators at the edges of what their header allows (needs a
GB300): rows without any score, outputs made on another stream, weights of
large scores, signed zeros, short rows in large objects, sums of the longest
sequence."""
import numpy as np
import pytest
import torch

from test_gpu_cache import attend_inputs, check_attend, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


# ---------------------------------------------------------------- rows without a score above -infinity

# heads, page, lens, sequences that lose every score; the blocks and the join that the batch's plan gives them
NOTHING = [
    ((12, 2, 128), 32, [100], [0]),                                          # a block a segment, no join
    ((12, 2, 128), 16, [15, 1], [1]),                                        # one position
    ((12, 2, 128), 16, [1000, 40], [0]),                                     # 8 blocks a segment, joined by the last
    ((14, 2, 64), 16, [20000], [0]),                                         # more than 24 parts: the join kernel
    ((16, 1, 128), 64, [9000, 77], [0, 1]),                                  # wide groups
    ((4, 4, 64), 16, [1 + 7 * i % 62 for i in range(300)], [0, 5, 123, 299]),  # a warp a segment
]


@pytest.mark.parametrize("how", ["pages", "scores"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,page,lens,gone", NOTHING)
def test_attend_without_a_score_gives_zeros(sf, heads, page, lens, gone, dtype, how):
    """Every page out of range (reported), or every score -infinity: zeros, and
    weights as they were; the other sequences of the batch are not affected."""
    a = attend_inputs(sf, heads, dtype, page, lens, seed=30)
    table = a["table"].copy()
    for s in gone:
        pages = -(-lens[s] // page)
        if how == "pages":
            a["table"][s, :pages] = -1
        else:
            a["q"][s] = a["q"][s].abs() + 0.1
            for c in range(pages):
                a["k"][table[s, c], :min(page, lens[s] - c * page)] = -float("inf")
    w_out = torch.full_like(a["w"], -3.0)
    calls = [a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights=a["w"], weights_out=w_out)]
    if how == "pages":
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "page" in str(e.value)
    calls.append(a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens)))
    torch.cuda.synchronize()
    for out in calls:
        for s in gone:
            assert not out[s].any(), s
    for s in gone:
        assert torch.equal(w_out[s, :, :lens[s]], a["w"][s, :, :lens[s]])
    rest = [s for s in range(len(lens)) if s not in gone]
    check_attend(heads, dtype, page, a, calls[0], w_out, w_in=a["w"], seqs=rest)
    check_attend(heads, dtype, page, a, calls[1], None, seqs=rest)
    a["c"].close()
