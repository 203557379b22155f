"""Outputs that SpecFold.verify and Head.verify make themselves, on a stream that
is not the current one (needs a GB300)."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


def _late(numel, dtype):
    """A block that is free again, but that the current stream, asleep for some
    100 ms, has still to copy: the copy, the block's address and its bytes."""
    block = torch.full((numel,), 7, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    return block.clone(), block.data_ptr(), block.numel() * block.element_size()


@pytest.mark.parametrize("by", ["stream", "handle"])
def test_outputs_come_from_the_memory_of_their_stream(by):
    import sparse_reuse_gb300 as sf
    cfg = synth.CONFIGS["tiny"].with_(n_layers=2, n_drafts=4, tree="random")
    wl = synth.make_workload(cfg, 5, device="cuda")
    gain, w_lm = synth.make_head_weights(cfg, 1024, 0, device="cuda")
    tok = torch.from_numpy(wl.tokens.astype(np.int32)).to("cuda")
    ctx = sf.from_config(cfg, wl.weights)
    head = sf.Head(d_model=cfg.d_model, vocab=1024, dtype=cfg.dtype, max_rows=cfg.rows, final_norm=gain, w_lm=w_lm,
                   rms_eps=cfg.rms_eps)
    want = ctx.verify(wl.hidden, wl.parents, wl.prefix_k, wl.prefix_v, 0.1)
    want = [*want, *head.verify(want[0], tok, wl.parents)]
    ctx.sync()
    want = [t.clone() for t in want]
    st = torch.cuda.Stream()
    stream = st if by == "stream" else st.cuda_stream
    shapes = [(t.numel(), t.dtype) for t in want]
    late = [_late(*x) for x in shapes[:4]]
    got = list(ctx.verify(wl.hidden, wl.parents, wl.prefix_k, wl.prefix_v, 0.1, stream=stream))
    late += [_late(*x) for x in shapes[4:]]
    got += head.verify(got[0], tok, wl.parents, stream=stream)
    for t in got:
        for _, address, size in late:
            assert t.data_ptr() + t.numel() * t.element_size() <= address or t.data_ptr() >= address + size
    ctx.sync(st)
    torch.cuda.synchronize()
    assert all(bool((copy == 7).all()) for copy, _, _ in late)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    head.close()
    ctx.close()


def test_the_default_stream_by_its_handle():
    """Handle 0 names the default stream, whichever is current."""
    import sparse_reuse_gb300 as sf
    cfg = synth.CONFIGS["tiny"].with_(n_layers=2)
    wl = synth.make_workload(cfg, 6, device="cuda")
    ctx = sf.from_config(cfg, wl.weights)
    want = [t.clone() for t in ctx.verify(wl.hidden, wl.parents, wl.prefix_k, wl.prefix_v, 0.1)]
    ctx.sync()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for stream in (0, torch.cuda.default_stream()):
            got = ctx.verify(wl.hidden, wl.parents, wl.prefix_k, wl.prefix_v, 0.1, stream=stream)
            ctx.sync(stream)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    ctx.close()
