"""What SpecFold.verify refuses before it reaches the library (CPU)."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


@pytest.fixture
def ctx(sf):
    """A SpecFold without a context: calls that the binding lets through come back
    as the library's refusal of a null one."""
    c = sf.SpecFold.__new__(sf.SpecFold)
    c.shapes = sf.SfShapes(2, 128, 4, 2, 64, 256, sf.SF_F32, 1e-6, 1e4, 8, 2, 3, 64)
    c.ctx = None
    return c


def _args():
    hidden, prefix = torch.zeros(2, 3, 8, 128), torch.zeros(2, 2, 48, 2, 64)
    return dict(hidden=hidden, parent=np.array([[-1, 0, 0]] * 2), prefix_k=prefix, prefix_v=prefix.clone(), delta=0.1,
                out=torch.zeros_like(hidden), want_masks=False, stream=0)


def _reaches_the_library(sf, ctx, args):
    with pytest.raises(sf.SpecFoldError) as e:
        ctx.verify(**args)
    assert e.value.status == sf.SF_ERR_INVALID_ARG


def test_dense_prefixes_pass(sf, ctx):
    _reaches_the_library(sf, ctx, _args())
    _reaches_the_library(sf, ctx, dict(_args(), prefix_k=None, prefix_v=None))
    # the prefix an eviction left, copied into a buffer of its own length
    a = _args()
    short = {n: a[n][:, :, :32].contiguous() for n in ("prefix_k", "prefix_v")}
    _reaches_the_library(sf, ctx, dict(a, **short))
    # flattened heads, and a buffer with more layers than the context
    _reaches_the_library(sf, ctx, dict(a, prefix_k=a["prefix_k"].flatten(3)))
    _reaches_the_library(sf, ctx, dict(a, prefix_v=torch.zeros(3, 2, 48, 2, 64)))
    empty = torch.zeros(2, 2, 0, 2, 64)
    _reaches_the_library(sf, ctx, dict(a, prefix_k=empty, prefix_v=empty))


@pytest.mark.parametrize("name,change", [
    ("prefix_k", lambda t: t[:, :, :32]), ("prefix_v", lambda t: t[:, :, :32]), ("hidden", lambda t: t[..., ::2]),
    ("out", lambda t: t.transpose(1, 2)), ("prefix_k", lambda t: t[0]), ("prefix_k", lambda t: t[:1]),
    ("prefix_v", lambda t: t[:, :1].contiguous()), ("prefix_v", lambda t: t[:, :, :32].contiguous()),
    ("prefix_k", lambda t: t[..., :32].contiguous()), ("prefix_v", lambda t: t[:, :, :0].contiguous())])
def test_other_layouts_are_refused(ctx, name, change):
    a = _args()
    a[name] = change(a[name])
    if name == "prefix_k" and a[name].dim() == 5 and a[name].shape[2] == 32:
        a["prefix_v"] = change(a["prefix_v"])          # both halves alike: only the strides are wrong
    with pytest.raises(ValueError, match=name if name != "prefix_k" else "prefix_"):
        ctx.verify(**a)
