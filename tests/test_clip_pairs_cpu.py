"""Which output tensor takes which gradient: dicts by name, lists by place, shapes compared (no GPU needed:
the pairing comes before the tensors are looked at)."""
import pytest
import torch

import sparse_mixture_experts_14_b200 as moe


def _t(*shape):
    return torch.zeros(*shape)


def _is(got, want):
    assert len(got) == len(want) and all(a is b for a, b in zip(got, want))


def test_dicts_are_paired_by_name():
    g = dict(dx=_t(2), dWg=_t(3), dW1=_t(4), dW3=_t(4), dW2=_t(4))
    o = dict(dW2=_t(4), dW3=_t(4), dWg=_t(3), dW1=_t(4))
    grads, outs = moe._grads_and_outs(g, o)
    _is(grads, [g[n] for n in ("dWg", "dW1", "dW3", "dW2")])
    _is(outs, [o[n] for n in ("dWg", "dW1", "dW3", "dW2")])
    g["dW3"] = None
    grads, outs = moe._grads_and_outs(g, dict(o, dx=_t(2)))
    _is(outs, [o[n] for n in ("dWg", "dW1", "dW2")])
    del o["dW1"]
    with pytest.raises(ValueError, match="dW1"):
        moe._grads_and_outs(g, o)
    with pytest.raises(ValueError, match="dW1"):
        moe.moe_clip_grads(g, 1.0, out=o)
    with pytest.raises(TypeError):
        moe.moe_clip_grads([_t(3), _t(4)], 1.0, out=dict(a=_t(3), b=_t(4)))


def test_lists_are_paired_by_place():
    a, b, p, q, r = (_t(4) for _ in range(5))
    _is(moe._grads_and_outs([a, None, b], [p, q, r])[1], [p, r])
    _is(moe._grads_and_outs([a, None, b], [p, None, r])[1], [p, r])
    _is(moe._grads_and_outs([a, None, b], [p, q])[1], [p, q])
    _is(moe._grads_and_outs((g for g in (a, b)), iter([p, q]))[1], [p, q])
    _is(moe._grads_and_outs(dict(dx=r, dWg=a, dW1=b), [p, q])[1], [p, q])
    with pytest.raises(ValueError):
        moe.moe_clip_grads([None, a], 1.0, out=[p, None])     # p stands beside no gradient
    for out in ([p], [p, None, q], [p, q, r, r], [None, p]):
        with pytest.raises(ValueError):
            moe._grads_and_outs([a, b], out)
