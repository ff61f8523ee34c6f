"""The bounds that the 8-bit decode attention is held to on the GPU (no GPU):
its documented roundings stay inside them, coarser ones do not."""
import pytest

import kv8_bounds as N
import kv8_testlib as K


def worst(inputs, code, out, **coarser):
    """The largest error over tolerance of the roundings of q and P alone."""
    kv, q, scale = inputs
    top = 0.0
    for s, qh, k, v, tail in N.heads(kv, q):
        want, tol = N.tolerance(qh, k, v, tail, scale, code, out)
        got = N.roundings(qh, k, v, tail, scale, code, **coarser)
        if out == "bf16":
            got = got.float().bfloat16().double()
        top = max(top, float(((got - want).abs() / tol).max()))
    return top


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("peak", [64.0, 300.0])
def test_query_digits(out, peak):
    assert worst(N.outlier(K.INT8, peak, "cpu"), K.INT8, out) <= 1
    assert worst(N.outlier(K.INT8, peak, "cpu"), K.INT8, out, digits=2) > 1.5
    assert worst(N.outlier(K.E4M3, peak, "cpu"), K.E4M3, out) <= 1


@pytest.mark.parametrize("code", [K.E4M3, K.INT8])
def test_terms_of_p(code):
    stored, tail = N.one_channel(code, True, "cpu"), N.one_channel(code, False, "cpu")
    assert worst(stored, code, "f32") <= 1 and worst(tail, code, "f32") <= 1
    assert worst(stored, code, "f32", terms=1) > 1.5
    assert worst(tail, code, "f32", tail_terms=2) > 1.5
